"""The index arithmetic of the head and the embedding at their largest sizes,
compiled for the host with every signed overflow an error (no GPU)."""
import os
import subprocess

from grad_row_online_gb300 import _build

MOST = (1 << 31) - 1025  # tokens, words


def run(tmp_path, body):
    """The output of a program that includes the kernels' index arithmetic."""
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text('#include <stdio.h>\n#include <stdlib.h>\n#include "grpo_index.cuh"\nusing namespace grpo;\n' + body)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=signed-integer-overflow", "-fsanitize-undefined-trap-on-error",
                    "-I" + _build.CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stdout[-500:], r.stderr[-500:])
    return r.stdout


PARTS = """
// every token of N is in one part, in order
static void tokens(int N) {
  const int64_t chunk = sort_chunk(N), chunks = (N + chunk - 1) / chunk;
  if (chunk % kSortThreads || chunks > 256 || chunk > 0x7FFFFFFF || (N <= 4096 && chunks > 1)) exit(2);
  int next = 0;
  for (int c = 0; c < chunks; ++c)
    for (int w = 0; w < kSortWarps; ++w) {
      const SortPart p = sort_part((int)chunk, c, w, N);
      if (p.from < 0 || p.end > N) exit(3);
      if (p.from >= N) { if (p.end > p.from) exit(4); continue; }
      if (p.from != next || p.end <= p.from) exit(5);
      // the last index a round of 128 tokens forms
      if ((int64_t)p.from + ((int64_t)p.end - p.from + 127) / 128 * 128 + 127 > 0x7FFFFFFF) exit(6);
      next = p.end;
    }
  if (next != N) exit(7);
}
int main() {
  const int sizes[] = {SIZES};
  for (int N : sizes) tokens(N);
  puts("ok");
}
"""


def test_every_token_is_in_one_part_of_the_sort(tmp_path):
    near = [MOST - i for i in (0, 1, 511, 1023, 4096, 65535, 130047, 130048, 131071, 131072, 1 << 19, 1 << 20)]
    small = [1, 31, 32, 511, 512, 513, 4095, 4096, 4097, 2048 * 256, 2048 * 256 + 1, 999999, 65536 * 32767,
             (1 << 30) + 1, 255 * (1 << 23), 255 * (1 << 23) + 1]
    assert run(tmp_path, PARTS.replace("SIZES", ", ".join(map(str, near + small)))) == "ok\n"
