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


TILES = """
static int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }
// the head's tiles of N tokens and V words, width K, as pairs of CTAs take them
static void tiles(int64_t N, int64_t K, int64_t V) {
  const int64_t row = 2 * 256 * up(K, 64) * 64, mt = up(N, 256), nt = up(V, 256);
  if (up(N, 128) * up(V, 64) > 0x7FFFFFFE) exit(2);  // (refused)
  const int mb = rows_together(row, mt);
  if (mb < 1 || mb > mt || (mb > 1 && mb * row > 32 << 20)) exit(3);
  // the first and the last tile, those around the ends of blocks, and some between
  for (int64_t i = 0; i < 4000; ++i) {
    int64_t u = i < 1000 ? i : i < 2000 ? mt * nt - 1 - (i - 1000) : i < 3000 ? (int64_t)mb * nt - 500 + (i - 2000)
                                                                              : mt * nt / 1000 * (i - 3000);
    if (u < 0 || u >= mt * nt) continue;
    const TilePlace p = tile_place((int)u, (int)mt, mb, (int)nt);
    if (p.row < 0 || p.row >= mt || p.col < 0 || p.col >= nt) exit(4);
    // the tiles before it: whole blocks, whole columns of this block, rows of this column
    const int64_t blk = p.row / mb, across = mt - blk * mb < mb ? mt - blk * mb : mb;
    if (blk * mb * nt + p.col * across + (p.row - blk * mb) != u) exit(5);
  }
}
int main() {
  const int64_t sizes[][3] = {SIZES};
  for (auto& s : sizes) tiles(s[0], s[1], s[2]);
  puts("ok");
}
"""


def test_every_tile_of_the_largest_vocabularies_has_its_place(tmp_path):
    sizes = [(129, 1, MOST), (129, 64, 1 << 30), (200, 8, (1 << 30) + 12345), (8192, 64, MOST // 2), (8000, 256, 1 << 24),
             (300, 1 << 20, 1 << 17), (MOST, 64, 64), (MOST // 2, 1, 100), (16384, 2048, 151936), (129, 64, 256)]
    assert run(tmp_path, TILES.replace("SIZES", ", ".join("{%d, %d, %d}" % s for s in sizes))) == "ok\n"
