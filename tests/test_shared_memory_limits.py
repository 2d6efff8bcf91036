"""Each kernel's limit of dynamic shared memory is the same whatever a call's
sizes: the limit is the function's, in all host threads, and a call that lowered
it would make another thread's launch fail.  The CUDA runtime's calls are
recorded by stand-ins, and nothing is launched (no GPU)."""
import collections
import os
import subprocess
import sys

from test_abi import ROOT, lib  # noqa: F401  (the built library)

STAND_INS = r"""
#include <cuda_runtime_api.h>
#include <stdio.h>
#include <string.h>
cudaError_t cudaFuncSetAttribute(const void* f, enum cudaFuncAttribute a, int v) {
  if (a == cudaFuncAttributeMaxDynamicSharedMemorySize) printf("limit %p %d\n", f, v);
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void** args) {
  printf("launch %p %d\n", f, (int)c->dynamicSmemBytes);
  return cudaSuccess;
}
cudaError_t cudaMemsetAsync(void* p, int v, size_t n, cudaStream_t s) { return cudaSuccess; }
cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
cudaError_t cudaGetLastError(void) { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, enum cudaDeviceAttr a, int d) { *v = 152; return cudaSuccess; }
static int encode(void) { return 0; }
cudaError_t cudaGetDriverEntryPointByVersion(const char* n, void** p, unsigned v, unsigned long long f,
                                             enum cudaDriverEntryPointQueryResult* r) {
  if (strcmp(n, "cuTensorMapEncodeTiled")) return cudaErrorInvalidValue;
  *p = (void*)encode;
  *r = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
"""

CALLS = """
import sys
sys.path[:0] = [ROOT, ROOT + '/tests']
import grad_row_online_gb300 as g
from test_linear_abi import _bwd, _embed_grad, _fwd
L = g.lib()
for dt in (0, 1):
    for N, K, V in [(1, 64, 100), (1, 4096, 200), (8, 64, 300), (8, 4096, 300), (16, 512, 99), (17, 64, 70), (17, 2048, 900),
                    (100, 640, 9000), (128, 4160, 5000), (129, 64, 256), (300, 64, 100), (300, 2048, 40000),
                    (5000, 8256, 3000)]:
        for sv in (K, K + 1):
            kw = dict(dt=dt, B=1, T=N, K=K, V=V, sb=N * K, st=K, sv=sv)
            assert _fwd(L, **kw, ent=1 << 20, stats=1 << 20) == 0
            assert _bwd(L, **kw, gsb=N * K, gst=K, gsv=K, wdt=dt) == 0
            assert _bwd(L, **kw, gsb=N * K, gst=K, gsv=K, wdt=0) == 0
    for N, V in [(1, 100), (100, 151936), (4096, 100), (4096, 151936), (4096, 1 << 28), (4097, 1000)]:
        assert _embed_grad(L, dt=dt, B=1, T=N, V=V, sb=N * 64, wdt=dt) == 0
"""


def test_a_kernels_limit_does_not_depend_on_the_call(lib, tmp_path):  # noqa: F811
    src, so = tmp_path / "stand_ins.c", tmp_path / "stand_ins.so"
    src.write_text(STAND_INS)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    subprocess.run(["gcc", "-shared", "-fPIC", "-O1", "-I" + os.path.join(cuda, "include"), str(src), "-o", str(so)], check=True)
    r = subprocess.run([sys.executable, "-c", CALLS.replace("ROOT", repr(ROOT))], capture_output=True, text=True,
                       env=dict(os.environ, LD_PRELOAD=str(so), CUDA_VISIBLE_DEVICES=""))
    assert r.returncode == 0, r.stderr[-2000:]
    limits, launches = collections.defaultdict(set), collections.defaultdict(set)
    for line in r.stdout.splitlines():
        kind, f, n = line.split()
        (limits if kind == "limit" else launches)[f].add(int(n))
    assert len(launches) > 20 and len(limits) > 10
    for f, n in launches.items():
        assert max(n) <= max(limits.get(f, {48 * 1024}))
    assert {f: sorted(n) for f, n in limits.items() if len(n) > 1} == {}
