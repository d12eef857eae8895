"""What fp8_w4_experts launches, on the CPU: a stub of the library's launchers,
loaded before it, writes down their arguments in place of launching.  Kernels that
take the tokens' order (the copy of rows into it, and the products of many tokens)
run only where the same call has made it."""
import json
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

STUB = r'''
#include <cstdio>
#include "internal.h"
namespace fp8lin {
cudaError_t launch_expert_order(const int *, int64_t slots, int E, int, int *counts, int *offsets, int *position,
                                int *, int *, cudaStream_t, W4List *, int, int) {
  std::printf("order %lld %d %p %p %p\n", (long long)slots, E, (void *)counts, (void *)offsets, (void *)position);
  return cudaSuccess;
}
cudaError_t launch_rows_gather(const void *, int64_t, int64_t, int, int, int, const int *counts, const int *offsets,
                               const int *position, void *, cudaStream_t) {
  std::printf("gather %p %p %p\n", (void *)counts, (void *)offsets, (void *)position);
  return cudaSuccess;
}
cudaError_t launch_w4_product(W4Args a, const W4Plan &p, int lists, cudaStream_t) {
  std::printf("product %d %d %p %p %d %d\n", (int)p.wide, lists, (void *)a.counts, (void *)a.offsets, a.order != nullptr,
              a.lists != nullptr);
  return cudaSuccess;
}
cudaError_t launch_w4_join(const float *, const int *, const int *position, const float *, int64_t, int64_t, int, int,
                           int, void *, cudaStream_t) {
  std::printf("join %p\n", (void *)position);
  return cudaSuccess;
}
}  // namespace fp8lin
'''

SHAPES = [
    (1, 1, 17, 4096, 4096, 4096), (1, 2, 48, 4096, 4096, 4096), (1, 2, 64, 4096, 4096, 4096), (1, 1, 17, 256, 32768, 16),
    (1, 1, 17, 32, 32768, 256),
    (1, 4, 1000, 2048, 2048, 2048), (1, 3, 4, 96, 64, 48), (1, 8, 2, 4096, 14336, 4096), (1, 8, 8, 512, 512, 512),
    (1, 1, 1, 4096, 4096, 4096), (2, 1, 17, 4096, 4096, 4096), (64, 32, 4, 4096, 2048, 4096),
    (600, 8, 2, 4096, 14336, 4096)]

CHILD = r'''
import ctypes, json, sys
import fp8_mixed_precision_gb300 as fp
L, libc = fp.lib(), ctypes.CDLL(None)
A = 1 << 20  # never dereferenced
for T, E, k, K, F, N in json.loads(sys.argv[1]):
    b = ctypes.c_size_t()
    assert L.fp8_w4_experts_workspace_size(T, k, E, K, F, N, ctypes.byref(b)) == 0
    gu, dn = fp._W4(A, A, None, E, 2 * F, K, 128), fp._W4(A, A, None, E, N, F, 128)
    assert L.fp8_w4_experts(A, T, k, A, A, gu, dn, 0, A, A, b.value, None) == 0
    libc.printf(b"end\n")
libc.fflush(None)
'''


@pytest.fixture(scope="module")
def launches(tmp_path_factory):
    """The launches of each shape, as lists of words."""
    from fp8_mixed_precision_gb300 import build
    build.build()
    tmp = tmp_path_factory.mktemp("stub")
    (tmp / "stub.cpp").write_text(STUB)
    so = str(tmp / "stub.so")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I" + build.CSRC, "-I" + build.INCLUDE,
                    "-I" + os.path.join(build._cuda_home(), "include"), str(tmp / "stub.cpp"), "-o", so], check=True)
    r = subprocess.run([sys.executable, "-c", CHILD, json.dumps(SHAPES)], cwd=ROOT, capture_output=True, text=True,
                       env=dict(os.environ, LD_PRELOAD=so, PYTHONPATH=ROOT))
    assert r.returncode == 0, r.stderr[-2000:]
    parts = r.stdout.split("end\n")
    assert len(parts) == len(SHAPES) + 1
    return {s: [line.split() for line in p.splitlines()] for s, p in zip(SHAPES, parts)}


@pytest.mark.parametrize("T,E,k,K,F,N", SHAPES)
def test_order_comes_before_what_takes_it(launches, T, E, k, K, F, N):
    calls = launches[T, E, k, K, F, N]
    assert [c[0] for c in calls if c[0] in ("product", "join")] == ["product", "product", "join"]
    made = [c for c in calls if c[0] == "order"]
    assert len(made) <= 1 and (not made or calls[0] is made[0])
    counts, offsets, position = made[0][3:6] if made else ("(nil)",) * 3
    for c in calls:
        if c[0] == "gather":
            assert made and c[1:] == [counts, offsets, position]
        if c[0] == "product":
            wide, lists, at, ordered, listed = c[1] == "1", int(c[2]), c[3:5], c[5] == "1", c[6] == "1"
            assert made or not wide
            assert ordered == listed == bool(made) and at == [counts, offsets]
            assert lists == (min(E, T * k) if made else k) and lists <= 65535   # a dimension of the grid
        if c[0] == "join":
            assert c[1] == position
