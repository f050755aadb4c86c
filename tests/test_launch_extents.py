"""Launches at the largest documented sizes that a GPU of 288 GB holds (no GPU needed):
HIP takes fewer than 2^32 threads in a dimension, and this GPU up to 65536 workgroups in the
second one.  The library runs with stand-ins for the
runtime's calls, which note every launch instead of making it; no address is read."""
import ctypes
import json
import os
import subprocess
import sys

import pytest

import shared_matrix_expert_amd as em

RUNTIME = r"""
#include <hip/hip_runtime_api.h>
#include <cstring>
#include <vector>
static std::vector<unsigned long long> seen;
static dim3 grid, block;
extern "C" {
hipError_t hipGetDevice(int* d) { *d = 0; return hipSuccess; }
hipError_t hipGetLastError(void) { return hipSuccess; }
hipError_t hipGetDevicePropertiesR0600(hipDeviceProp_tR0600* p, int) {
    std::memset(p, 0, sizeof *p);
    std::strcpy(p->gcnArchName, "gfx950");
    return hipSuccess;
}
hipError_t __hipPushCallConfiguration(dim3 g, dim3 b, size_t, hipStream_t) { grid = g; block = b; return hipSuccess; }
hipError_t __hipPopCallConfiguration(dim3* g, dim3* b, size_t* shared, hipStream_t* s) {
    *g = grid; *b = block; *shared = 0; *s = nullptr;
    return hipSuccess;
}
hipError_t hipLaunchKernel(const void*, dim3 g, dim3 b, void**, size_t, hipStream_t) {
    for (unsigned v : {g.x, g.y, g.z, b.x, b.y, b.z}) seen.push_back(v);
    return hipSuccess;
}
size_t launches(unsigned long long* to, size_t most) {
    const size_t n = seen.size() < most ? seen.size() : most;
    std::memcpy(to, seen.data(), 8 * n);
    seen.clear();
    return n;
}
}
"""

BASE = 1 << 40                                                    # never read
FITS = 280 << 30


def norms():
    """(name, arguments) of the norm's calls at T and d on both sides of every row width."""
    for d in (8, 512, 520, 1024, 1032, 2048, 2056, 4096, 4104, 8192, 8200, 16384, 16392, 32768):
        T = min(1 << 25, (FITS // (2 * d)))
        yield "norm", dict(T=T, d=d)
        for dx in (False, True):
            yield "norm_backward", dict(T=min(T, FITS // ((6 if dx else 4) * d)), d=d, dx=dx)


def products():
    """(name, arguments) of the products': many rows, tokens, columns and matrices of them."""
    dims = []
    for M in (1, 8, 200, 1024):
        for N in (8, 72, 1032, 4096, 32768):
            for K in (32, 512, 4096, 16384, 32768):
                for R in (2000, 1 << 18, 1 << 25):
                    for T in (1 << 10, 1 << 20):
                        dims.append((T, R, M, N, K))
    for T, R, M, N, K in dims:
        if 2 * (T * K + R * N + M * N * K) <= FITS:
            yield "dense_product", dict(T=T, R=R, M=M, N=N, K=K)
        if 2 * (T * K + R * N + M * N * K) <= FITS:
            yield "dense_backward", dict(T=T, R=R, M=M, N=N, K=K, tokens=True)
        if 2 * (R * K + R * N + M * N * K) <= FITS:
            yield "dense_backward", dict(T=T, R=R, M=M, N=N, K=K, tokens=False)
        if 2 * (T * K + R * N + 2 * M * N * K) <= FITS:
            yield "dense_backward_dw", dict(T=T, R=R, M=M, N=N, K=K)
        if 2 * (T * K + R * N) + M * N * K // 2 <= FITS:
            yield "packed_product", dict(T=T, R=R, M=M, N=N, K=K)
            yield "packed_product", dict(T=T, R=R, M=M, N=N - 1, K=K)
        if K % 128 == 0 and T * K + 2 * R * N + M * N * K // 2 <= FITS:
            yield "mx_product_coded", dict(T=T, R=R, M=M, N=N, K=K)


def launch(lib, name, a):
    """Status of the call."""
    if name == "norm":
        g = em.CNormArgs(T=a["T"], d=a["d"], eps=1e-5, x=BASE, x_stride=a["d"], gain=BASE, rstd=BASE)
        return lib.edge_moe_norm(ctypes.byref(g), None)
    if name == "norm_backward":
        g = em.CNormGrad(T=a["T"], d=a["d"], x=BASE, x_stride=a["d"], gain=BASE, rstd=BASE, dy=BASE, dy_stride=a["d"],
                         dx=BASE if a["dx"] else None, dx_stride=a["d"], dgain=BASE)
        return lib.edge_moe_norm_backward(ctypes.byref(g), BASE, 1 << 62, None)
    T, R, M, N, K = (a[n] for n in ("T", "R", "M", "N", "K"))
    if name == "packed_product":
        return lib.edge_moe_packed_product(ctypes.byref(em.CPackedDims(T, R, M, N, K, 32)), BASE, K, BASE, BASE, BASE, BASE, 0, BASE, N, BASE,
                                           1 << 62, None)
    if name == "mx_product_coded":
        return lib.edge_moe_mx_product_coded(ctypes.byref(em.CMxDims(T, R, M, N, K, em.MX_FP8)), BASE, BASE, BASE, BASE, BASE, BASE, BASE, N, None)
    dims = ctypes.byref(em.CDenseDims(T, R, M, N, K))
    if name == "dense_product":
        return lib.edge_moe_dense_product(dims, BASE, K, BASE, BASE, BASE, 0, BASE, N, BASE, 1 << 62, None)
    g = em.CDenseGrad(dy=BASE, dy_stride=N, row_src=BASE, offsets=BASE)
    if name == "dense_backward":
        g.w, g.dx, g.dx_stride = BASE, BASE, K
        if a["tokens"]:
            g.token_rows, g.per_token = BASE, 8
    else:
        g.x, g.x_stride, g.dw = BASE, K, BASE
    return lib.edge_moe_dense_product_backward(dims, ctypes.byref(g), BASE, 1 << 62, None)


def run(runtime, cases):
    """Every case's status and launches (grid and block sizes)."""
    ctypes.CDLL(runtime, ctypes.RTLD_GLOBAL)                      # found before the library's own runtime
    lib, rt = ctypes.CDLL(em.LIB_PATH), ctypes.CDLL(runtime)
    vp, i64, sz, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
    lib.edge_moe_norm.argtypes = [vp, vp]
    lib.edge_moe_norm_backward.argtypes = [vp, vp, sz, vp]
    lib.edge_moe_dense_product.argtypes = [vp, vp, i64, vp, vp, vp, i32, vp, i64, vp, sz, vp]
    lib.edge_moe_dense_product_backward.argtypes = [vp, vp, vp, sz, vp]
    lib.edge_moe_packed_product.argtypes = [vp, vp, i64, vp, vp, vp, vp, i32, vp, i64, vp, sz, vp]
    lib.edge_moe_mx_product_coded.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i64, vp]
    rt.launches.restype, rt.launches.argtypes = sz, [vp, sz]
    out, buf = [], (ctypes.c_ulonglong * 6000)()
    for name, a in cases:
        st = launch(lib, name, a)
        n = rt.launches(buf, len(buf))
        out.append((st, [buf[i:i + 6] for i in range(0, n, 6)]))
    return out


@pytest.fixture(scope="module")
def runtime(tmp_path_factory):
    d = tmp_path_factory.mktemp("runtime")
    src, so = d / "runtime.cpp", d / "libruntime.so"
    src.write_text(RUNTIME)
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", str(src), "-o", str(so)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return str(so)


@pytest.mark.parametrize("which", ["norms", "products"])
def test_launches_within_the_limits(runtime, which):
    cases = list(globals()[which]())
    r = subprocess.run([sys.executable, os.path.abspath(__file__), runtime], input=json.dumps(cases), capture_output=True, text=True,
                       env={**os.environ, "PYTHONPATH": os.path.dirname(em.HERE)})
    assert r.returncode == 0, r.stderr
    results = json.loads(r.stdout)
    assert len(results) == len(cases) and len(cases) > 40
    bad = []
    for (name, a), (status, launched) in zip(cases, results):
        ok = status == em.EDGE_MOE_OK and len(launched) > 0
        for gx, gy, gz, bx, by, bz in launched:
            ok &= 0 < gx * bx < 1 << 32 and 0 < gy <= 65536 and gz == bz == 1 and bx * by <= 1024
        if not ok:
            bad.append((name, a, status, launched))
    assert not bad, f"{len(bad)} of {len(cases)}: {bad[:8]}"


if __name__ == "__main__":
    print(json.dumps(run(sys.argv[1], json.load(sys.stdin))))
