"""CPU checks of the MXFP4 and routing entry points of the C ABI: arguments are
refused on the host, before the device is looked at."""
import ctypes
import os

import pytest

from quantized_moe_weight_amd import _lib

if not os.path.exists(_lib.LIB_PATH):
    pytest.skip("libpqmoe.so not built", allow_module_level=True)

PQ_OK, NULL, SHAPE, ALIGN, WORKSPACE = 0, -1, -2, -3, -4
FAKE = ctypes.c_void_p(1 << 20)          # non-null, 16-byte aligned; never dereferenced
MIS = ctypes.c_void_p((1 << 20) + 8)     # misaligned
NUL = ctypes.c_void_p(0)


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def test_quantise(lib):
    q = lib.pq_quantize_mxfp4
    assert q(NUL, 0, 1, 32, FAKE, FAKE, NUL) == NULL
    assert q(FAKE, 0, 1, 32, NUL, FAKE, NUL) == NULL
    assert q(FAKE, 0, 1, 32, FAKE, NUL, NUL) == NULL
    for rows, K in ((0, 32), (-1, 32), (1, 0), (1, 16), (1, 48), (1, -32)):
        assert q(FAKE, 1, rows, K, FAKE, FAKE, NUL) == SHAPE, (rows, K)
    assert q(MIS, 0, 1, 32, FAKE, FAKE, NUL) == ALIGN
    assert q(FAKE, 0, 1, 32, FAKE, MIS, NUL) == ALIGN
    d = lib.pq_dequantize_mxfp4
    assert d(NUL, FAKE, 1, 32, 0, FAKE, NUL) == NULL
    assert d(FAKE, FAKE, 1, 40, 0, FAKE, NUL) == SHAPE
    assert d(FAKE, MIS, 1, 32, 0, FAKE, NUL) == ALIGN


def test_gemv(lib):
    def g(x=FAKE, M=1, K=512, w=FAKE, s=FAKE, N=256, epi=0, y=FAKE):
        return lib.pq_gemv_mxfp4(x, M, K, w, s, N, epi, y, NUL)
    assert g(x=NUL) == NULL and g(w=NUL) == NULL and g(s=NUL) == NULL and g(y=NUL) == NULL
    for kw in (dict(M=0), dict(M=17), dict(K=16), dict(K=48), dict(K=0), dict(N=0), dict(epi=2), dict(epi=1, N=255),
               dict(M=16, K=4384), dict(M=1, K=69664), dict(K=65536, N=65536)):
        assert g(**kw) == SHAPE, kw
    assert g(x=MIS) == ALIGN and g(s=MIS) == ALIGN


def test_gemm(lib):
    def g(x=FAKE, M=64, K=512, w=FAKE, s=FAKE, N=256, epi=0, y=FAKE, ws=FAKE, wsn=1 << 30):
        return lib.pq_gemm_mxfp4(x, M, K, w, s, N, epi, y, ws, wsn, NUL)
    assert g(x=NUL) == NULL and g(y=NUL) == NULL
    for kw in (dict(M=0), dict(K=48), dict(K=0), dict(N=0), dict(epi=3), dict(epi=1, N=3), dict(K=65536, N=65536),
               dict(K=65536, M=65536)):
        assert g(**kw) == SHAPE, kw
    assert g(w=MIS) == ALIGN
    assert g(ws=NUL) == WORKSPACE and g(wsn=1000) == WORKSPACE and g(ws=MIS) == ALIGN
    need = lib.pq_gemm_mxfp4_workspace(64, 512, 256, 0)
    assert need >= 64 * 256 + 64 * 16 and g(wsn=need - 1) == WORKSPACE
    assert lib.pq_gemm_mxfp4_workspace(64, 500, 256, 0) == 0
    p = lib.pq_gemm_mxfp4_prequant
    assert p(NUL, FAKE, 64, 512, FAKE, FAKE, 256, 0, FAKE, NUL) == NULL
    assert p(FAKE, FAKE, 64, 512, FAKE, FAKE, 257, 1, FAKE, NUL) == SHAPE
    assert p(FAKE, MIS, 64, 512, FAKE, FAKE, 256, 0, FAKE, NUL) == ALIGN


def test_grouped(lib):
    def g(x=FAKE, rows=64, K=512, order=FAKE, k=2, off=FAKE, P=128, E=4, N=256, epi=0, y=FAKE, ws=FAKE, wsn=1 << 30):
        return lib.pq_gemm_mxfp4_grouped(x, rows, K, order, k, off, P, E, FAKE, FAKE, N, epi, y, ws, wsn, NUL)
    assert g(x=NUL) == NULL and g(off=NUL) == NULL and g(y=NUL) == NULL
    for kw in (dict(rows=63), dict(P=0), dict(P=127), dict(E=0), dict(E=1025), dict(k=0), dict(K=40), dict(epi=1, N=255),
               dict(order=NUL), dict(order=NUL, rows=64, P=64, k=0)):
        assert g(**kw) == SHAPE, kw
    assert g(order=MIS) == ALIGN and g(off=MIS) == ALIGN
    assert g(ws=NUL) == WORKSPACE and g(wsn=64) == WORKSPACE
    assert lib.pq_gemm_mxfp4_grouped_workspace(64, 512, 256, 0) > 0
    p = lib.pq_gemm_mxfp4_grouped_prequant
    assert p(FAKE, FAKE, 64, 512, FAKE, 2, NUL, 128, 4, FAKE, FAKE, 256, 0, FAKE, NUL) == NULL
    assert p(FAKE, FAKE, 64, 512, NUL, 2, FAKE, 128, 4, FAKE, FAKE, 256, 0, FAKE, NUL) == SHAPE


def test_routing(lib):
    def s(ids=FAKE, M=8, k=2, E=4, order=FAKE, inv=FAKE, off=FAKE, ws=NUL, wsn=0):
        return lib.pq_moe_sort(ids, M, k, E, order, inv, off, ws, wsn, NUL)
    assert s(ids=NUL) == NULL and s(order=NUL) == NULL and s(inv=NUL) == NULL and s(off=NUL) == NULL
    for kw in (dict(M=0), dict(k=0), dict(E=0), dict(E=1025), dict(M=1 << 30, k=2), dict(M=-1)):
        assert s(**kw) == SHAPE, kw
    assert s(ids=MIS) == ALIGN and s(ws=MIS) == ALIGN
    assert lib.pq_moe_sort_workspace(256, 8, 64) == 0
    need = lib.pq_moe_sort_workspace(257, 8, 64)
    assert need > 0 and s(M=257, k=8, E=64, ws=FAKE, wsn=need - 1) == WORKSPACE
    assert s(M=257, k=8, E=64) == WORKSPACE
    assert lib.pq_moe_sort_workspace(0, 8, 64) == 0

    def d(x=FAKE, M=8, H=64, k=2, order=FAKE, inv=FAKE, xs=FAKE):
        return lib.pq_moe_dispatch(x, 0, M, H, k, order, inv, xs, NUL)
    assert d(x=NUL) == NULL and d(order=NUL) == NULL and d(inv=NUL) == NULL and d(xs=NUL) == NULL
    for kw in (dict(M=0), dict(H=0), dict(H=12), dict(k=0)):
        assert d(**kw) == SHAPE, kw
    assert d(x=MIS) == ALIGN

    def c(ys=FAKE, M=8, H=64, k=2, inv=FAKE, w=FAKE, y=FAKE):
        return lib.pq_moe_combine(ys, 0, M, H, k, inv, w, y, NUL)
    assert c(ys=NUL) == NULL and c(inv=NUL) == NULL and c(y=NUL) == NULL
    assert c(H=4) == SHAPE and c(M=0) == SHAPE and c(w=MIS) == ALIGN

    def g(dy=FAKE, ys=FAKE, H=64, w=FAKE, dys=FAKE, dw=FAKE):
        return lib.pq_moe_combine_grad(dy, ys, 0, 8, H, 2, FAKE, FAKE, w, dys, dw, NUL)
    assert g(dy=NUL) == NULL and g(ys=NUL) == NULL and g(w=NUL) == NULL and g(dys=NUL) == NULL and g(dw=NUL) == NULL
    assert g(H=20) == SHAPE and g(dw=MIS) == ALIGN


def test_launch_counts(lib):
    f = lib.pq_launches_per_call
    for n in (b"pq_gemm_mxfp4", b"pq_gemm_mxfp4_grouped", b"pq_moe_sort"):
        assert f(n) == 2, n
    for n in (b"pq_quantize_mxfp4", b"pq_dequantize_mxfp4", b"pq_gemv_mxfp4", b"pq_gemm_mxfp4_prequant",
              b"pq_gemm_mxfp4_grouped_prequant", b"pq_moe_dispatch", b"pq_moe_combine", b"pq_moe_combine_grad"):
        assert f(n) == 1, n
