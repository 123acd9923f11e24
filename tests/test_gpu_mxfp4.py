"""GPU tests of the MXFP4 operators against the float64 oracle.

Tolerances, set by arithmetic:
* codes, scale bytes and decoded values are exact;
* a product's fp32 sum of K terms is within K 2^-23 S of the exact one, S the
  sum of the terms' magnitudes (each addition is off by at most 2^-23 of a
  partial sum that S bounds, truncation included), and its bf16 rounding
  within 2^-8 of the value;
* under SiLU(gate)*up the sums' errors eg, eu move the result by at most
  1.1 |u| eg + |silu(g)| eu + 1.1 eg eu (|silu'| < 1.1), the fp32 exponential
  and quotient by 2^-16 of the value, and the bf16 rounding by 2^-8 of it.
"""
import numpy as np
import pytest

import oracle
from _helpers import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pq():
    need_gpu()
    import quantized_moe_weight_amd as pq
    return pq


def _t(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t.to(dtype) if dtype is not None else t


def _np(t):
    return t.detach().double().cpu().numpy()


def _bf16(a):
    """fp64 values of `a` rounded to bf16, as (tensor, array)."""
    import torch
    t = torch.from_numpy(np.asarray(a, dtype=np.float32)).to(torch.bfloat16).cuda()
    return t, _np(t)


def _weights(rng, *shape):
    w = (0.02 * rng.standard_normal(shape)).astype(np.float32)
    p, b = oracle.mx_quant(w.reshape(-1, shape[-1]))
    K = shape[-1]
    p, b = p.reshape(*shape[:-1], K // 2), b.reshape(*shape[:-1], K // 32)
    return _t(p), _t(b), oracle.mx_values(p, b)


def expect(x, w, silu):
    """(values, bound) of epi(x w^T) in float64."""
    K = x.shape[1]
    y, S = oracle.mx_product(x, w)
    e = K * 2.0 ** -23 * S
    if not silu:
        return y, e + 2.0 ** -8 * (np.abs(y) + e)
    n = w.shape[0] // 2
    g, u, eg, eu = y[:, :n], y[:, n:], e[:, :n], e[:, n:]
    sg = g / (1.0 + np.exp(-g))
    h = sg * u
    e = 1.1 * np.abs(u) * eg + np.abs(sg) * eu + 1.1 * eg * eu + 2.0 ** -16 * np.abs(h)
    return h, e + 2.0 ** -8 * (np.abs(h) + e)


def close(got, want, bound, what):
    err = np.abs(_np(got) - want)
    assert got.shape == want.shape and np.isfinite(err).all(), what
    bad = err > bound
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {(err / np.maximum(bound, 1e-300)).max():.3g} of the bound"


# ---------------------------------------------------------------------------
# quantiser
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("R,K", [(1, 32), (3, 96), (17, 160), (5, 5120), (129, 512), (1000, 2048)])
def test_quantise_is_exact(pq, dtype, R, K):
    import torch
    rng = np.random.default_rng(R * K)
    v = (rng.standard_normal((R, K)) * np.exp2(rng.integers(-20, 20, (R, 1)))).astype(np.float32)
    v[rng.random((R, K)) < 0.05] = 0.0
    t = _t(v, torch.bfloat16 if dtype == "bf16" else None)
    p, b = oracle.mx_quant(_np(t))
    codes, scales = pq.quantize_mxfp4(t)
    assert np.array_equal(codes.cpu().numpy(), p) and np.array_equal(scales.cpu().numpy(), b)
    for dt in (torch.bfloat16, torch.float32):
        got = pq.dequantize_mxfp4(codes, scales, dt)
        assert got.dtype == dt and np.array_equal(_np(got), oracle.mx_values(p, b))


def test_quantise_edges(pq):
    """Ties, saturation, zeros of both signs, subnormals, the largest values, infinities and NaN."""
    import torch
    rows = []
    for e in (-149, -140, -127, -126, -125, -124, -3, 0, 7, 125):
        s = 2.0 ** e
        with np.errstate(over="ignore", under="ignore"):
            base = np.array([4, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, 6, 7.9999995, .2500001, .7499999] * 2 + [0.0] * 8)
            rows.append(np.nan_to_num((base * np.where(np.arange(32) % 2, -1, 1) * s).astype(np.float32),
                                      posinf=3.4e38, neginf=-3.4e38))
    rows.append(np.zeros(32, np.float32))
    rows.append(-np.zeros(32, np.float32))
    for bad in (np.inf, -np.inf, np.nan):
        r = np.linspace(-3, 3, 32).astype(np.float32)
        r[13] = bad
        rows.append(r)
    v = np.stack(rows)
    p, b = oracle.mx_quant(v)
    codes, scales = pq.quantize_mxfp4(_t(v))
    assert np.array_equal(scales.cpu().numpy(), b)
    assert np.array_equal(codes.cpu().numpy(), p)
    got = _np(pq.dequantize_mxfp4(codes, scales, torch.float32))
    want = oracle.mx_values(p, b)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[~np.isnan(want)], want[~np.isnan(want)])


def test_dequantise_every_byte_and_code(pq):
    import torch
    c = np.array([i | (15 - i) << 4 for i in range(16)], dtype=np.uint8)
    p, b = np.tile(c, (256, 1)), np.arange(256, dtype=np.uint8)[:, None]
    want = oracle.mx_values(p, b)
    for dt, top in ((torch.bfloat16, 253), (torch.float32, 253)):
        got = _np(pq.dequantize_mxfp4(_t(p), _t(b), dt))
        assert np.array_equal(got[:top], want[:top])
        assert np.isnan(got[255]).all()
        big = np.abs(want[253:255]) >= 2.0 ** 128                 # past the type's range
        assert np.isinf(got[253:255][big]).all() and np.array_equal(np.sign(got[253:255]), np.sign(want[253:255]))


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("M,K,N", [(1, 32, 2), (1, 64, 34), (1, 5120, 512), (2, 288, 100), (3, 256, 16), (4, 1056, 18),
                                   (5, 512, 8192), (7, 544, 1000), (8, 2048, 258), (9, 320, 66), (15, 4640, 20),
                                   (16, 4352, 40), (16, 96, 6), (1, 17408, 512)])
def test_gemv(pq, M, K, N, silu):
    rng = np.random.default_rng(M * K + N)
    x, xv = _bf16(rng.standard_normal((M, K)))
    w, s, wv = _weights(rng, N, K)
    y = pq.gemv_mxfp4(x, w, s, pq.EPI_SILU_MUL if silu else pq.EPI_NONE)
    close(y, *expect(xv, wv, silu), f"gemv M={M} K={K} N={N} silu={silu}")


def test_gemv_does_not_depend_on_the_other_tokens(pq):
    import torch
    rng = np.random.default_rng(1)
    x, _ = _bf16(rng.standard_normal((16, 1056)))
    w, s, _ = _weights(rng, 300, 1056)
    y = pq.gemv_mxfp4(x, w, s)
    for M in (1, 2, 5, 8, 13):
        assert torch.equal(pq.gemv_mxfp4(x[:M].contiguous(), w, s), y[:M])


def test_gemv_infinities_stay_in_their_token(pq):
    import torch
    rng = np.random.default_rng(2)
    for K in (96, 288, 512):                                        # last steps with and without blocks past K
        x, xv = _bf16(rng.standard_normal((6, K)))
        w, s, wv = _weights(rng, 64, K)
        x[1, K - 1] = float("inf")
        x[3, 0] = float("nan")
        y = pq.gemv_mxfp4(x, w, s)
        ok = [0, 2, 4, 5]
        close(y[ok], *expect(xv[ok], wv, False), f"K={K}")
        assert torch.isnan(y[3]).all() and not torch.isfinite(y[1]).any()


def test_extreme_scales(pq):
    """Weights of any scale byte; a NaN block poisons its row only."""
    import torch
    rng = np.random.default_rng(4)
    K, N = 256, 64
    p = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    b = rng.integers(100, 150, (N, K // 32), dtype=np.uint8)
    b[0] = 0
    b[1] = 1
    b[2] = 220
    b[5, 3] = 255
    wv = oracle.mx_values(p, b)
    x, xv = _bf16(rng.standard_normal((8, K)))
    y = pq.gemv_mxfp4(x, _t(p), _t(b))
    xq = pq.dequantize_mxfp4(*pq.quantize_mxfp4(x), dtype=torch.float32)
    z = pq.gemm_mxfp4(x, _t(p), _t(b))
    keep = np.arange(N) != 5
    for got, src, what in ((y, xv, "gemv"), (z, _np(xq), "gemm")):
        assert torch.isnan(got[:, 5]).all()
        want, bound = expect(src, wv[keep], False)
        # results of the smallest scales are subnormal, where a rounding step is fixed
        close(got[:, torch.from_numpy(keep).cuda()], want, bound + 2.0 ** -133, what)


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("M,K,N", [(1, 32, 2), (1, 128, 64), (5, 96, 130), (16, 512, 256), (31, 160, 34), (64, 1024, 514),
                                   (129, 256, 66), (200, 1312, 1000), (257, 640, 300), (333, 2560, 512), (700, 288, 1026)])
def test_gemm(pq, M, K, N, silu):
    import torch
    rng = np.random.default_rng(M + K + N)
    x, _ = _bf16(rng.standard_normal((M, K)) * np.exp2(rng.integers(-4, 4, (M, 1))))
    w, s, wv = _weights(rng, N, K)
    epi = pq.EPI_SILU_MUL if silu else pq.EPI_NONE
    xq, xs = pq.quantize_mxfp4(x)
    xv = oracle.mx_values(xq.cpu().numpy(), xs.cpu().numpy())
    y = pq.gemm_mxfp4(x, w, s, epi)
    close(y, *expect(xv, wv, silu), f"gemm M={M} K={K} N={N} silu={silu}")
    assert torch.equal(pq.gemm_mxfp4_prequant(xq, xs, w, s, epi), y)
    if M > 2:                                                      # a row's bits do not depend on the others
        cut = M // 2
        assert torch.equal(pq.gemm_mxfp4(x[cut:].contiguous(), w, s, epi), y[cut:])


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("M,K,N", [(65, 128, 260), (130, 640, 520), (300, 896, 390), (513, 1152, 774)])
def test_gemm_tiles_agree(pq, monkeypatch, M, K, N, silu):
    """Every tile of the tiled kernel gives the same bits, and leaves what lies around the output alone."""
    import torch
    rng = np.random.default_rng(M)
    x, _ = _bf16(rng.standard_normal((M, K)))
    w, s, _ = _weights(rng, N, K)
    epi = pq.EPI_SILU_MUL if silu else pq.EPI_NONE
    xq, xs = pq.quantize_mxfp4(x)
    R = N // 2 if silu else N
    want, bound = expect(oracle.mx_values(xq.cpu().numpy(), xs.cpu().numpy()),
                         oracle.mx_values(w.cpu().numpy(), s.cpu().numpy()), silu)
    seen = []
    for tile in ("1", "2", "3", "4"):
        monkeypatch.setenv("PQ_MXFP4_TILE", tile)
        room = torch.full((M + 600, R), 7.0, dtype=torch.bfloat16, device="cuda")
        pad = 304                                           # a multiple of 8: the output stays 16-byte aligned
        out = room[pad:pad + M]
        assert out.data_ptr() % 16 == 0
        y = pq.gemm_mxfp4_prequant(xq, xs, w, s, epi, out=out)
        assert (room[:pad] == 7.0).all() and (room[pad + M:] == 7.0).all()
        close(y, want, bound, f"tile {tile}")
        seen.append(y.clone())
    assert all(torch.equal(y, seen[0]) for y in seen)


def test_gemm_nan_rows_stay_alone(pq):
    import torch
    rng = np.random.default_rng(8)
    for K in (160, 256, 1152):                                     # both kernels, last scales part of a load
        x, xv = _bf16(rng.standard_normal((140, K)))
        w, s, wv = _weights(rng, 70, K)
        x[7, K - 1] = float("inf")
        x[139, 0] = float("nan")
        y = pq.gemm_mxfp4(x, w, s)
        assert torch.isnan(y[[7, 139]]).all()
        row = torch.arange(140, device="cuda")
        assert torch.isfinite(y[(row != 7) & (row != 139)]).all()


def test_gemv_activation_and_sums_past_one_cus_lds(pq):
    """139 KB of activation leave room for few partial sums: the rows are split over more blocks than CUs."""
    rng = np.random.default_rng(12)
    for M, K, N, silu in ((16, 4352, 20002, True), (2, 34816, 60000, False)):
        x, xv = _bf16(rng.standard_normal((M, K)))
        p = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
        b = rng.integers(118, 123, (N, K // 32), dtype=np.uint8)
        y = pq.gemv_mxfp4(x, _t(p), _t(b), pq.EPI_SILU_MUL if silu else pq.EPI_NONE)
        R = N // 2 if silu else N
        at = np.unique(np.concatenate([rng.integers(0, R, 300), [0, 1, R - 2, R - 1]]))
        rows = np.concatenate([at, at + R]) if silu else at
        want, bound = expect(xv, oracle.mx_values(p[rows], b[rows]), silu)
        import torch
        close(y[:, torch.from_numpy(at).cuda()], want, bound, f"M={M} K={K} N={N}")


def _routing(rng, M, k, E, how):
    if how == "even":
        ids = np.stack([rng.permutation(E)[:k] if k <= E else rng.integers(0, E, k) for _ in range(M)])
    elif how == "one":                                             # every pair at one expert
        ids = np.full((M, k), E // 2)
    elif how == "none":
        ids = np.full((M, k), -1)
    else:                                                          # single slots and whole tokens left out
        ids = rng.integers(0, E, (M, k))
        ids[rng.random((M, k)) < 0.3] = -1
        ids[rng.random(M) < 0.2] = -1
        ids[rng.random((M, k)) < 0.05] = E + 7
    return ids.astype(np.int32)


@pytest.mark.parametrize("how", ["even", "one", "drop", "none"])
@pytest.mark.parametrize("M,k,E,K,N,silu", [(1, 1, 1, 32, 2, False), (1, 8, 16, 128, 64, True), (5, 2, 3, 96, 66, True),
                                            (61, 8, 64, 256, 130, False), (200, 4, 6, 320, 96, True),
                                            (333, 3, 1024, 64, 34, False), (600, 2, 4, 512, 258, False)])
def test_grouped(pq, M, k, E, K, N, silu, how):
    import torch
    rng = np.random.default_rng(M * k + E)
    ids = _routing(rng, M, k, E, how)
    order, inverse, offsets = oracle.route_sort(np.where((ids < 0) | (ids >= E), -1, ids), E)
    plan = pq.MoePlan(_t(order), _t(inverse), _t(offsets))
    w, s, wv = _weights(rng, E, N, K)
    epi = pq.EPI_SILU_MUL if silu else pq.EPI_NONE
    for gather in (True, False):
        x, _ = _bf16(rng.standard_normal((M if gather else M * k, K)))
        xq, xs = pq.quantize_mxfp4(x)
        xv = oracle.mx_values(xq.cpu().numpy(), xs.cpu().numpy())
        rows = oracle.route_dispatch(xv, order, k) if gather else xv
        R = N // 2 if silu else N
        want, bound = np.zeros((M * k, R)), np.zeros((M * k, R))
        for e in range(E):
            lo, hi = offsets[e], offsets[e + 1]
            if hi > lo:
                want[lo:hi], bound[lo:hi] = expect(rows[lo:hi], wv[e], silu)
        out = torch.full((M * k, R), float("nan"), dtype=torch.bfloat16, device="cuda")
        y = pq.gemm_mxfp4_grouped(x, w, s, plan, epi, gather=gather, out=out)
        assert y is out
        close(y, want, bound, f"grouped {how} gather={gather}")
        assert torch.equal(pq.gemm_mxfp4_grouped_prequant(xq, xs, w, s, plan, epi, gather=gather), y)


@pytest.mark.parametrize("K", [64, 128])
def test_grouped_offsets_out_of_range_stay_inside(pq, K):
    """Offsets and order entries that moe_sort does not make are clamped: no access leaves x, w or y."""
    import torch
    rng = np.random.default_rng(0)
    M, k, E, N = 8, 2, 4, 32
    w, s, _ = _weights(rng, E, N, K)
    x, _ = _bf16(rng.standard_normal((M, K)))
    guard = torch.zeros((3 * M * k, N), dtype=torch.bfloat16, device="cuda")
    out = guard[M * k:2 * M * k]
    for off in ([0, 100, -5, 3, 1 << 30], [5, 4, 3, 2, 1], [-9, -8, -7, -6, -5]):
        order = _t(np.array([1 << 20, -1, 3, 16] * (M * k // 4), dtype=np.int32))
        plan = pq.MoePlan(order, _t(np.zeros((M, k), np.int32)), _t(np.array(off, dtype=np.int32)))
        pq.gemm_mxfp4_grouped(x, w, s, plan, out=out)
        torch.cuda.synchronize()
        assert not guard[:M * k].any() and not guard[2 * M * k:].any()


# ---------------------------------------------------------------------------
# the operators together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("M,k,E,H,I", [(1, 2, 4, 128, 64), (37, 4, 8, 256, 96), (300, 8, 16, 512, 256)])
def test_prefill_layer(pq, M, k, E, H, I):
    """The layer against the oracle, step by step on the device's own intermediates (a 4-bit code of h may fall on
    the other side of a rounding border in float64; from the same h every step has its own bound)."""
    import torch
    rng = np.random.default_rng(M)
    ids = _routing(rng, M, k, E, "drop" if M > 1 else "even")
    x, _ = _bf16(rng.standard_normal((M, H)))
    w13, s13, v13 = _weights(rng, E, 2 * I, H)
    w2, s2, v2 = _weights(rng, E, H, I)
    tw = rng.random((M, k)).astype(np.float32)
    y = pq.moe_prefill_layer_mxfp4(x, w13, s13, w2, s2, _t(ids), _t(tw))
    plan = pq.moe_sort(_t(ids), E)
    order, inverse, offsets = oracle.route_sort(np.where((ids < 0) | (ids >= E), -1, ids), E)
    for got, want in zip(plan, (order, inverse, offsets)):
        assert np.array_equal(got.cpu().numpy(), want)
    h = pq.gemm_mxfp4_grouped(x, w13, s13, plan, pq.EPI_SILU_MUL)
    z = pq.gemm_mxfp4_grouped(h, w2, s2, plan, gather=False)
    assert torch.equal(y, pq.moe_combine(z, plan, _t(tw)))
    n = offsets[-1]
    expert = np.repeat(np.arange(E), np.diff(offsets))
    for src, wv, got, silu in ((oracle.route_dispatch(oracle.mx_values(*oracle.mx_quant(_np(x))), order, k), v13, h, True),
                               (oracle.mx_values(*oracle.mx_quant(_np(h))), v2, z, False)):
        for e in range(E):
            at = np.nonzero(expert == e)[0]
            if len(at):
                close(got[at[0]:at[-1] + 1], *expect(src[at], wv[e], silu), f"expert {e}")
        assert not got[n:].any()
    want, mag = oracle.route_combine(_np(z), inverse, tw)
    close(y, want, 2.0 ** -8 * np.abs(want) + (k + 1) * 2.0 ** -23 * mag, "combine")
    none = (inverse < 0).all(1)
    assert not y[torch.from_numpy(none).cuda()].any()


def test_prefill_layer_in_a_graph_and_on_another_stream(pq):
    import torch
    rng = np.random.default_rng(11)
    M, k, E, H, I = 700, 4, 8, 256, 128
    w13, s13, _ = _weights(rng, E, 2 * I, H)
    w2, s2, _ = _weights(rng, E, H, I)
    sets = []
    for _ in range(3):
        x, _ = _bf16(rng.standard_normal((M, H)))
        sets.append((x, _t(_routing(rng, M, k, E, "drop")), _t(rng.random((M, k)).astype(np.float32))))
    want = [pq.moe_prefill_layer_mxfp4(x, w13, s13, w2, s2, i, t) for x, i, t in sets]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = pq.moe_prefill_layer_mxfp4(sets[1][0], w13, s13, w2, s2, sets[1][1], sets[1][2])
    side.synchronize()
    assert torch.equal(got, want[1])
    bufs = [t.clone() for t in sets[0]]
    graphs, outs = [], []
    for _ in range(2):                              # two graphs of the same call share no scratch
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(pq.moe_prefill_layer_mxfp4(bufs[0], w13, s13, w2, s2, bufs[1], bufs[2]))
        graphs.append(g)
    for rep in range(4):
        for b, t in zip(bufs, sets[rep % 3]):
            b.copy_(t)
        for g in graphs:
            g.replay()
        eager = pq.moe_prefill_layer_mxfp4(*[bufs[0], w13, s13, w2, s2, bufs[1], bufs[2]])
        torch.cuda.synchronize()
        for o in outs:
            assert torch.equal(o, want[rep % 3]) and torch.equal(eager, want[rep % 3])


def test_single_calls_in_a_graph(pq):
    """Each call captured with others on one stream; every replay equals the eager calls on the same buffers."""
    import torch
    rng = np.random.default_rng(21)
    M, k, E, H = 300, 8, 16, 512
    w, s, _ = _weights(rng, 96, H)
    sets = []
    for _ in range(3):
        x, _ = _bf16(rng.standard_normal((M, H)))
        dy, _ = _bf16(rng.standard_normal((M, H)))
        sets.append((x, dy, _t(_routing(rng, M, k, E, "drop")), _t(rng.random((M, k)).astype(np.float32))))
    bufs = [t.clone() for t in sets[0]]

    def calls(x, dy, ids, tw):
        few = x[:12].contiguous()
        plan = pq.moe_sort(ids, E)
        xs = pq.moe_dispatch(x, plan)
        return [pq.gemv_mxfp4(few, w, s), pq.gemv_mxfp4(few, w, s, pq.EPI_SILU_MUL), pq.gemm_mxfp4(x, w, s),
                pq.dequantize_mxfp4(*pq.quantize_mxfp4(x)), *plan, xs, pq.moe_combine(xs, plan, tw),
                pq.moe_dispatch_grad(xs, plan), *pq.moe_combine_grad(dy, xs, plan, tw)]

    want = [calls(*c) for c in sets]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = calls(*bufs)
    for rep in range(5):
        for b, t in zip(bufs, sets[rep % 3]):
            b.copy_(t)
        g.replay()
        eager = calls(*bufs)
        torch.cuda.synchronize()
        for a, b, c in zip(got, eager, want[rep % 3]):
            assert torch.equal(a, c) and torch.equal(b, c)


def test_two_threads_on_two_streams(pq):
    """Calls of two host threads at once, each on its own stream, share nothing."""
    import threading
    import torch
    rng = np.random.default_rng(31)
    M, k, E, H, I = 200, 4, 8, 256, 128
    w13, s13, _ = _weights(rng, E, 2 * I, H)
    w2, s2, _ = _weights(rng, E, H, I)
    jobs = []
    for _ in range(2):
        x, _ = _bf16(rng.standard_normal((M, H)))
        a = (x, w13, s13, w2, s2, _t(_routing(rng, M, k, E, "drop")), _t(rng.random((M, k)).astype(np.float32)))
        jobs.append((a, pq.moe_prefill_layer_mxfp4(*a)))
    torch.cuda.synchronize()
    bad = []

    def work(a, want):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            outs = [pq.moe_prefill_layer_mxfp4(*a) for _ in range(20)]
        st.synchronize()
        bad.extend(o for o in outs if not torch.equal(o, want))

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_past_4_gib(pq):
    """Byte offsets past 32 bits: in the quantiser's input, and in the grouped product's rows."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((70000, 32768), generator=g, device="cuda", dtype=torch.bfloat16)      # 4.6 GB
    codes, scales = pq.quantize_mxfp4(x)
    c, s = pq.quantize_mxfp4(x[-300:].contiguous())
    assert torch.equal(codes[-300:], c) and torch.equal(scales[-300:], s)
    assert torch.equal(pq.dequantize_mxfp4(codes, scales)[-300:], pq.dequantize_mxfp4(c, s))
    del x, codes, scales
    M, k, E, K, N = 100000, 2, 4, 128, 12288                                                # 4.9 GB of results
    ids = torch.randint(0, E, (M, k), generator=g, device="cuda", dtype=torch.int32)
    x = torch.randn((M, K), generator=g, device="cuda", dtype=torch.bfloat16)
    w = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    ws = torch.randint(118, 123, (E, N, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    plan = pq.moe_sort(ids, E)
    y = pq.gemm_mxfp4_grouped(x, w, ws, plan)
    last = pq.moe_dispatch(x, plan)[-500:].contiguous()
    assert torch.equal(y[-500:], pq.gemm_mxfp4(last, w[E - 1], ws[E - 1]))
    first = pq.moe_dispatch(x, plan)[:500].contiguous()
    assert torch.equal(y[:500], pq.gemm_mxfp4(first, w[0], ws[0]))


# ---------------------------------------------------------------------------
# refusals of the binding
# ---------------------------------------------------------------------------
def test_refusals(pq, monkeypatch):
    import torch
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    w, s = torch.zeros((8, 32), dtype=torch.uint8, device="cuda"), torch.zeros((8, 2), dtype=torch.uint8, device="cuda")
    for call in (pq.gemv_mxfp4, pq.gemm_mxfp4):
        with pytest.raises(TypeError):
            call(x.float(), w, s)
        with pytest.raises(TypeError):
            call(x.cpu(), w, s)
        with pytest.raises(ValueError):
            call(x[:, ::2], w, s)
        with pytest.raises(ValueError):
            call(x[:, :32].contiguous(), w, s)
        with pytest.raises(ValueError):
            call(x, w, s[:4].contiguous())
        with pytest.raises(ValueError):
            call(x, w, s, out=torch.zeros((4, 7), dtype=torch.bfloat16, device="cuda"))
        with pytest.raises(TypeError):
            call(x, w, s, out=torch.zeros((4, 8), device="cuda"))
        with pytest.raises(pq.PqError):
            call(x[:0], w, s)
    with pytest.raises(pq.PqError):
        pq.gemv_mxfp4(torch.zeros((17, 64), dtype=torch.bfloat16, device="cuda"), w, s)
    with pytest.raises(TypeError):
        pq.quantize_mxfp4(x.half())
    with pytest.raises(pq.PqError):
        pq.quantize_mxfp4(torch.zeros((2, 40), device="cuda"))
    with pytest.raises(TypeError):
        pq.dequantize_mxfp4(w, s, torch.float16)
    with pytest.raises(ValueError):
        pq.dequantize_mxfp4(w, s[:, :1].contiguous())
    e4 = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    tw = torch.ones((4, 2), device="cuda")
    w13, s13 = torch.zeros((3, 64, 32), dtype=torch.uint8, device="cuda"), torch.zeros((3, 64, 2), dtype=torch.uint8, device="cuda")
    w2, s2 = torch.zeros((3, 64, 16), dtype=torch.uint8, device="cuda"), torch.zeros((3, 64, 1), dtype=torch.uint8, device="cuda")
    assert tuple(pq.moe_prefill_layer_mxfp4(x, w13, s13, w2, s2, e4, tw).shape) == (4, 64)
    for bad in ((w13[:2].contiguous(), s13[:2].contiguous(), w2, s2), (w13, s13, w2[:, :32].contiguous(), s2[:, :32].contiguous()),
                (w13[:, :32].contiguous(), s13[:, :32].contiguous(), w2, s2)):
        with pytest.raises(ValueError):
            pq.moe_prefill_layer_mxfp4(x, *bad, e4, tw)
    with pytest.raises(TypeError):
        pq.moe_prefill_layer_mxfp4(x, w13, s13, w2, s2, e4, None)
    buf = torch.zeros(64 * 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):                 # an output on top of an input that other blocks still read
        pq.gemv_mxfp4(buf[:256].view(4, 64), w, s, out=buf[128:160].view(4, 8))
    plan = pq.moe_sort(torch.zeros((4, 2), dtype=torch.int32, device="cuda"), 3)
    wg, sg = w[None].repeat(3, 1, 1), s[None].repeat(3, 1, 1)
    with pytest.raises(ValueError):
        pq.gemm_mxfp4_grouped(x, wg[:2].contiguous(), sg[:2].contiguous(), plan)
    with pytest.raises(ValueError):
        pq.gemm_mxfp4_grouped(x, wg, sg, plan, gather=False)
    with pytest.raises(ValueError):
        pq.gemm_mxfp4_grouped(x, wg, sg[:, :4].contiguous(), plan)
    monkeypatch.setattr(pq, "_current_device", lambda: 1)
    with pytest.raises(ValueError):                 # a tensor of another device than the current one
        pq.gemv_mxfp4(x, w, s)
