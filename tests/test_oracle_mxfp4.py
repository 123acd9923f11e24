"""The MXFP4 and routing oracle against values that do not come from it:
exhaustive nearest-level search in exact rationals, the format's own limits,
numpy's stable sort, and torch's autograd for the gradients."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle

LEVELS = [Fraction(x) for x in ("0", "1/2", "1", "3/2", "2", "3", "4", "6")]


def _row(block):
    v = np.zeros((1, 32), dtype=np.float32)
    v[0, :len(block)] = block
    return v


def _code(packed, i):
    return int(packed[0, i // 2] >> (4 * (i % 2))) & 15


def test_levels_ties_and_saturation():
    """amax 4..8 fixes the scale at 1: every midpoint goes to the even code, and (6, 8) saturates."""
    cases = {0.25: 0, 0.75: 2, 1.25: 2, 1.75: 4, 2.5: 4, 3.5: 6, 5.0: 6, 0.2500001: 1, 0.7499999: 1, 1.2500001: 3,
             1.7499999: 3, 2.5000002: 5, 3.4999998: 5, 5.0000005: 7, 7.9999995: 7, 6.5: 7}
    for v, want in cases.items():
        for sign in (1, -1):
            p, b = oracle.mx_quant(_row([4.0, sign * v]))
            assert b[0, 0] == 127 and _code(p, 1) == want | (8 if sign < 0 else 0), v


@pytest.mark.parametrize("seed", range(4))
def test_nearest_level_in_exact_rationals(seed):
    rng = np.random.default_rng(seed)
    v = (rng.standard_normal((1, 64)) * np.exp2(rng.integers(-30, 30))).astype(np.float32)
    p, b = oracle.mx_quant(v)
    for i in range(64):
        blk = v[0, i // 32 * 32:][:32]
        top = max(abs(Fraction(float(x))) for x in blk)
        e = 0
        while top >= Fraction(2) ** (e + 1):
            e += 1
        while top < Fraction(2) ** e:
            e -= 1
        assert b[0, i // 32] == e - 2 + 127
        a = min(abs(Fraction(float(v[0, i]))) / Fraction(2) ** (e - 2), Fraction(6))
        best = min(abs(a - lv) for lv in LEVELS)
        c = _code(p, i) & 7
        assert abs(a - LEVELS[c]) == best
        if sum(abs(a - lv) == best for lv in LEVELS) > 1:
            assert c % 2 == 0


def test_scale_bytes_at_the_edges():
    tiny, huge = np.float32(2.0 ** -149), np.float32(3.4028235e38)
    for top, byte in ((0.0, 127), (tiny, 0), (2.0 ** -126, 0), (2.0 ** -125, 0), (2.0 ** -124, 1), (1.0, 125),
                      (huge, 252), (np.inf, 255), (np.nan, 255)):
        p, b = oracle.mx_quant(_row([top, -0.0]))
        assert b[0, 0] == byte, top
        if byte == 255:
            assert not p.any()


def test_values_of_every_code_and_byte():
    packed = np.tile(np.arange(16, dtype=np.uint8), 1).repeat(1)
    row = np.array([[c | (c ^ 8) << 4 for c in packed]], dtype=np.uint8)     # 32 values: c, -c
    for b in range(256):
        got = oracle.mx_values(row, np.array([[b]], dtype=np.uint8))[0]
        for i, c in enumerate(packed):
            lv = float(LEVELS[c & 7]) * (-1 if c & 8 else 1)
            if b == 255:
                assert np.isnan(got[2 * i]) and np.isnan(got[2 * i + 1])
            else:
                assert got[2 * i] == lv * 2.0 ** (b - 127) and got[2 * i + 1] == -lv * 2.0 ** (b - 127)


def test_quantising_its_own_values_changes_nothing():
    rng = np.random.default_rng(5)
    v = rng.standard_normal((4, 96)).astype(np.float32)
    p, b = oracle.mx_quant(v)
    p2, b2 = oracle.mx_quant(oracle.mx_values(p, b))
    assert np.array_equal(oracle.mx_values(p, b), oracle.mx_values(p2, b2))


@pytest.mark.parametrize("M,k,E,drop", [(1, 1, 1, 0), (7, 3, 5, 0.3), (40, 4, 16, 0), (9, 2, 300, 1.0)])
def test_sort_is_numpys_stable_sort(M, k, E, drop):
    rng = np.random.default_rng(M)
    ids = rng.integers(0, E, (M, k))
    ids[rng.random((M, k)) < drop] = -1
    order, inverse, offsets = oracle.route_sort(ids, E)
    flat = np.where(ids.reshape(-1) < 0, E, ids.reshape(-1))
    want = np.argsort(flat, kind="stable")
    n = int((flat < E).sum())
    assert np.array_equal(order[:n], want[:n]) and (order[n:] == -1).all()
    assert offsets[0] == 0 and offsets[-1] == n
    for p in range(M * k):
        r = inverse.reshape(-1)[p]
        assert (r == -1) == (flat[p] == E)
        if r >= 0:
            assert order[r] == p and offsets[flat[p]] <= r < offsets[flat[p] + 1]


def test_moves_and_gradients_are_autograds():
    rng = np.random.default_rng(3)
    M, k, E, H = 6, 3, 4, 8
    ids = rng.integers(-1, E, (M, k))
    order, inverse, offsets = oracle.route_sort(ids, E)
    x = torch.tensor(rng.standard_normal((M, H)), requires_grad=True)
    w = torch.tensor(rng.standard_normal((M, k)), requires_grad=True)
    o, inv = torch.tensor(order).long(), torch.tensor(inverse).long()
    xs = torch.where((o >= 0)[:, None], x[o.clamp_min(0) // k], 0.0)
    assert np.array_equal(xs.detach().numpy(), oracle.route_dispatch(x.detach().numpy(), order, k))
    ys = torch.tensor(rng.standard_normal((M * k, H)), requires_grad=True)
    y = torch.where((inv >= 0)[..., None], ys[inv.clamp_min(0)] * w[..., None], 0.0).sum(1)
    got, _ = oracle.route_combine(ys.detach().numpy(), inverse, w.detach().numpy())
    assert np.allclose(got, y.detach().numpy(), rtol=1e-14, atol=1e-14)
    dy = torch.tensor(rng.standard_normal((M, H)))
    y.backward(dy)
    dys, dw, _ = oracle.route_combine_grad(dy.numpy(), ys.detach().numpy(), order, inverse, w.detach().numpy())
    assert np.allclose(dys, ys.grad.numpy(), rtol=1e-14, atol=1e-14)
    assert np.allclose(dw, w.grad.numpy(), rtol=1e-13, atol=1e-13)
    dxs = torch.tensor(rng.standard_normal((M * k, H)))
    xs.backward(dxs)
    dx, _ = oracle.route_combine(dxs.numpy(), inverse, np.ones((M, k)))
    assert np.allclose(dx, x.grad.numpy(), rtol=1e-14, atol=1e-14)
