"""GPU tests of the routed rows' sort and moves.

The sort is exact.  A combined row is an fp32 sum of k products (each product
and each addition off by at most 2^-24 of what the terms' magnitudes sum to,
so at most (k + 1) 2^-23 of that sum with room for fused and separate
roundings), rounded to its type (bf16 2^-8, fp32 2^-24 of the value).  A row
gradient is one product rounded once more to its type; a weight gradient an
fp32 sum of H products, within H 2^-23 of the sum of their magnitudes."""
import numpy as np
import pytest

import oracle
from _helpers import need_gpu

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


@pytest.fixture(scope="module")
def pq():
    need_gpu()
    import quantized_moe_weight_amd as pq
    return pq


def _t(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _np(t):
    return t.detach().double().cpu().numpy()


def _rows(rng, n, H, dtype):
    import torch
    t = torch.from_numpy(rng.standard_normal((n, H)).astype(np.float32)).cuda()
    return t.to(torch.bfloat16) if dtype == "bf16" else t


def _ids(rng, M, k, E, drop):
    ids = rng.integers(0, E, (M, k))
    ids[rng.random((M, k)) < drop] = -1
    ids[rng.random(M) < drop] = -1
    return ids.astype(np.int32)


@pytest.mark.parametrize("M,k,E", [(1, 1, 1), (1, 8, 256), (9, 7, 3), (8, 8, 2), (64, 1, 64), (65, 1, 1024), (256, 8, 256),
                                   (257, 8, 256), (2047, 1, 5), (2049, 1, 129), (1000, 6, 60), (4099, 8, 256),
                                   (9000, 3, 1000), (70001, 8, 17)])
@pytest.mark.parametrize("drop", [0.0, 0.3, 1.0])
def test_sort(pq, M, k, E, drop):
    rng = np.random.default_rng(M + E)
    ids = _ids(rng, M, k, E, drop)
    plan = pq.moe_sort(_t(ids), E)
    flat = np.where(ids.reshape(-1) < 0, E, ids.reshape(-1))
    n = int((flat < E).sum())
    want = np.argsort(flat, kind="stable")
    order, inverse, offsets = (t.cpu().numpy() for t in plan)
    assert np.array_equal(order[:n], want[:n]) and (order[n:] == -1).all()
    inv = np.full(M * k, -1)
    inv[want[:n]] = np.arange(n)
    assert np.array_equal(inverse.reshape(-1), inv)
    assert np.array_equal(offsets, np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E + 1)[:E])]))


def test_sort_ids_out_of_range_are_no_expert(pq):
    ids = np.array([[3, -1, 4, 2 ** 31 - 1], [-2 ** 31, 0, 5, 3]], dtype=np.int32)
    plan = pq.moe_sort(_t(ids), 4)
    for got, want in zip(plan, oracle.route_sort(np.where((ids < 0) | (ids > 3), -1, ids), 4)):
        assert np.array_equal(got.cpu().numpy(), want)


def test_sort_same_expert_twice_in_a_token(pq):
    ids = np.array([[1, 1, 0], [0, 1, 1]], dtype=np.int32)
    plan = pq.moe_sort(_t(ids), 2)
    assert plan.order.tolist() == [2, 3, 0, 1, 4, 5] and plan.offsets.tolist() == [0, 2, 6]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("M,k,E,H,drop", [(1, 1, 1, 8, 0.0), (1, 8, 16, 6144, 0.0), (3, 2, 4, 24, 0.5), (8, 8, 256, 2056, 0.0),
                                          (61, 9, 5, 512, 0.2), (500, 8, 64, 1032, 0.1), (20, 3, 7, 64, 1.0)])
def test_moves_and_gradients(pq, dtype, M, k, E, H, drop):
    import torch
    rng = np.random.default_rng(M * H)
    ids = _ids(rng, M, k, E, drop)
    order, inverse, offsets = oracle.route_sort(ids, E)
    plan = pq.moe_sort(_t(ids), E)
    P = M * k
    x = _rows(rng, M, H, dtype)
    nan = lambda n: torch.full((n, H), float("nan"), dtype=x.dtype, device="cuda")  # noqa: E731
    xs = pq.moe_dispatch(x, plan, out=nan(P))
    assert np.array_equal(_np(xs), oracle.route_dispatch(_np(x), order, k))
    ys, w = _rows(rng, P, H, dtype), rng.standard_normal((M, k)).astype(np.float32)
    ys[int(offsets[-1]):] = float("nan")            # rows without a pair are not read
    ysn = np.nan_to_num(_np(ys))
    for weights, got in ((w, pq.moe_combine(ys, plan, _t(w), out=nan(M))),
                         (np.ones((M, k)), pq.moe_combine(ys, plan, out=nan(M))),
                         (np.ones((M, k)), pq.moe_dispatch_grad(ys, plan))):
        want, mag = oracle.route_combine(ysn, inverse, weights)
        err = np.abs(_np(got) - want)
        assert got.dtype == x.dtype and (err <= HALF[dtype] * np.abs(want) + (k + 1) * 2.0 ** -23 * mag).all()
    dy = _rows(rng, M, H, dtype)
    dys, dw = pq.moe_combine_grad(dy, ys, plan, _t(w), out=nan(P))
    gys, gw, mag = oracle.route_combine_grad(_np(dy), ysn, order, inverse, w)
    assert dys.dtype == x.dtype and dw.dtype == torch.float32
    assert (np.abs(_np(dys) - gys) <= (HALF[dtype] + 2.0 ** -23) * np.abs(gys)).all()
    assert (np.abs(_np(dw) - gw) <= H * 2.0 ** -23 * mag).all()


def test_gradients_are_the_differences(pq):
    """Small integers and weights in eighths: every value is exact in fp32, so central differences of
    <dy, combine(ys, w)> are the gradient exactly, and those of <dxs, dispatch(x)> too."""
    import torch
    rng = np.random.default_rng(7)
    M, k, E, H = 5, 3, 4, 16
    ids = _ids(rng, M, k, E, 0.2)
    plan = pq.moe_sort(_t(ids), E)
    ints = lambda *s: _t(rng.integers(-4, 5, s).astype(np.float32))  # noqa: E731
    ys, w, dy, x, dxs = ints(M * k, H), ints(M, k) / 8, ints(M, H), ints(M, H), ints(M * k, H)
    dys, dw = pq.moe_combine_grad(dy, ys, plan, w)
    dx = pq.moe_dispatch_grad(dxs, plan)
    n = int(plan.offsets[-1])

    def loss(ys, w):
        return (pq.moe_combine(ys, plan, w).double() * dy.double()).sum().item()

    for m in range(M):
        for s in range(k):
            d = torch.zeros_like(w)
            d[m, s] = 1
            assert (loss(ys, w + d) - loss(ys, w - d)) / 2 == dw[m, s].item()
    for r in range(M * k):
        for h in (0, 7, 15):
            d = torch.zeros_like(ys)
            d[r, h] = 1
            assert (loss(ys + d, w) - loss(ys - d, w)) / 2 == dys[r, h].item()
            assert r < n or dys[r, h] == 0
    for m in range(M):
        for h in (0, 9):
            d = torch.zeros_like(x)
            d[m, h] = 1
            up, dn = (pq.moe_dispatch(v, plan).double() * dxs.double() for v in (x + d, x - d))
            assert (up.sum() - dn.sum()).item() / 2 == dx[m, h].item()


def test_rows_past_4_gib(pq):
    """Byte offsets past 32 bits in the sorted rows."""
    import torch
    M, k, E, H = 40000, 8, 64, 8192                 # 5.2 GB of sorted bf16 rows
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.randint(0, E, (M, k), generator=g, device="cuda", dtype=torch.int32)
    x = torch.randn((M, H), generator=g, device="cuda").to(torch.bfloat16)
    plan = pq.moe_sort(ids, E)
    xs = pq.moe_dispatch(x, plan)
    at = torch.cat([torch.arange(100, device="cuda"), torch.arange(M * k - 20000, M * k, device="cuda")])
    assert torch.equal(xs[at], x[plan.order[at].long() // k])
    w = torch.ones((M, k), device="cuda") / 8       # eight equal rows, an eighth each: the row itself, exactly
    y = pq.moe_combine(xs, plan, w)
    assert torch.equal(y, x)
    dys, dw = pq.moe_combine_grad(x, xs, plan, w)
    assert torch.equal(dys[at], (x.float() / 8).to(torch.bfloat16)[plan.order[at].long() // k])
    want = x[-50:].double().square().sum(1, keepdim=True)
    assert ((dw[-50:].double() - want).abs() <= H * 2.0 ** -23 * want).all()


def test_refusals(pq, monkeypatch):
    import torch
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        pq.moe_sort(ids.long(), 4)
    with pytest.raises(ValueError):
        pq.moe_sort(ids[:, :1], 4)
    for bad in (0, 1025, -3, 2 ** 32 + 4):
        with pytest.raises(pq.PqError):
            pq.moe_sort(ids, bad)
    with pytest.raises(pq.PqError):
        pq.moe_sort(ids[:0], 4)
    plan = pq.moe_sort(ids, 4)
    x = torch.zeros((4, 16), device="cuda")
    with pytest.raises(TypeError):
        pq.moe_dispatch(x.half(), plan)
    with pytest.raises(ValueError):
        pq.moe_dispatch(x[:3], plan)
    with pytest.raises(pq.PqError):
        pq.moe_dispatch(torch.zeros((4, 12), device="cuda"), plan)
    with pytest.raises(ValueError):
        pq.moe_dispatch(x, plan._replace(order=plan.order[:4]))
    ys = torch.zeros((8, 16), device="cuda")
    w = torch.zeros((4, 2), device="cuda")
    with pytest.raises(ValueError):
        pq.moe_combine(x, plan, w)
    with pytest.raises(TypeError):
        pq.moe_combine(ys, plan, w.double())
    with pytest.raises(ValueError):
        pq.moe_combine(ys, plan, w[:2])
    with pytest.raises(ValueError):
        pq.moe_combine(ys, plan, w, out=ys[:4])      # an output on top of the rows
    with pytest.raises(TypeError):
        pq.moe_combine_grad(x, ys.to(torch.bfloat16), plan, w)
    with pytest.raises(ValueError):
        pq.moe_combine_grad(x, ys, plan, w, out=torch.zeros((8, 8), device="cuda"))
    monkeypatch.setattr(pq, "_current_device", lambda: 1)
    with pytest.raises(ValueError):
        pq.moe_sort(ids, 4)
