"""Infinities and NaN in x and dy: every output has them where the formula in 64 bits has them, and the exact
whole number everywhere else, on the kernel for few tokens and on the tiled ones, at every padded rank.

Weights are whole numbers, 0 among them (0 times infinity is NaN in the formula too). The rank rows past an
adapter's rank hold NaN in the pools and have gradients of 0.
"""
import numpy as np
import pytest
import torch

import lora_plain as L

pytestmark = pytest.mark.gpu

bs = pytest.importorskip("lossless_entropy_coding_interleaved_b200")
BF, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


def _dev(v, dt=BF):
    return torch.from_numpy(np.ascontiguousarray(v, np.float32)).to(dt).cuda()


def _equal(got, want, what):
    got = got.detach().double().cpu().numpy()
    bad = np.argwhere(~((got == want) | (np.isnan(got) & np.isnan(want))))
    assert bad.size == 0, (what, len(bad), bad[:3].tolist(), [(got[tuple(i)], want[tuple(i)]) for i in bad[:3]])


# x at (token, column) and dy at (token, row) of each adapter's tokens; every adapter has one kind, the last none
KINDS = [dict(x=[INF]), dict(dy=[INF]), dict(x=[-INF, INF]), dict(dy=[INF, -INF]), dict(x=[NAN]), dict(dy=[NAN]), dict(x=[INF], dy=[-INF]),
         dict(x=[INF, NAN, -INF]), dict(dy=[INF, INF, -INF]), {}]


# 60: the kernel for few tokens; 9000: sums over several chains of matrix instructions, and over CTAs
@pytest.mark.parametrize("tokens", [60, 700, 9000])
@pytest.mark.parametrize("r", [8, 16, 32, 64, 72, 128])
@pytest.mark.parametrize("dt", [F32, BF])
def test_infinities_and_nan_stand_where_the_formula_has_them(tokens, r, dt):
    rng = np.random.default_rng(r + tokens)
    n, rows, cols = len(KINDS), 136, 264
    ranks = np.array([r - (3 * i) % r for i in range(n)], np.int32)
    a, b = rng.integers(-1, 2, (n, r, cols)).astype(np.float64), rng.integers(-1, 2, (n, rows, r)).astype(np.float64)
    idx = rng.integers(-1, n, tokens).astype(np.int32)
    idx[:n] = np.arange(n)
    x, dy = rng.integers(-2, 3, (tokens, cols)).astype(np.float64), rng.integers(-1, 2, (tokens, rows)).astype(np.float64)
    for i, kind in enumerate(KINDS):
        at = np.flatnonzero(idx == i)
        for v, width, bad in ((x, cols, kind.get("x", [])), (dy, rows, kind.get("dy", []))):
            for k, value in enumerate(bad):
                v[at[len(at) * k // 3], 37 + 50 * (k % 2)] = value
    off = np.flatnonzero(idx < 0)
    x[off], dy[off] = NAN, INF  # padding: reaches nothing
    pa, pb = a.copy(), b.copy()
    for i in range(n):
        pa[i, ranks[i]:], pb[i, :, ranks[i]:] = NAN, NAN
    s = bs.LoraAdapters([_dev(pa)], [_dev(pb)], None, torch.from_numpy(ranks).cuda())
    plan = bs.LoraPlan(tokens, n).update(torch.from_numpy(idx).cuda())
    state, y, dx = s.state(tokens), torch.full((tokens, rows), 3.0, dtype=dt, device="cuda"), torch.empty(tokens, cols, dtype=dt, device="cuda")
    das, dbs = [torch.empty(a.shape, device="cuda")], [torch.empty(b.shape, device="cuda")]
    s.forward(plan, [_dev(x)], [y], state=state)
    s.backward(plan, [_dev(x)], [_dev(dy)], state, das, dbs, dxs=[dx])
    with np.errstate(invalid="ignore"):
        want_y, _ = L.forward(x, idx, pa, pb, np.ones(n), ranks, np.full((tokens, rows), 3.0))
        want_dx, want_da, want_db = L.backward(x, dy, idx, pa, pb, np.ones(n), ranks, np.zeros((tokens, cols)))
    rounded = lambda v: torch.from_numpy(v).to(F32).to(dt).double().numpy()  # noqa: E731
    _equal(y, rounded(want_y), "y")
    _equal(dx, rounded(want_dx), "dx")
    _equal(das[0], want_da, "da")
    _equal(dbs[0], want_db, "db")
    assert int(plan.err) == 0
    # added to what is there: the rows past a rank stay as they are
    das, dbs = [torch.full(a.shape, 5.0, device="cuda")], [torch.full(b.shape, 5.0, device="cuda")]
    s.backward(plan, [_dev(x)], [_dev(dy)], state, das, dbs, accumulate=True)
    _equal(das[0], want_da + 5, "da")
    _equal(dbs[0], want_db + 5, "db")
