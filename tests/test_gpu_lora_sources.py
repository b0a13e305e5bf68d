"""dx of many projections: the chains of matrix instructions whose sums the tensor cores round towards zero stay
short whatever their number.

Source 0 gives 2^24, each other one 1.875, all of them exact in one link. FP32 has a spacing of 2 there, so a chain
that adds them one by one to 2^24 loses every one of them, 15 x 1.875 in all. A chain holds 3 sources at rank
128 and 64, 6 and 12 at 32 and 16: the first chain may lose its others (2 each at most), and each chain's sum is
added in FP32 and rounded to nearest, by 1 at most.
"""
import numpy as np
import pytest
import torch

import lora_plain as L

pytestmark = pytest.mark.gpu

bs = pytest.importorskip("lossless_entropy_coding_interleaved_b200")
BF, F32 = torch.bfloat16, torch.float32


def _dev(v, dt=BF):
    return torch.from_numpy(np.ascontiguousarray(v, np.float32)).to(dt).cuda()


@pytest.mark.parametrize("tokens", [5, 300])
@pytest.mark.parametrize("r,each", [(8, 12), (16, 12), (32, 6), (64, 3), (128, 3)])
@pytest.mark.parametrize("base", [False, True])
def test_many_small_parts_beside_a_large_one(tokens, r, each, base):
    n, rows, cols, sources = 2, 64, 200, 16
    a = np.zeros((n, r, cols))
    a[:, 0] = 1
    b = np.zeros((n, rows, r))
    b[:, 3, 0] = 1
    s = bs.LoraAdapters([_dev(a)] * sources, [_dev(b)] * sources)
    idx = (np.arange(tokens) % n).astype(np.int32)
    plan = bs.LoraPlan(tokens, n).update(torch.from_numpy(idx).cuda())
    dys = []
    for k in range(sources):
        dy = np.zeros((tokens, rows))
        dy[:, 3] = 2.0 ** 24 if k == 0 else 1.875
        dys.append(_dev(dy))
    x = torch.zeros(tokens, cols, dtype=BF, device="cuda")
    das, dbs = [torch.empty(a.shape, device="cuda") for _ in dys], [torch.empty(b.shape, device="cuda") for _ in dys]
    state = s.state(tokens)
    s.forward(plan, [x] * sources, state=state)
    dx = torch.empty(tokens, cols, device="cuda")
    start = torch.full((tokens, cols), -2.0 ** 24, device="cuda")  # exact: what is left of the sum is small
    s.backward(plan, [x] * sources, dys, state, das, dbs, dxs=[dx] * sources, dx_bases=[start] * sources if base else None)
    want = (0 if base else 2.0 ** 24) + 15 * 1.875
    chains = -(-sources // each)
    assert int(plan.err) == 0
    assert float((dx.double() - want).abs().max()) <= 2 * (each - 1) + (chains - 1) + (0 if base else 1)


@pytest.mark.parametrize("tokens", [150, 700])
@pytest.mark.parametrize("r", [16, 32, 64, 128])
@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("sources", [2, 4, 7, 13, 16])
def test_sources_by_the_dozen_are_all_there(tokens, r, dt, sources):
    # whole numbers: exact whatever the order. Tokens without an adapter keep their base; a rank of 0 too
    rng = np.random.default_rng(sources)
    n, rows, cols = 3, 72, 1032
    ranks = np.array([r, 0, max(1, r - 5)], np.int32)
    a, b = (rng.integers(-1, 2, (sources, n) + shape).astype(np.float64) for shape in ((r, cols), (rows, r)))
    idx = rng.integers(-1, n, tokens).astype(np.int32)
    x, base = rng.integers(-1, 2, (tokens, cols)).astype(np.float64), rng.integers(-3, 4, (tokens, cols)).astype(np.float64)
    dys = rng.integers(-1, 2, (sources, tokens, rows)).astype(np.float64)
    s = bs.LoraAdapters([_dev(v) for v in a], [_dev(v) for v in b], None, torch.from_numpy(ranks).cuda())
    plan = bs.LoraPlan(tokens, n).update(torch.from_numpy(idx).cuda())
    state, xs = s.state(tokens), [_dev(x)] * sources
    s.forward(plan, xs, state=state)
    das, dbs = [torch.empty(v.shape, device="cuda") for v in a], [torch.empty(v.shape, device="cuda") for v in b]
    want = base.copy()
    for k in range(sources):
        want += L.backward(x, dys[k], idx, a[k], b[k], np.ones(n), ranks, np.zeros_like(x))[0]
    assert np.abs(want).max() < 2 ** 24
    want = torch.from_numpy(want).to(F32).to(dt)
    for in_place in (False, True):
        bd = _dev(base, dt)
        dx = bd if in_place else torch.empty_like(bd)
        s.backward(plan, xs, [_dev(v) for v in dys], state, das, dbs, dxs=[dx] * sources, dx_bases=[bd] * sources)
        assert torch.equal(dx.cpu(), want), in_place
    assert int(plan.err) == 0


@pytest.mark.parametrize("tokens", [1, 40, 300])
@pytest.mark.parametrize("r", [16, 32, 64, 128])
def test_lower_parts_are_added_up_before_they_meet_a_large_sum(tokens, r):
    # h_0 = 2^24, then pairs of 1024 + 15/64 and -1024, whose upper parts cancel: y is 2^24 + (r/2 - 1) 15/64. 8 pairs
    # are a matrix instruction, 1.875 of the lower parts together: at the size of 2^24 each of them would be lost. Added
    # up first they are exact, and one rounding towards zero, by less than 2, is left
    n, rows, cols = 2, 72, 136
    x = np.zeros((tokens, cols))
    x[:, 0], x[:, 60], x[:, 130] = 2.0 ** 24, 1024, 15 / 64
    a = np.zeros((n, r, cols))
    a[:, 0, 0] = 1
    a[:, 2::2, 60], a[:, 2::2, 130] = 1, 1
    a[:, 3::2, 60] = -1
    b = np.ones((n, rows, r))
    s = bs.LoraAdapters([_dev(a)], [_dev(b)])
    plan = bs.LoraPlan(tokens, n).update((torch.arange(tokens, device="cuda") % n).int())
    y = torch.full((tokens, rows), -2.0 ** 24, device="cuda")
    s.forward(plan, [_dev(x)], [y])
    assert int(plan.err) == 0
    assert float((y.double() - (r // 2 - 1) * 15 / 64).abs().max()) < 2
