"""The adapters' intermediates h and g are held in 24 bits, whatever the type of the outputs and the size
of the batch.

h = +-(2^23 + 2^11 + v) with v in 1 .. 7 needs all three BF16 parts: 2^23, then 2^11 (what is left of
2^23 + 2^11 + v above 2^23 is a multiple of 16 to 8 bits), then v. Everything else is chosen so that the
products and partial sums are whole numbers below 2^24, exact in FP32 in any order: y is h itself, or the
difference of two such h that leaves v, which BF16 holds too. The same for g with dx, dA and dB.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

bs = pytest.importorskip("lossless_entropy_coding_interleaved_b200")
BF, F32 = torch.bfloat16, torch.float32
BIG, MID = 2.0 ** 23, 2.0 ** 11


def _dev(v, dt=BF):
    return torch.from_numpy(np.ascontiguousarray(v, np.float32)).to(dt).cuda()


def _equal(got, want, what):
    got = got.detach().double().cpu().numpy()
    bad = np.argwhere(got != want)
    assert bad.size == 0, (what, len(bad), bad[:3].tolist(), [(got[tuple(i)], want[tuple(i)]) for i in bad[:3]])


def _batch(tokens, n):
    """An adapter for each token, signs that alternate within each adapter, and the third part's value."""
    idx = (np.arange(tokens) * 5 + np.arange(tokens) // 3) % n
    sign = np.ones(tokens)
    for a in range(n):
        at = np.flatnonzero(idx == a)
        sign[at[1::2]] = -1
    return idx.astype(np.int32), sign, 1.0 + np.arange(tokens) % 7


# 2 adapters: up to 80 tokens go through the kernel for few tokens, more through the tiled ones
@pytest.mark.parametrize("tokens", [1, 40, 300])
@pytest.mark.parametrize("r", [8, 16, 24, 32, 64, 72, 128])
@pytest.mark.parametrize("dt", [F32, BF])
def test_h_keeps_24_bits(tokens, r, dt):
    n, rows, cols = 2, 136, 72
    idx, sign, v = _batch(tokens, n)
    x = np.zeros((tokens, cols))
    x[:, 3], x[:, 17], x[:, 70] = sign * BIG, sign * MID, sign * v
    a = np.zeros((n, r, cols))
    a[:, 0, [3, 17, 70]] = 1      # h_0 = +-(2^23 + 2^11 + v)
    a[:, r - 1, [3, 17]] = 1      # h_{r-1} = +-(2^23 + 2^11)
    b = np.zeros((n, rows, r))
    b[:, 0, 0] = 1                # y_0 = h_0
    b[:, 1::2, 0], b[:, 1::2, r - 1] = 1, -1   # y_1, y_3, .. = +-v
    s = bs.LoraAdapters([_dev(a)], [_dev(b)])
    plan = bs.LoraPlan(tokens, n).update(torch.from_numpy(idx).cuda())
    y, state = torch.full((tokens, rows), 1.0, dtype=dt, device="cuda"), s.state(tokens)
    s.forward(plan, [_dev(x)], [y], state=state)
    want = np.ones((tokens, rows))
    want[:, 0] += sign * (BIG + MID + v)
    want[:, 1::2] += (sign * v)[:, None]
    want = torch.from_numpy(want).to(F32).to(dt).double().numpy()
    _equal(y, want, "y")
    # dB = sum dy h with dy = 1 in rows 2 and 5: alternating signs leave at most one h
    dy = np.zeros((tokens, rows))
    dy[:, [2, 5]] = 1
    das, dbs = [torch.empty(a.shape, device="cuda")], [torch.empty(b.shape, device="cuda")]
    s.backward(plan, [_dev(x)], [_dev(dy)], state, das, dbs)
    want = np.zeros(b.shape)
    for i in range(n):
        at = idx == i
        want[i, [2, 5], 0] += np.sum(sign[at] * (BIG + MID + v[at]))
        want[i, [2, 5], r - 1] += np.sum(sign[at] * (BIG + MID))
    _equal(dbs[0], want, "db")
    assert int(plan.err) == 0


@pytest.mark.parametrize("tokens", [1, 40, 300])
@pytest.mark.parametrize("r", [8, 16, 24, 32, 64, 72, 128])
@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("sources", [1, 3])
def test_g_keeps_24_bits(tokens, r, dt, sources):
    n, rows, cols = 2, 72, 136
    idx, sign, v = _batch(tokens, n)
    dy = np.zeros((tokens, rows))
    dy[:, 3], dy[:, 17], dy[:, 70] = sign * BIG, sign * MID, sign * v
    b = np.zeros((n, rows, r))
    b[:, [3, 17, 70], 0] = 1
    b[:, [3, 17], r - 1] = 1
    a = np.zeros((n, r, cols))
    a[:, 0, 0] = 1
    a[:, 0, 1::2], a[:, r - 1, 1::2] = 1, -1
    x = np.zeros((tokens, cols))
    x[:, [2, 5]] = 1
    first = np.zeros_like(a)  # the other sources add nothing to column 0
    first[:, 0, 1::2], first[:, r - 1, 1::2] = 1, -1
    s = bs.LoraAdapters([_dev(a)] + [_dev(first)] * (sources - 1), [_dev(b)] * sources)
    plan = bs.LoraPlan(tokens, n).update(torch.from_numpy(idx).cuda())
    xs, state = [_dev(x)] * sources, s.state(tokens)
    s.forward(plan, xs, state=state)
    das, dbs = [torch.empty(a.shape, device="cuda") for _ in xs], [torch.empty(b.shape, device="cuda") for _ in xs]
    dx = torch.full((tokens, cols), float("nan"), dtype=dt, device="cuda")
    s.backward(plan, xs, [_dev(dy)] * sources, state, das, dbs, dxs=[dx] * sources)
    want = np.zeros((tokens, cols))
    want[:, 0] = sign * (BIG + MID + v)
    want[:, 1::2] = sources * (sign * v)[:, None]
    _equal(dx, torch.from_numpy(want).to(F32).to(dt).double().numpy(), "dx")
    want = np.zeros(a.shape)
    for i in range(n):
        at = idx == i
        want[i, 0, [2, 5]] += np.sum(sign[at] * (BIG + MID + v[at]))
        want[i, r - 1, [2, 5]] += np.sum(sign[at] * (BIG + MID))
    for k in range(sources):
        _equal(das[k], want, ("da", k))
    assert int(plan.err) == 0
