"""Forms of the adapters' calls: rows with gaps on every side, outputs of both types in one call, gradients added to in
place, and calls whose x is what the call before wrote. Whole numbers: exact, in any order.
"""
import numpy as np
import pytest
import torch

import lora_plain as L

pytestmark = pytest.mark.gpu

bs = pytest.importorskip("lossless_entropy_coding_interleaved_b200")
BF, F32 = torch.bfloat16, torch.float32


def _dev(v, dt=BF, gap=0):
    """v on the device, `gap` more elements between rows, 77 in them."""
    v = np.ascontiguousarray(v, np.float32)
    t = torch.full((*v.shape[:-1], v.shape[-1] + gap), 77.0, dtype=dt, device="cuda")
    t[..., :v.shape[-1]] = torch.from_numpy(v).to(dt)
    return t[..., :v.shape[-1]]


def _gaps_kept(t, gap):
    return gap == 0 or bool((t.as_strided((t.shape[0] - 1, gap), (t.stride(0), 1), t.storage_offset() + t.shape[1]) == 77).all())


def _as(v, dt):
    return torch.from_numpy(v).to(F32).to(dt)


class Made:
    def __init__(self, tokens, r, projs, n=3, seed=0):
        rng = np.random.default_rng(seed + r + tokens)
        self.rng, self.n, self.tokens, self.projs = rng, n, tokens, projs
        self.ranks = np.array(([r, max(1, r - 5), 0] * n)[:n], np.int32)
        self.a = [rng.integers(-1, 2, (n, r, c)).astype(np.float64) for _, c in projs]
        self.b = [rng.integers(-1, 2, (n, rows, r)).astype(np.float64) for rows, _ in projs]
        self.idx = rng.integers(-1, n, tokens).astype(np.int32)
        self.scales = 2.0 ** rng.integers(-1, 2, n)
        self.set = bs.LoraAdapters([_dev(v) for v in self.a], [_dev(v) for v in self.b], _dev(self.scales, F32).contiguous(),
                                   torch.from_numpy(self.ranks).cuda())
        self.plan = bs.LoraPlan(tokens, n).update(torch.from_numpy(self.idx).cuda())

    def whole(self, *shape, most=2):
        return self.rng.integers(-most, most + 1, shape).astype(np.float64)

    def forward(self, k, x, base):
        return L.forward(x, self.idx, self.a[k], self.b[k], self.scales, self.ranks, base)[0]

    def backward(self, k, x, dy, base):
        return L.backward(x, dy, self.idx, self.a[k], self.b[k], self.scales, self.ranks, base)


# 50: the kernel for few tokens (forward); 400: the tiled ones
@pytest.mark.parametrize("tokens", [2, 50, 400])
@pytest.mark.parametrize("r", [8, 16, 24, 32, 64, 72, 128])
@pytest.mark.parametrize("dt", [F32, BF])
def test_rows_with_gaps_everywhere(tokens, r, dt):
    rows, cols = 136, 200
    m = Made(tokens, r, [(rows, cols)])
    x, dy, by, bx = m.whole(tokens, cols), m.whole(tokens, rows, most=1), m.whole(tokens, rows), m.whole(tokens, cols)
    xd, dyd, byd, bxd = _dev(x, BF, 8), _dev(dy, BF, 16), _dev(by, dt, 24), _dev(bx, dt, 40)
    y, dx, state = _dev(0 * by, dt, 32), _dev(0 * bx, dt, 8), m.set.state(tokens)
    das, dbs = [torch.empty(m.a[0].shape, device="cuda")], [torch.empty(m.b[0].shape, device="cuda")]
    m.set.forward(m.plan, [xd], [y], [byd], state)
    m.set.backward(m.plan, [xd], [dyd], state, das, dbs, [dx], [bxd])
    want_dx, want_da, want_db = m.backward(0, x, dy, bx)
    assert torch.equal(y.cpu(), _as(m.forward(0, x, by), dt)) and torch.equal(dx.cpu(), _as(want_dx, dt))
    assert torch.equal(das[0].cpu(), _as(want_da, F32)) and torch.equal(dbs[0].cpu(), _as(want_db, F32))
    # the same in place, with gaps
    m.set.forward(m.plan, [xd], [byd], state=state)
    m.set.backward(m.plan, [xd], [dyd], state, das, dbs, [bxd], [bxd])
    assert torch.equal(byd, y) and torch.equal(bxd, dx)
    for t, gap in ((xd, 8), (dyd, 16), (byd, 24), (bxd, 40), (y, 32), (dx, 8)):
        assert _gaps_kept(t, gap)
    assert int(m.plan.err) == 0


@pytest.mark.parametrize("tokens", [50, 400])
@pytest.mark.parametrize("r", [16, 64, 128])
@pytest.mark.parametrize("base", [False, True])
def test_outputs_of_both_types_in_one_call(tokens, r, base):
    projs = [(136, 200), (264, 72), (72, 200), (16, 136), (136, 72)]
    types = [F32, BF, BF, F32, F32]
    m = Made(tokens, r, projs)
    xs = [m.whole(tokens, c) for _, c in projs]
    dys = [m.whole(tokens, rows, most=1) for rows, _ in projs]
    bys = [m.whole(tokens, rows) if base else np.zeros((tokens, rows)) for rows, _ in projs]
    bxs = [m.whole(tokens, c) if base else np.zeros((tokens, c)) for _, c in projs]
    xd, dyd = [_dev(v) for v in xs], [_dev(v) for v in dys]
    ys, dxs = [torch.empty(tokens, rows, dtype=t, device="cuda") for (rows, _), t in zip(projs, types)], [torch.empty(tokens, c, dtype=t, device="cuda") for (_, c), t in zip(projs, types)]
    dxs[3] = None  # and one dx that is not wanted
    state = m.set.state(tokens)
    das, dbs = [torch.empty(v.shape, device="cuda") for v in m.a], [torch.empty(v.shape, device="cuda") for v in m.b]
    for _ in range(2):
        m.set.forward(m.plan, xd, ys, [_dev(v, t) if base else None for v, t in zip(bys, types)], state)
        m.set.backward(m.plan, xd, dyd, state, das, dbs, dxs, [_dev(v, t) if base and k != 3 else None for k, (v, t) in enumerate(zip(bxs, types))])
    for k in range(5):
        want_dx, want_da, want_db = m.backward(k, xs[k], dys[k], bxs[k])
        assert torch.equal(ys[k].cpu(), _as(m.forward(k, xs[k], bys[k]), types[k])), k
        assert dxs[k] is None or torch.equal(dxs[k].cpu(), _as(want_dx, types[k])), k
        assert torch.equal(das[k].cpu(), _as(want_da, F32)) and torch.equal(dbs[k].cpu(), _as(want_db, F32)), k
    assert int(m.plan.err) == 0


@pytest.mark.parametrize("tokens", [6, 50, 400])
def test_calls_whose_x_the_call_before_wrote(tokens):
    # a chain of layers, y in BF16 as the next one's x, through the adapters and through a coded product, many times
    # over with nothing in between; and the routing written just before the plan that reads it
    width = 256
    m = Made(tokens, 16, [(width, width)], n=4)
    x = m.whole(tokens, width, most=1)
    first = _dev(x)
    w = m.whole(width, width, most=1)
    fw, info = bs.fw_transcode(_dev(w).view(torch.int16).reshape(-1))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    bufs, out = [torch.zeros(tokens, width, dtype=BF, device="cuda") for _ in range(3)], torch.zeros(tokens, width, device="cuda")
    idx, plan, product = torch.from_numpy(m.idx).cuda(), bs.LoraPlan(tokens, 4), bs.fw_gemv if tokens <= 8 else bs.fw_gemm
    mine = torch.full_like(idx, -1)
    # every layer by itself, waiting for each
    want, at = [], first
    for _ in range(3):
        y = torch.zeros(tokens, width, dtype=BF, device="cuda")
        m.set.forward(m.plan, [at], [y])
        torch.cuda.synchronize()
        want.append(y)
        at = y
    got = torch.zeros(tokens, width, device="cuda")
    torch.cuda.synchronize()
    product([(fw, info, width, width, want[-1], got)], err)
    torch.cuda.synchronize()
    for _ in range(50):
        for t in bufs:
            t.zero_()
        mine.copy_(idx)
        plan.update(mine)
        m.set.forward(plan, [first], [bufs[0]])
        m.set.forward(plan, [bufs[0]], [bufs[1]])
        m.set.forward(plan, [bufs[1]], [bufs[2]])
        product([(fw, info, width, width, bufs[2], out)], err)
        assert all(torch.equal(a, b) for a, b in zip(bufs, want)) and torch.equal(out, got)
    assert int(err) == 0 and int(plan.err) == 0


@pytest.mark.parametrize("pairs", [((16, 300), (64, 300)), ((64, 1500), (8, 1500)), ((128, 300), (16, 900)), ((32, 700), (32, 40)), ((64, 400), (64, 400))])
def test_two_batches_at_once_on_two_streams(pairs):
    made, streams = [], [torch.cuda.Stream() for _ in pairs]
    for seed, (r, tokens) in enumerate(pairs):
        m = Made(tokens, r, [(1024, 512), (512, 512)], n=5, seed=seed)
        m.x, m.dy = [_dev(m.whole(tokens, 512))] * 2, [_dev(m.whole(tokens, rows, most=1)) for rows, _ in m.projs]
        m.state, m.work = m.set.state(tokens), m.set.state(tokens)

        def go(m=m, stream=None):
            o = dict(ys=[torch.zeros(m.tokens, rows, device="cuda") for rows, _ in m.projs], das=[torch.zeros(v.shape, device="cuda") for v in m.a],
                     dbs=[torch.zeros(v.shape, device="cuda") for v in m.b], dx=[torch.zeros(m.tokens, 512, device="cuda")])
            if stream is not None:
                stream.wait_stream(torch.cuda.current_stream())
            for _ in range(30):
                m.set.forward(m.plan, m.x, o["ys"], [None] * 2, state=m.state, stream=stream)
                m.set.backward(m.plan, m.x, m.dy, m.state, o["das"], o["dbs"], o["dx"] * 2, work=m.work, stream=stream)
            return o
        made.append(go)
    alone = [go() for go in made]
    torch.cuda.synchronize()
    together = [go(stream=s) for go, s in zip(made, streams)]
    torch.cuda.synchronize()
    for a, b in zip(alone, together):
        for k in a:
            assert all(torch.equal(u, v) for u, v in zip(a[k], b[k])), k
