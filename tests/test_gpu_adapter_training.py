"""Adapters trained beside a frozen, coded projection, and served: the products, the gradients, the
norm and the step as a program runs them, and the trained pools through the encoder.

Two projections of the same x, W in the fixed-width layout (bs_fw_gemm, bs_fw_gemv), three adapters.
Every step's outputs are held against the same step in 64 bits from the pools as they then are, within
the bounds of the single operators: a sum of K exact products in FP32 is off by at most 4 K 2^-24 of
the sum of their magnitudes; an escaped weight of W enters as a placeholder and a correction, whose
magnitude is below that of twice the largest weight (the tolerance takes K of them).
"""
import numpy as np
import pytest
import torch

import adamw_plain as A
import lora_plain as L

pytestmark = pytest.mark.gpu

bs = pytest.importorskip("lossless_entropy_coding_interleaved_b200")
BF, U = torch.bfloat16, 2.0 ** -24
ROWS, COLS, N, R = (256, 128), 512, 3, 16
RANKS = [16, 5, 9]


def _make(seed, tokens):
    g = torch.Generator("cuda").manual_seed(seed)
    rnd = lambda *s, scale=1.0: (torch.randn(*s, generator=g, device="cuda") * scale).to(BF)  # noqa: E731
    o = type("O", (), {})()
    o.w = [rnd(r, COLS, scale=0.05) for r in ROWS]
    o.fw = [bs.fw_transcode(w.view(torch.int16).reshape(-1)) for w in o.w]
    o.a, o.b = [rnd(N, R, COLS, scale=COLS ** -0.5) for _ in ROWS], [rnd(N, r, R, scale=0.1) for r in ROWS]
    o.scales = torch.tensor([1.0, 0.5, 2.0], device="cuda")
    o.set = bs.LoraAdapters(o.a, o.b, o.scales, torch.tensor(RANKS, dtype=torch.int32, device="cuda"))
    o.idx = (torch.arange(tokens, dtype=torch.int32, device="cuda") * 7 // 5) % (N + 1) - 1
    o.plan = bs.LoraPlan(tokens, N).update(o.idx)
    o.x, o.dy = rnd(tokens, COLS), [rnd(tokens, r, scale=0.1) for r in ROWS]
    o.y = [torch.zeros(tokens, r, device="cuda") for r in ROWS]
    o.state, o.work = o.set.state(tokens), o.set.state(tokens)
    o.da, o.db = [torch.zeros(t.shape, device="cuda") for t in o.a], [torch.zeros(t.shape, device="cuda") for t in o.b]
    o.dx = torch.zeros(tokens, COLS, device="cuda")
    o.err = torch.zeros(1, dtype=torch.int32, device="cuda")
    o.products = [(f, i, r, COLS, o.x, y) for (f, i), r, y in zip(o.fw, ROWS, o.y)]
    return o


def _np(t):
    return t.detach().double().cpu().numpy()


def _near(got, want, tol, what):
    bad = np.argwhere(~(np.abs(_np(got) - want) <= tol + 1e-30))
    assert bad.size == 0, (what, bad[:3].tolist())


def _step(o, opt):
    bs.fw_gemm(o.products, o.err, adapters=(o.set, o.plan, o.state))
    o.set.backward(o.plan, [o.x] * 2, o.dy, o.state, o.da, o.db, dxs=[o.dx] * 2, work=o.work)
    opt.step(max_norm=1.0)


def _check_products(o, y):
    x, idx, sc = _np(o.x), o.idx.cpu().numpy(), _np(o.scales)
    for k in range(2):
        w, a, b = _np(o.w[k]), _np(o.a[k]), _np(o.b[k])
        want, _ = L.forward(x, idx, a, b, sc, RANKS, x @ w.T)
        mag, _ = L.forward(abs(x), idx, abs(a), abs(b), sc, RANKS, abs(x) @ (abs(w).T + 2 * abs(w).max()))
        _near(y[k], want, 4 * U * (COLS + 3 * R) * mag, ("y", k))


def test_training_beside_a_coded_projection():
    o = _make(1, 200)
    params = o.a + o.b
    opt = bs.AdamW(params, o.da + o.db, lr=1e-2, weight_decay=0.1, masters=[p.float() for p in params])
    for t in range(1, 4):
        before = [_np(p) for p in params]
        pools = [v.clone() for v in params]
        masters, ms, vs = ([v.clone() for v in ts] for ts in (opt.masters, opt.exp_avg, opt.exp_avg_sq))
        _step(o, opt)
        torch.cuda.synchronize()
        assert int(o.err) == 0 and int(o.plan.err) == 0 and int(opt.steps) == t
        after = [p.clone() for p in params]
        for p, old in zip(params, pools):  # the products of this step came from the pools before it
            p.copy_(old)
        _check_products(o, o.y)
        for p, new in zip(params, after):
            p.copy_(new)
        x, idx, sc, dx, tol_dx = _np(o.x), o.idx.cpu().numpy(), _np(o.scales), 0, 0
        for k in range(2):
            dy = _np(o.dy[k])
            pdx, da, db = L.backward(x, dy, idx, before[k], before[2 + k], sc, RANKS, np.zeros_like(x))
            mdx, ma, mb = L.backward(abs(x), abs(dy), idx, abs(before[k]), abs(before[2 + k]), sc, RANKS, np.zeros_like(x))
            dx, tol_dx = dx + pdx, tol_dx + 4 * U * (ROWS[k] + 3 * R) * mdx
            _near(o.da[k], da, 4 * U * (ROWS[k] + 600) * ma, ("da", t, k))
            _near(o.db[k], db, 4 * U * (COLS + 600) * mb, ("db", t, k))
        _near(o.dx, dx, tol_dx, ("dx", t))
        grads = [_np(g) for g in o.da + o.db]
        norm = np.sqrt(sum((g ** 2).sum() for g in grads))
        assert abs(float(opt.norm) - norm) <= 40 * U * norm
        clip = float(opt.clip)
        for p, old, g, m, v, master in zip(params, masters, grads, ms, vs, opt.masters):
            want, m1, _ = A.step(_np(old), g, _np(m).reshape(g.shape), _np(v).reshape(g.shape), t, 1e-2, (0.9, 0.999), 1e-8, float(np.float32(0.1)), clip, np.float64)
            # the step is at most lr / (1 - 0.9) long; 64 roundings of it and of the parameter
            _near(master, want, 64 * U * (np.abs(want) + 0.1), "master")
            assert torch.equal(p, master.to(BF))
    # what was trained is coded and decoded to the same words
    d, _ = bs.encode([("p%d" % k, p) for k, p in enumerate(params)], model="joint")
    plan = bs.Plan(d_container=d)
    for k, p in enumerate(params):
        assert torch.equal(plan.decode(k).view(BF).view(p.shape), p)
    plan.check()


def test_a_captured_training_step_is_the_eager_one():
    a, b = _make(2, 70), _make(2, 70)
    opts = [bs.AdamW(o.a + o.b, o.da + o.db, bits=8, lr=1e-2, seed=5) for o in (a, b)]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        _step(b, opts[1])
    for _ in range(4):
        _step(a, opts[0])
        graph.replay()
        torch.cuda.synchronize()
        for s, t in zip(a.a + a.b + a.da + a.db + a.y + [a.dx], b.a + b.b + b.da + b.db + b.y + [b.dx]):
            assert torch.equal(s, t)
    assert int(opts[1].steps) == 4


@pytest.mark.parametrize("tokens", [1, 5, 8])
def test_serving_few_tokens(tokens):
    o = _make(3, tokens)
    bs.fw_gemv(o.products, o.err, layouts_resident=True, adapters=(o.set, o.plan))
    torch.cuda.synchronize()
    assert int(o.err) == 0 and int(o.plan.err) == 0
    _check_products(o, o.y)
    if tokens == 1:  # vectors instead of one-row matrices
        y = [torch.zeros(r, device="cuda") for r in ROWS]
        bs.fw_gemv([(f, i, r, COLS, o.x.view(-1).view(torch.int16), v) for (f, i), r, v in zip(o.fw, ROWS, y)], o.err, adapters=(o.set, o.plan))
        assert all(torch.equal(u, v[0]) for u, v in zip(y, o.y))
