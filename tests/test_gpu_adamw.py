"""bs_adamw, bs_grad_norm and bs_adamw_read_states on the GPU against numpy.

Tolerances, in roundings of 2^-24 each. m: a term of it has its factor, the clip product, the
product and the sum rounded: 4 of the sum of the terms' magnitudes (they can cancel). v: its factor,
the clip product (squared: 2), two products and the sum: 6, taken as 8. The step
s = lr / c1 * m / (sqrt(v) r + eps): lr 1, c1 4 (its argument and two units in the last place of
expm1f), their quotient 1, r 2 + 4 (half of c2's, two units of rsqrtf), root 2 + half of v's 8,
product 1, sum 1, quotient 4 (two units), product 1: 24, plus m's own; the parameter is rounded
three times on its way: 3 of (|p| + |s|). A BF16 parameter is rounded once more, 2^-8 of its value.
8-bit codes have to be equal to those of the same formula in rounded FP32 operations, bit for bit.
"""
import numpy as np
import pytest
import torch

import adamw_plain as A

pytestmark = pytest.mark.gpu

bs = pytest.importorskip("lossless_entropy_coding_interleaved_b200")
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def _tensor(n, dt, rng, scale, offset=0):
    """n values in a buffer of their own, `offset` elements behind its aligned start."""
    t = torch.zeros(n + offset + 8, dtype=dt, device="cuda")[offset:offset + n]
    t.copy_(torch.from_numpy((rng.standard_normal(n) * scale).astype(np.float32)))
    return t


def _np(t):
    return t.detach().float().cpu().numpy()


def _close(got, want, tol, what):
    err = np.abs(got.astype(np.float64) - want)
    bad = np.flatnonzero(~(err <= tol))
    assert bad.size == 0, (what, bad[:4], got[bad[:4]], want[bad[:4]], tol[bad[:4]])


def _check_step(p0, g0, m0, v0, p1, m1, v1, t, lr, betas, eps, decay, clip, param_bf16):
    """One tensor: values before (numpy float32) and after."""
    p, m, v = A.step(p0, g0, m0, v0, t, lr, betas, eps, decay, clip, np.float64)
    gc = np.abs(g0.astype(np.float64) * clip)
    tm = 4 * U * (betas[0] * np.abs(m0) + (1 - betas[0]) * gc) + 1e-45
    tv = 8 * U * v + 1e-45
    if m1 is not None:
        _close(m1, m, tm, "m")
        _close(v1, v, tv, "v")
    c1, r2 = 1 - betas[0] ** t, np.sqrt(1 - betas[1] ** t)
    den = np.sqrt(v) / r2 + eps
    tol = lr / c1 / den * (24 * U * np.abs(m) + tm) + 3 * U * (np.abs(p0) + np.abs(p)) + 1e-45
    if param_bf16:
        tol = tol + 2.0 ** -8 * (np.abs(p) + tol)
    _close(p1, p, tol, "p")


CASES32 = [([1], F32, F32, False), ([255, 256, 257, 4097], F32, F32, False), ([1000, 3, 8192], BF, BF, False),
           ([70000, 1, 5], BF, F32, True), ([513] * 700, F32, BF, False), ([0, 77, 0], BF, BF, True)]


@pytest.mark.parametrize("sizes,pt,gt,master", CASES32)
@pytest.mark.parametrize("offset", [0, 1])
def test_step_in_32_bits(sizes, pt, gt, master, offset):
    rng = np.random.default_rng(5 + offset)
    ps = [_tensor(n, pt, rng, 0.02, offset) for n in sizes]
    gs = [_tensor(n, gt, rng, 0.01, offset) for n in sizes]
    ms, vs = ([_tensor(n, F32, rng, 0.003, offset) for n in sizes] for _ in range(2))
    for v in vs:
        v.square_()
    masters = [_tensor(n, F32, rng, 0.02, offset) for n in sizes] if master else None
    decay = [0.1 * (k % 3) for k in range(len(sizes))]
    kw = dict(lr=2e-3, betas=(0.9, 0.999), eps=1e-8)
    opt = bs.AdamW(ps, gs, weight_decay=decay, masters=masters, step=11, clip=0.5, states=(ms, vs), **kw)
    before = [[_np(t) for t in ts] for ts in (masters or ps, gs, ms, vs)]
    opt.step()
    torch.cuda.synchronize()
    assert int(opt.steps) == 12
    for k in range(len(sizes)):
        after = _np(masters[k]) if master else _np(ps[k])
        _check_step(*[b[k] for b in before], after, _np(ms[k]), _np(vs[k]), 12, kw["lr"], kw["betas"], kw["eps"],
                    float(np.float32(decay[k])), 0.5, not master and pt is BF)
        if master:
            assert torch.equal(ps[k].float(), masters[k].to(pt).float()), k


@pytest.mark.parametrize("sizes,pt,gt", [([1], F32, F32), ([255, 256, 257, 1], F32, BF), ([65536, 4099], BF, BF),
                                         ([300] * 400, F32, F32)])
@pytest.mark.parametrize("offset", [0, 3])
def test_steps_in_8_bits_are_the_formulas_bits(sizes, pt, gt, offset):
    rng = np.random.default_rng(9)
    ps = [_tensor(n, pt, rng, 0.02, offset) for n in sizes]
    gs = [_tensor(n, gt, rng, 0.01, offset) for n in sizes]
    betas, eps, lr, seed = (0.9, 0.999), 1e-8, 1e-3, 12345678901234567890
    codes = [torch.zeros(n + 16, dtype=torch.uint8, device="cuda")[offset:offset + n] for n in sizes for _ in range(2)]
    scales = [torch.zeros(-(-n // 256), device="cuda") for n in sizes for _ in range(2)]
    opt = bs.AdamW(ps, gs, lr=lr, betas=betas, eps=eps, weight_decay=0.1, bits=8, seed=seed, clip=0.75,
                   states=((codes[::2], scales[::2]), (codes[1::2], scales[1::2])))
    host = [dict(mc=np.zeros(n, np.uint8), vc=np.zeros(n, np.uint8), ms=np.zeros(-(-n // 256), np.float32),
                 vs=np.zeros(-(-n // 256), np.float32)) for n in sizes]
    for t in range(1, 5):
        for g in gs:
            g.copy_(torch.from_numpy((rng.standard_normal(g.numel()) * 10.0 ** rng.uniform(-6, 0, g.numel())).astype(np.float32)))
        before = [_np(p) for p in ps]
        opt.step()
        ms, vs = opt.read_states()
        torch.cuda.synchronize()
        for k, (n, h) in enumerate(zip(sizes, host)):
            m0, v0 = A.decode(h["mc"], h["ms"], "m"), A.decode(h["vc"], h["vs"], "v")
            _, m, v = A.step(before[k], _np(gs[k]), m0, v0, t, lr, betas, eps, 0.1, 0.75, np.float32)
            _check_step(before[k], _np(gs[k]), m0, v0, _np(ps[k]), None, None, t, lr, betas, eps, float(np.float32(0.1)), 0.75, pt is BF)
            um, uv = A.random_bits(seed, t, k, n)
            h["mc"], h["ms"] = A.encode(m, um, "m")
            h["vc"], h["vs"] = A.encode(v, uv, "v")
            for name, t_ in (("mc", opt.exp_avg), ("vc", opt.exp_avg_sq), ("ms", opt.exp_avg_scale), ("vs", opt.exp_avg_sq_scale)):
                got = t_[k].cpu().numpy()
                assert np.array_equal(got, h[name]), (t, k, name, np.flatnonzero(got != h[name])[:5])
            assert np.array_equal(_np(ms[k]), A.decode(h["mc"], h["ms"], "m")), (t, k)
            assert np.array_equal(_np(vs[k]), A.decode(h["vc"], h["vs"], "v")), (t, k)


def test_8_bit_blocks_of_zeros_of_tiny_values_and_with_a_nan():
    n = 256 * 5
    g = torch.zeros(n, device="cuda")
    g[256:512] = 1e-38                       # a block below 2^-100
    g[512] = float("nan")
    g[768:1024] = 1.0
    g[768] = 1e-4                            # v 10^8 below its block's largest stays above zero
    g[1024] = float("inf")
    p = torch.ones(n, device="cuda")
    opt = bs.AdamW([p], [g], bits=8, weight_decay=0.0)
    opt.step()
    (m,), (v,) = opt.read_states()
    assert torch.all(m[:512] == 0) and torch.all(v[:512] == 0) and torch.all(torch.isfinite(p[:512]))
    assert torch.all(torch.isnan(m[512:768])) and torch.all(torch.isnan(v[512:768]))
    assert torch.isnan(p[512]) and torch.all(torch.isfinite(p[513:1024]))
    assert torch.all(torch.isfinite(m[768:1024])) and torch.all(v[768:1024] > 0)
    assert torch.all(~torch.isfinite(m[1024:]))


@pytest.mark.parametrize("pt,gt,master", [(F32, F32, False), (BF, BF, False), (BF, F32, True), (F32, BF, False)])
def test_8_bit_codes_of_blocks_of_every_magnitude(pt, gt, master):
    # blocks from 1e-14 to 1e14 (m above 28672 and v above 1e9 among them), a third of each zero and a
    # few elements far below their block's largest
    n, betas, seed = 256 * 70 + 100, (0.9, 0.999), 7
    rng = np.random.default_rng(17)
    p, g = _tensor(n, pt, rng, 1.0), _tensor(n, gt, rng, 1.0)
    mc, vc, ms, vs = np.zeros(n, np.uint8), np.zeros(n, np.uint8), np.zeros(-(-n // 256), np.float32), np.zeros(-(-n // 256), np.float32)
    opt = bs.AdamW([p], [g], lr=1e-3, betas=betas, bits=8, seed=seed, masters=[p.float()] if master else None)
    for t in range(1, 4):
        x = rng.standard_normal(n) * np.repeat(10.0 ** rng.uniform(-14, 14, ms.size), 256)[:n]
        x = np.where(rng.random(n) < 0.01, x * 1e-5, x) * (rng.random(n) > 1 / 3)
        g.copy_(torch.from_numpy(x.astype(np.float32)))
        opt.step()
        torch.cuda.synchronize()
        m0, v0 = A.decode(mc, ms, "m"), A.decode(vc, vs, "v")
        _, m, v = A.step(np.zeros(n, np.float32), _np(g), m0, v0, t, 0.0, betas, 1e-8, 0.0, 1.0, np.float32)
        um, uv = A.random_bits(seed, t, 0, n)
        mc, ms = A.encode(m, um, "m")
        vc, vs = A.encode(v, uv, "v")
        for name, got, want in (("mc", opt.exp_avg, mc), ("vc", opt.exp_avg_sq, vc), ("ms", opt.exp_avg_scale, ms), ("vs", opt.exp_avg_sq_scale, vs)):
            got = got[0].cpu().numpy()
            assert np.array_equal(got, want), (t, name, np.flatnonzero(got != want)[:5])


def test_v_in_8_bits_follows_its_mean():
    # with rounding to nearest, v would stop far below the mean square of the gradients
    n, steps = 1 << 14, 3000
    rng = np.random.default_rng(3)
    g = _tensor(n, F32, rng, 1.0)
    p = torch.zeros(n, device="cuda")
    opt = bs.AdamW([p], [g], bits=8, lr=0.0)
    gen = torch.Generator("cuda").manual_seed(1)
    for _ in range(steps):
        g.normal_(generator=gen)
        opt.step()
    mean = float(opt.read_states()[1][0].mean())
    # E v = 1 - 0.999^3000 = 0.9503. Spread of the mean over n elements: each v has a variance below
    # (0.001 / 2) * 2 from the gradients and below 1/16 from the rounding (spacing / 2): 0.0025 at 16384
    assert abs(mean - 0.9503) < 6 * 0.0025, mean


@pytest.mark.parametrize("sizes,gt", [([1], F32), ([100003, 7, 0, 256], F32), ([513] * 900, BF), ([1 << 22], BF)])
@pytest.mark.parametrize("max_norm", [1e-3, 1e9, float("inf")])
def test_norm_and_clip(sizes, gt, max_norm):
    rng = np.random.default_rng(2)
    gs = [_tensor(n, gt, rng, 0.01, 1) for n in sizes]
    ps = [torch.zeros(n, device="cuda") for n in sizes]
    opt = bs.AdamW(ps, gs)
    got = float(opt.grad_norm(max_norm))
    want = np.sqrt(sum(np.sum(_np(g).astype(np.float64) ** 2) for g in gs))
    # 64 squares are added in FP32 before they go on in 64 bits: at most 65 roundings of the sum
    # of squares, half of that of its root, and the result's own rounding
    assert abs(got - want) <= (65 / 2 + 1) * U * want
    assert abs(float(opt.clip) - min(1.0, max_norm / (got + 1e-6))) <= 4 * U * min(1.0, max_norm / got) + (65 / 2) * U
    first = got
    assert all(float(opt.grad_norm(max_norm)) == first for _ in range(5))  # a fixed order


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 3e38])
def test_a_norm_that_is_not_finite_leaves_the_step_out(bad):
    rng = np.random.default_rng(4)
    ps = [_tensor(n, BF, rng, 1.0) for n in (1000, 5)]
    gs = [_tensor(n, F32, rng, 1.0) for n in (1000, 5)]
    opt = bs.AdamW(ps, gs, bits=8)
    opt.step(max_norm=1.0)
    keep = [t.clone() for t in ps + opt.exp_avg + opt.exp_avg_sq + opt.exp_avg_scale + opt.exp_avg_sq_scale]
    gs[1][3] = bad
    opt.step(max_norm=1.0)
    assert int(opt.steps) == 1
    assert all(torch.equal(a, b) for a, b in zip(keep, ps + opt.exp_avg + opt.exp_avg_sq + opt.exp_avg_scale + opt.exp_avg_sq_scale))
    gs[1][3] = 0.5
    opt.step(max_norm=1.0)
    assert int(opt.steps) == 2 and not torch.equal(keep[0], ps[0])


@pytest.mark.parametrize("bits", [8, 32])
def test_a_captured_step_is_the_eager_one(bits):
    def make():
        rng = np.random.default_rng(8)
        ps = [_tensor(n, BF, rng, 0.02) for n in (5000, 257)]
        gs = [_tensor(n, BF, rng, 0.01) for n in (5000, 257)]
        return bs.AdamW(ps, gs, bits=bits, masters=[p.float() for p in ps], seed=3)
    a, b = make(), make()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            b.step(max_norm=0.5)
    torch.cuda.synchronize()
    assert int(b.steps) == 0
    for t in range(6):
        a.lr = b.lr = 1e-3 / (t + 1)
        a.step(max_norm=0.5)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(a.params + a.masters + a.exp_avg + a.exp_avg_sq, b.params + b.masters + b.exp_avg + b.exp_avg_sq):
            assert torch.equal(x, y), t
    assert int(b.steps) == 6


def test_only_the_tensors_are_written():
    buf = {k: torch.full((4096,), 7, dtype=dt, device="cuda") for k, dt in (("p", BF), ("m", torch.uint8), ("v", torch.uint8), ("g", BF))}
    cut = lambda k: [buf[k][16:16 + 259], buf[k][1024:1024 + 1000]]  # noqa: E731
    for k in "mv":
        for t in cut(k):
            t.zero_()
    scales = lambda: [torch.zeros(2, device="cuda"), torch.zeros(4, device="cuda")]  # noqa: E731
    opt = bs.AdamW(cut("p"), cut("g"), bits=8, states=((cut("m"), scales()), (cut("v"), scales())))
    opt.step(max_norm=1.0)
    torch.cuda.synchronize()
    inside = torch.zeros(4096, dtype=torch.bool, device="cuda")
    inside[16:16 + 259] = True
    inside[1024:2024] = True
    for k in "pmv":
        assert torch.all(buf[k][~inside] == 7), k
        # the step on p is below 0.002, half the spacing of BF16 at 7 is 0.0156: p is written as 7 again
        assert torch.all((buf[k][inside] == 7) if k == "p" else (buf[k][inside] != 7)), k
    assert torch.all(buf["g"] == 7)


def test_overlapping_buffers_and_wrong_sizes_are_refused():
    p, g = torch.zeros(100, device="cuda"), torch.zeros(100, device="cuda")
    z = lambda: torch.zeros(100, device="cuda")  # noqa: E731
    for kw in (dict(params=[p, p], grads=[g, g]), dict(params=[p, p[50:]], grads=[g, g[50:]]), dict(params=[p], grads=[p]),
               dict(params=[p], grads=[g], states=([p], [z()])), dict(params=[p], grads=[g], masters=[g]),
               dict(params=[p], grads=[g[:99]]), dict(params=[p], grads=[g, g]), dict(params=[p], grads=[g.half()]),
               dict(params=[p], grads=[g.cpu()]), dict(params=[p.view(10, 10).t()], grads=[g]), dict(params=[], grads=[]),
               dict(params=[p], grads=[g], bits=16), dict(params=[p], grads=[g], weight_decay=[0.1, 0.2])):
        with pytest.raises(bs.BsError) as e:
            bs.AdamW(**kw)
        assert e.value.code == bs.E_ARG
    shared = bs.AdamW([p, z()], [g, g])  # two tensors may read one gradient
    shared.step()
    for kw in (dict(betas=(1.0, 0.9)), dict(betas=(0.9, -0.1)), dict(eps=-1.0), dict(weight_decay=-1.0), dict(weight_decay=float("nan"))):
        with pytest.raises(bs.BsError) as e:
            bs.AdamW([z()], [g], **kw).step()
        assert e.value.code == bs.E_ARG


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("sizes", [(5000, 257, 3), (300,) * 300])
def test_a_step_into_a_twin_is_the_step_in_place(bits, sizes):
    def make():
        rng = np.random.default_rng(8)
        ps = [_tensor(n, BF, rng, 0.02) for n in sizes]
        return bs.AdamW(ps, [_tensor(n, BF, rng, 0.01) for n in sizes], bits=bits, masters=[p.float() for p in ps], seed=3)
    held = lambda o: [t.clone() for ts in (o.params, o.masters, o.exp_avg, o.exp_avg_sq, o.exp_avg_scale or [], o.exp_avg_sq_scale or [])  # noqa: E731
                      for t in ts]
    a, b = make(), make()
    there, here = b, b.twin()
    for t in range(4):
        a.step(max_norm=0.5)
        before = held(there)
        for _ in range(2):  # its results do not depend on what stands in the twin
            there.step(max_norm=0.5, into=here, number=t + 1)
        assert all(torch.equal(x, y) for x, y in zip(before, held(there)))
        assert all(torch.equal(x, y) for x, y in zip(held(a), held(here))), t
        assert int(b.steps) == int(a.steps) == t + 1
        there, here = here, there
    with pytest.raises(bs.BsError) as e:
        a.step(into=b)
    assert e.value.code == bs.E_ARG
