"""bs_lora_plan, bs_lora_forward and bs_lora_backward on the GPU against numpy in 64 bits.

Most cases have small whole numbers and power-of-two scales: every product and partial sum is then
below 2^24 and exact in FP32, so outputs have to be equal, whatever the order of a sum (BF16 outputs
to the result rounded once). The other cases have normally distributed inputs. There a sum of K
products that are exact in FP32 is off by at most 4 K 2^-24 of the sum of their magnitudes (each
addition rounds, towards zero inside the tensor cores, 2^-23 at most, and not more than two follow
one product), which is what the framework's other products are held to; a second sum takes the first
one's error on, and its own; an output adds its rounding.
"""
import numpy as np
import pytest
import torch

import lora_plain as L

pytestmark = pytest.mark.gpu

bs = pytest.importorskip("lossless_entropy_coding_interleaved_b200")
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def _idx(rng, tokens, n, route, none=0.1):
    if route == "one":
        return np.full(tokens, n - 1, np.int32)
    if route == "none":
        return np.full(tokens, -1, np.int32)
    idx = rng.integers(0, n, tokens).astype(np.int32)
    idx[rng.random(tokens) < none] = -1
    return np.sort(idx)[::-1].copy() if route == "runs" else idx


class Case:
    """One set of adapters over projections (rows, cols), a batch, and the same in numpy."""

    def __init__(self, seed, tokens, n, r, projs, route="mixed", ranks=None, whole=True, x_pad=0):
        self.rng = rng = np.random.default_rng(seed)
        self.T, self.n, self.r, self.projs, self.whole = tokens, n, r, projs, whole
        self.ranks = np.full(n, r, np.int32) if ranks is None else np.resize(np.asarray(ranks, np.int32), n)
        self.idx = _idx(rng, tokens, n, route)
        self.scales = (2.0 ** rng.integers(-1, 2, n) if whole else rng.uniform(0.5, 2, n)).astype(np.float32)
        self.a, self.b, self.x = [], [], []
        for rows, cols in projs:
            a = self.draw((n, r, cols), 1 if whole else cols ** -0.5)
            b = self.draw((n, rows, r), 1 if whole else r ** -0.5)
            for i in range(n):  # what is past a rank is not read
                a[i, self.ranks[i]:] = np.nan
                b[i, :, self.ranks[i]:] = np.nan
            self.a.append(a)
            self.b.append(b)
        shared = self.draw((tokens, projs[0][1]), 2 if whole else 1.0)
        self.x = [shared if c == projs[0][1] else self.draw((tokens, c), 2 if whole else 1.0) for _, c in projs]
        self.dx_shared = len({c for _, c in projs}) == 1
        dev = lambda v: torch.from_numpy(v).to(BF).cuda()  # noqa: E731
        self.set = bs.LoraAdapters([dev(v) for v in self.a], [dev(v) for v in self.b], torch.from_numpy(self.scales).cuda(),
                                   None if ranks is None else torch.from_numpy(self.ranks).cuda())
        self.xd = [self.place(v, BF, x_pad) for v in self.x]
        self.plan = bs.LoraPlan(tokens, n).update(torch.from_numpy(self.idx).cuda())

    def draw(self, shape, scale):
        """Whole numbers up to `scale`, or normal values that BF16 holds."""
        if self.whole:
            return self.rng.integers(-scale, scale + 1, shape).astype(np.float32)
        return torch.from_numpy((self.rng.standard_normal(shape) * scale).astype(np.float32)).to(BF).float().numpy()

    def place(self, v, dt, pad=0):
        """On the device, `pad` more elements between the rows, NaN in them."""
        t = torch.full((v.shape[0], v.shape[1] + pad), float("nan"), dtype=dt, device="cuda")
        t[:, :v.shape[1]] = torch.from_numpy(v).to(dt)
        return t[:, :v.shape[1]]

    def f64(self, k):
        return [v.astype(np.float64) for v in (self.x[k], self.a[k], self.b[k])]

    def abs64(self, k):
        return [np.nan_to_num(np.abs(v)).astype(np.float64) for v in (self.x[k], self.a[k], self.b[k])]


def _equal(got, want, dt, what):
    got = got.detach().float().cpu().numpy()
    want = torch.from_numpy(want).float().to(dt).float().numpy()
    bad = np.argwhere(got != want)
    assert bad.size == 0, (what, len(bad), bad[:3].tolist(), [(float(got[tuple(i)]), float(want[tuple(i)])) for i in bad[:3]])


def _near(got, want, tol, dt, what):
    got = got.detach().double().cpu().numpy()
    tol = tol + np.abs(want) * U * 2 + 1e-30
    if dt is BF:
        tol = tol + (np.abs(want) + tol) * 2.0 ** -8
    bad = np.argwhere(~(np.abs(got - want) <= tol))
    assert bad.size == 0, (what, len(bad), bad[:3].tolist())


def check_forward(c, dt, in_place=False, y_pad=0, base=True):
    base_np = [c.draw((c.T, rows), 3 if c.whole else 1.0) if base else np.zeros((c.T, rows), np.float32) for rows, _ in c.projs]
    based = [c.place(v, dt, y_pad) for v in base_np]
    ys = based if in_place else [c.place(np.full_like(v, np.nan), dt, 8 - y_pad if y_pad else 0) for v in base_np]
    state = c.set.state(c.T)
    c.set.forward(c.plan, c.xd, ys, bases=None if in_place else based if base else [None] * len(ys), state=state)
    torch.cuda.synchronize()
    assert int(c.plan.err) & 2 == 0  # no wait ran out
    for k in range(len(c.projs)):
        x, a, b = c.f64(k)
        want, h = L.forward(x, c.idx, a, b, c.scales, c.ranks, base_np[k].astype(np.float64))
        if c.whole:
            assert np.abs(want).max(initial=0) < 2 ** 24 and np.abs(h).max(initial=0) < 2 ** 22
            _equal(ys[k], want, dt, k)
        else:
            xa, aa, ba = c.abs64(k)
            mag, _ = L.forward(xa, c.idx, aa, ba, c.scales, c.ranks, np.abs(base_np[k]).astype(np.float64))
            _near(ys[k], want, 4 * U * (x.shape[1] + 3 * c.r) * mag, dt, k)
        if y_pad and not in_place:  # nothing between the rows was written
            whole = ys[k].as_strided((c.T, ys[k].stride(0)), (ys[k].stride(0), 1))
            assert c.T == 0 or torch.all(torch.isnan(whole[:, ys[k].shape[1]:]))
    return state


def check_backward(c, dt, state, dx=True, base=True, accumulate=False):
    n = len(c.projs)
    dys = [c.draw((c.T, rows), 1 if c.whole else 0.1) for rows, _ in c.projs]
    dyd = [c.place(v, BF) for v in dys]
    start = 5.0 if accumulate else float("nan")
    das = [torch.full(v.shape, start, device="cuda") for v in c.a]
    dbs = [torch.full(v.shape, start, device="cuda") for v in c.b]
    dxb = [c.draw(x.shape, 3 if c.whole else 1.0) if base else np.zeros_like(x) for x in c.x]
    dxd, dxs = [c.place(v, dt) for v in dxb], [c.place(np.full_like(v, np.nan), dt) for v in dxb]
    if c.dx_shared:
        dxb, dxd, dxs = [dxb[0]] * n, [dxd[0]] * n, [dxs[0]] * n
    c.set.backward(c.plan, c.xd, dyd, state, das, dbs, dxs=dxs if dx else None, dx_bases=dxd if base and dx else None,
                   accumulate=accumulate)
    torch.cuda.synchronize()
    assert int(c.plan.err) & 2 == 0
    want_dx = [v.astype(np.float64) for v in dxb]
    tol_dx = [np.abs(v).astype(np.float64) * 4 * U for v in dxb]
    for k in range(n):
        x, a, b = c.f64(k)
        dy = dys[k].astype(np.float64)
        p, da, db = L.backward(x, dy, c.idx, a, b, c.scales, c.ranks, np.zeros_like(x))
        at = 0 if c.dx_shared else k
        want_dx[at] += p
        if accumulate:
            for i in range(c.n):
                if np.any(c.idx == i):
                    da[i] += 5
                    db[i] += 5
                else:
                    da[i] = db[i] = 5
        if c.whole:
            assert max(np.abs(v).max(initial=0) for v in (p, da, db)) < 2 ** 24
            _equal(das[k], da, F32, ("da", k))
            _equal(dbs[k], db, F32, ("db", k))
        else:
            xa, aa, ba = c.abs64(k)
            px, ma, mb = L.backward(xa, np.abs(dy), c.idx, aa, ba, c.scales, c.ranks, np.zeros_like(x))
            rows, cols = c.projs[k]
            tol_dx[at] += 4 * U * (rows + 3 * c.r) * px
            _near(das[k], da, 4 * U * (rows + 3 * c.T) * ma, F32, ("da", k))
            _near(dbs[k], db, 4 * U * (cols + 3 * c.T) * mb, F32, ("db", k))
    if dx:
        for k in range(1 if c.dx_shared else n):
            (_equal if c.whole else lambda g, w, d, s: _near(g, w, tol_dx[k], d, s))(dxs[k], want_dx[k], dt, ("dx", k))


SIZES = [  # tokens, adapters, rank_max, projections, route, ranks
    (1, 1, 8, [(8, 8)], "one", None),
    (1, 3, 16, [(256, 512), (128, 512), (128, 512)], "mixed", [3, 16, 1]),
    (7, 2, 64, [(136, 1032)], "mixed", [64, 33]),
    (8, 8, 24, [(264, 264)], "mixed", [1, 7, 8, 9, 17, 24, 0, 23]),
    (37, 24, 32, [(520, 768), (520, 768)], "mixed", [31, 5, 32]),
    (129, 4, 8, [(128, 64)], "runs", None),
    (128, 1, 128, [(256, 128)], "one", None),
    (257, 3, 40, [(72, 200)], "mixed", [40, 12, 1]),
    (300, 200, 16, [(64, 128)], "mixed", [16, 3]),
    (333, 5, 72, [(392, 328), (200, 328)], "runs", [72, 70, 65, 2]),
    (1025, 7, 128, [(136, 144)], "mixed", [128, 127, 64, 65, 3]),
    (64, 5, 16, [(4096, 3584)], "none", None),
    (200, 6, 16, [(136, 2056)], "one", None),
    # many blocks a CTA, the last tiles without an adapter (a run of blocks with nothing to multiply)
    (700, 2, 16, [(14336, 64)], "runs", None),
    (400, 3, 128, [(8200, 72)], "runs", [100, 0, 128]),
    (257, 2, 16, [(64, 8200), (72, 8200), (80, 8200), (64, 8200), (72, 8200)], "runs", None),
]


@pytest.mark.parametrize("tokens,n,r,projs,route,ranks", SIZES)
@pytest.mark.parametrize("dt", [F32, BF])
def test_whole_numbers(tokens, n, r, projs, route, ranks, dt):
    c = Case(1, tokens, n, r, projs, route, ranks)
    state = check_forward(c, dt)
    check_backward(c, dt, state)
    check_forward(c, dt, in_place=True)
    check_forward(c, dt, base=False)
    check_backward(c, dt, state, base=False, accumulate=True)
    check_backward(c, dt, state, dx=False)


@pytest.mark.parametrize("tokens,n,r,projs,route,ranks", [
    (5, 3, 16, [(512, 3584), (256, 3584)], "mixed", [16, 9]), (100, 4, 64, [(776, 1160)], "mixed", [64, 50, 3]),
    (700, 3, 32, [(1288, 648)], "runs", None), (513, 2, 128, [(264, 5120)], "mixed", [128, 100])])
@pytest.mark.parametrize("dt", [F32, BF])
def test_normal_values(tokens, n, r, projs, route, ranks, dt):
    c = Case(2, tokens, n, r, projs, route, ranks, whole=False)
    check_backward(c, dt, check_forward(c, dt))


@pytest.mark.parametrize("tokens", [3, 65, 300])
def test_strided_rows(tokens):
    c = Case(3, tokens, 3, 16, [(72, 136)], "mixed", [16, 5, 11], x_pad=24)
    for dt in (F32, BF):
        check_backward(c, dt, check_forward(c, dt, y_pad=4 if dt is F32 else 0))
        check_forward(c, dt, in_place=True, y_pad=8)


def test_outputs_of_one_buffer():
    # q, k and v as columns of one buffer, as a fused projection leaves them
    c = Case(4, 50, 4, 16, [(64, 256), (32, 256), (32, 256)])
    buf = torch.zeros(50, 128, device="cuda")
    ys = [buf[:, :64], buf[:, 64:96], buf[:, 96:]]
    c.set.forward(c.plan, c.xd, ys)
    for k in range(3):
        x, a, b = c.f64(k)
        _equal(ys[k], L.forward(x, c.idx, a, b, c.scales, c.ranks, np.zeros((50, c.projs[k][0])))[0], F32, k)


@pytest.mark.parametrize("tokens,n", [(0, 3), (1, 1), (31, 2), (1000, 8192), (5000, 1), (70001, 37), (1024, 8), (1025, 8)])
def test_plan_groups_in_order(tokens, n):
    rng = np.random.default_rng(tokens)
    idx = rng.integers(-3, n, tokens).astype(np.int32)
    plan = bs.LoraPlan(tokens, n).update(torch.from_numpy(idx).cuda())
    w = plan.data.cpu().numpy().view(np.uint32)
    up4 = lambda v: (v + 3) // 4 * 4  # noqa: E731
    begin = w[16:16 + n + 2]
    bucket = np.where(idx < 0, n, idx)
    assert np.array_equal(begin, np.concatenate([[0], np.cumsum(np.bincount(bucket, minlength=n + 1))]))
    at = 16 + up4(n + 2)
    rows, count = w[at:at + 4 * n].reshape(n, 4), np.bincount(bucket, minlength=n + 1)[:n]
    order = rows[:, 0]
    assert np.array_equal(rows[:, 1], begin[order]) and np.array_equal(rows[:, 2], begin[order + 1]) and not rows[:, 3].any()
    assert np.array_equal(np.sort(order), np.arange(n))  # every adapter once, the ones with most tokens first:
    assert np.all(count[order][1:] * 8 <= count[order][:-1] * 9 + 8)  # none after one an eighth smaller
    at += 4 * n
    assert np.array_equal(w[at:at + tokens], np.argsort(bucket, kind="stable"))
    assert int(plan.err) == 0
    for size, count, start in ((128, w[:2], at + up4(tokens)), (8, w[2:4], at + up4(tokens) + 4 * min(tokens, tokens // 128 + n + 1))):
        want = [(a, f, min(size, int(begin[a + 1]) - f), 0) for a in range(n + 1) for f in range(int(begin[a]), int(begin[a + 1]), size)]
        if size == 8 and tokens > 1024:
            assert count[0] == count[1] == 0
            continue
        assert count[1] == len(want) and count[0] == sum(t[0] < n for t in want)
        words = 4 if size == 128 else 12
        got = w[start:start + words * len(want)].reshape(-1, words)
        assert np.array_equal(got[:, :4], np.array(want, np.uint32).reshape(-1, 4))
        if size == 8:  # the tokens themselves follow, -1 behind the last
            perm = np.concatenate([np.argsort(bucket, kind="stable"), np.zeros(8, np.int64)])
            for row, (_, f, c, _) in zip(got, want):
                assert np.array_equal(row[4:4 + c], perm[f:f + c]) and np.all(row[4 + c:] == 0xFFFFFFFF)


def test_an_index_past_the_adapters_counts_as_none_and_is_reported():
    c = Case(5, 20, 3, 8, [(64, 64)])
    idx = torch.from_numpy(np.where(c.idx == 1, 3, c.idx)).cuda()
    c.plan.update(idx)
    c.idx = np.where(c.idx == 1, -1, c.idx)
    check_forward(c, F32)
    assert int(c.plan.err) == 4


@pytest.mark.parametrize("tokens", [60, 200])
def test_a_plan_of_another_batch_is_refused_on_the_device(tokens):
    c = Case(14, tokens, 3, 16, [(64, 128)])
    other = bs.LoraPlan(tokens + 1, 3)
    state, y, das, dbs = c.set.state(tokens), torch.full((tokens, 64), 3.0, device="cuda"), torch.full((3, 16, 128), 3.0, device="cuda"), \
        torch.full((3, 64, 16), 3.0, device="cuda")
    items, _ = c.set._begin(c.plan, (), state)
    dx, dy = torch.full((tokens, 128), 3.0, device="cuda"), torch.zeros(tokens, 64, dtype=BF, device="cuda")
    it = items[0]
    it.d_a, it.d_b, it.rows, it.cols = c.set._fixed[0]
    it.d_x, it.x_stride, it.d_h, it.d_y, it.y_stride = c.xd[0].data_ptr(), 128, state[0].data_ptr(), y.data_ptr(), 64
    it.d_dy, it.dy_stride, it.d_g, it.d_dx, it.dx_stride = dy.data_ptr(), 64, c.set.state(tokens)[0].data_ptr(), dx.data_ptr(), 128
    it.d_da, it.d_db = das.data_ptr(), dbs.data_ptr()
    import ctypes
    batch = bs.LoraBatch(tokens, 3, 16, 0, None, c.set._scales_at, other.data.data_ptr(), other.data.numel(), other.err.data_ptr())
    st = torch.cuda.current_stream().cuda_stream
    assert bs.lib.bs_lora_forward(1, items, ctypes.byref(batch), st) == bs.OK
    assert int(other.err) == 8
    other.err.zero_()
    assert bs.lib.bs_lora_backward(1, items, ctypes.byref(batch), 0, st) == bs.OK
    assert int(other.err) == 8
    for t in (y, dx, das, dbs):
        assert torch.all(t == 3)


def test_a_new_plan_gives_no_token_an_adapter():
    c = Case(15, 150, 3, 16, [(64, 128)])
    plan = bs.LoraPlan(150, 3)
    y = torch.full((150, 64), 3.0, device="cuda")
    c.set.forward(plan, c.xd, [y])
    das, dbs = [torch.full((3, 16, 128), 3.0, device="cuda")], [torch.full((3, 64, 16), 3.0, device="cuda")]
    c.set.backward(plan, c.xd, [torch.ones(150, 64, dtype=BF, device="cuda")], c.set.state(150), das, dbs)
    assert torch.all(y == 3) and not das[0].any() and not dbs[0].any() and int(plan.err) == 0


def test_tokens_without_an_adapter_are_left_as_they_are():
    # NaN payloads in base survive, and NaN and infinities in x of such tokens reach nothing
    c = Case(6, 40, 3, 16, [(64, 128)])
    off = torch.from_numpy(c.idx < 0).cuda()
    assert off.any() and not off.all()
    c.xd[0][off] = float("nan")
    y = torch.full((40, 64), float("nan"), device="cuda")
    y.view(torch.int32)[:] = 0x7FC12345
    keep = y.clone()
    c.set.forward(c.plan, c.xd, [y])
    assert torch.equal(y.view(torch.int32)[off], keep.view(torch.int32)[off])
    y.zero_()
    c.set.forward(c.plan, c.xd, [y])
    assert torch.all(torch.isfinite(y))


def test_infinities_stay_infinities():
    x = torch.zeros(2, 64, dtype=BF, device="cuda")
    x[0, 3] = float("inf")
    x[1, 4] = 1
    a = torch.ones(1, 8, 64, dtype=BF, device="cuda")
    b = torch.ones(1, 16, 8, dtype=BF, device="cuda")
    s = bs.LoraAdapters([a], [b])
    y = torch.zeros(2, 16, device="cuda")
    s.forward(bs.LoraPlan(2, 1).update(torch.zeros(2, dtype=torch.int32, device="cuda")), [x], [y])
    assert torch.all(y[0] == float("inf")) and torch.all(y[1] == 8)


def test_gradients_against_differences():
    # f(A, B, x) = sum w y: its derivative along a direction against central differences in 64 bits
    c = Case(7, 30, 3, 16, [(72, 80)], "mixed", [16, 5, 9], whole=False)
    state = c.set.state(c.T)
    c.set.forward(c.plan, c.xd, None, state=state)
    w = c.draw((c.T, 72), 1.0)
    das, dbs = [torch.empty(3, 16, 80, device="cuda")], [torch.empty(3, 72, 16, device="cuda")]
    dx = torch.empty(c.T, 80, device="cuda")
    c.set.backward(c.plan, c.xd, [c.place(w, BF)], state, das, dbs, dxs=[dx])
    x, a, b = [np.nan_to_num(v) for v in c.f64(0)]
    rng = np.random.default_rng(0)
    f = lambda x, a, b: np.sum(w * L.forward(x, c.idx, a, b, c.scales, c.ranks, np.zeros((c.T, 72)))[0])  # noqa: E731
    for which, grad in ((0, dx), (1, das[0]), (2, dbs[0])):
        args = [x, a, b]
        d = rng.standard_normal(args[which].shape)
        plus, minus = list(args), list(args)
        plus[which], minus[which] = args[which] + 1e-4 * d, args[which] - 1e-4 * d
        diff = (f(*plus) - f(*minus)) / 2e-4  # f is linear in each of them: exact but for 64-bit rounding
        got = float(np.sum(grad.double().cpu().numpy() * d))
        assert abs(got - diff) <= 1e-4 * np.sqrt(np.sum(grad.double().cpu().numpy() ** 2)) , which


def test_same_bits_again_and_captured():
    c = Case(8, 300, 4, 32, [(264, 520), (136, 520)], whole=False)
    base = [torch.randn(300, r, device="cuda") for r, _ in c.projs]
    dys = [torch.randn(300, r, device="cuda").to(BF) for r, _ in c.projs]
    idx = torch.from_numpy(c.idx).cuda()
    outs = lambda: dict(ys=[torch.empty_like(t) for t in base], das=[torch.empty(v.shape, device="cuda") for v in c.a],  # noqa: E731
                        dbs=[torch.empty(v.shape, device="cuda") for v in c.b], dx=torch.empty(300, 520, device="cuda"),
                        state=c.set.state(300), work=c.set.state(300))

    def go(o):
        c.plan.update(idx)
        c.set.forward(c.plan, c.xd, o["ys"], bases=base, state=o["state"])
        c.set.backward(c.plan, c.xd, dys, o["state"], o["das"], o["dbs"], dxs=[o["dx"]] * 2, work=o["work"])
    a, b, g = outs(), outs(), outs()
    go(a)
    go(b)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        go(g)
    same = lambda p, q: all(torch.equal(u, v) for key in ("ys", "das", "dbs") for u, v in zip(p[key], q[key])) and torch.equal(p["dx"], q["dx"])  # noqa: E731
    torch.cuda.synchronize()
    assert same(a, b)
    for t in g["ys"] + g["das"] + g["dbs"] + [g["dx"]]:
        t.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    assert same(a, g)
    idx.copy_(torch.from_numpy(c.idx[::-1].copy()))  # another routing under the same graph
    graph.replay()
    go(b)
    torch.cuda.synchronize()
    assert same(b, g) and not same(a, g)


def test_on_another_stream():
    c = Case(9, 100, 4, 16, [(264, 520)])
    s = torch.cuda.Stream()
    y = torch.zeros(100, 264, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    c.set.forward(c.plan, c.xd, [y], stream=s)
    s.synchronize()
    x, a, b = c.f64(0)
    _equal(y, L.forward(x, c.idx, a, b, c.scales, c.ranks, np.zeros((100, 264)))[0], F32, 0)


@pytest.mark.parametrize("raw", [False, True])
def test_a_state_of_a_call_on_another_stream_is_not_given_away_before_it_has_run(raw):
    c = Case(31, 300, 2, 16, [(264, 520)])  # the tiled kernels: h goes through the state
    s, x = torch.cuda.Stream(), torch.randn(4096, 4096, device="cuda")
    y, y2 = (torch.zeros(300, 264, device="cuda") for _ in range(2))
    size = c.set.state(300)[0].numel()
    s.wait_stream(torch.cuda.current_stream())
    taken = []
    with torch.cuda.stream(s):
        for _ in range(20):
            x = x @ x * 1e-3
    for out in (y, y2):
        c.set.forward(c.plan, c.xd, [out], stream=s.cuda_stream if raw else s)
        taken += [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
        with torch.cuda.stream(s):
            x = x @ x * 1e-3
    torch.cuda.synchronize()
    xs, a, b = c.f64(0)
    want = L.forward(xs, c.idx, a, b, c.scales, c.ranks, np.zeros((300, 264)))[0]
    _equal(y, want, F32, 0)
    _equal(y2, want, F32, 0)
    assert all(bool((t == 255).all()) for t in taken)  # nor is memory written that others have


def test_more_projections_than_one_launch_holds():
    c = Case(10, 9, 2, 8, [(16, 64)] * 21)
    check_forward(c, F32)
    c.dx_shared = False
    check_backward(c, F32, check_forward(c, F32), dx=False)


def test_empty_batch():
    c = Case(11, 0, 2, 8, [(16, 64)])
    check_backward(c, F32, check_forward(c, F32), dx=False)
    das, dbs = [torch.full((2, 8, 64), 3.0, device="cuda")], [torch.full((2, 16, 8), 3.0, device="cuda")]
    c.set.backward(c.plan, c.xd, [torch.zeros(0, 16, dtype=BF, device="cuda")], c.set.state(0), das, dbs, accumulate=True)
    assert torch.all(das[0] == 3) and torch.all(dbs[0] == 3)


@pytest.mark.parametrize("tokens", [1, 3])
def test_rows_that_are_not_contiguous_are_refused(tokens):
    c = Case(5, tokens, 2, 8, [(64, 64)])
    wide = lambda dt: torch.zeros(64, 2 * tokens, dtype=dt, device="cuda")[:, :tokens].t()  # noqa: E731
    x, y = c.xd, [torch.zeros(tokens, 64, device="cuda")]
    das, dbs = [torch.zeros(2, 8, 64, device="cuda")], [torch.zeros(2, 64, 8, device="cuda")]
    state = c.set.state(tokens)
    for call in (lambda: c.set.forward(c.plan, [wide(BF)], y), lambda: c.set.forward(c.plan, x, [wide(F32)]),
                 lambda: c.set.forward(c.plan, x, y, [wide(F32)]), lambda: c.set.backward(c.plan, x, [wide(BF)], state, das, dbs)):
        with pytest.raises(bs.BsError) as e:
            call()
        assert e.value.code == bs.E_ARG


def test_binding_refusals():
    c = Case(12, 10, 2, 8, [(16, 64)])
    y = torch.zeros(10, 16, device="cuda")
    bad = [dict(ys=[y[:9]]), dict(ys=[y.half()]), dict(ys=[y.t().contiguous().t()]), dict(ys=[y, y]), dict(xs=[c.xd[0].float()]),
           dict(xs=[c.xd[0][:, :56]]), dict(state=[torch.zeros(16, dtype=torch.uint8, device="cuda")]),
           dict(bases=[y.to(BF)]), dict(plan=bs.LoraPlan(10, 3)), dict(ys=[y.cpu()])]
    for kw in bad:
        with pytest.raises(bs.BsError) as e:
            c.set.forward(**{**dict(plan=c.plan, xs=c.xd, ys=[y]), **kw})
        assert e.value.code in (bs.E_ARG, bs.E_SIZE)
    two = Case(13, 10, 2, 8, [(16, 64), (16, 64)])
    for kw in (dict(ys=[y, y]), dict(ys=None, state=[two.set.state(10)[0]] * 2)):
        with pytest.raises(bs.BsError):
            two.set.forward(two.plan, two.xd, **kw)
    with pytest.raises(bs.BsError):
        c.plan.update(torch.zeros(9, dtype=torch.int32, device="cuda"))
    with pytest.raises(bs.BsError):
        bs.LoraAdapters([torch.zeros(2, 8, 64, device="cuda")], [torch.zeros(2, 16, 8, dtype=BF, device="cuda")])
