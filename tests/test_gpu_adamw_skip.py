"""Steps that are left out, and what a norm leaves behind for the steps after it.

Everything is compared bit for bit: a step into other buffers with the step in place, and what a step
that is left out leaves with what was there before.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

bs = pytest.importorskip("lossless_entropy_coding_interleaved_b200")
BF, F32 = torch.bfloat16, torch.float32
INF = float("inf")


def _make(sizes, bits, pt, master, offset=0, **kw):
    rng = np.random.default_rng(8)

    def tensor(n, dt, scale):
        t = torch.zeros(n + offset + 8, dtype=dt, device="cuda")[offset:offset + n]
        return t.copy_(torch.from_numpy((rng.standard_normal(n) * scale).astype(np.float32)))
    ps, gs = [tensor(n, pt, 0.02) for n in sizes], [tensor(n, BF, 0.01) for n in sizes]
    kw = dict(lr=1e-2, weight_decay=0.1, seed=3) | kw
    return bs.AdamW(ps, gs, bits=bits, masters=[p.float() for p in ps] if master else None, **kw)


def _held(o):
    return [t for ts in (o.params, o.masters, o.exp_avg, o.exp_avg_sq, o.exp_avg_scale, o.exp_avg_sq_scale) if ts is not None for t in ts]


def _bits(t):
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def _same(a, b):
    return all(torch.equal(_bits(x), _bits(y)) for x, y in zip(a, b))


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("pt,master", [(BF, True), (BF, False), (F32, False)])
@pytest.mark.parametrize("sizes,offset", [((5000, 257, 3, 0, 256), 0), ((4099, 300), 1), ((300,) * 300, 0)])
@pytest.mark.parametrize("bad_at", [1, 3])
def test_a_step_into_a_twin_that_is_left_out_leaves_it_with_the_values_as_they_were(bits, pt, master, sizes, offset, bad_at):
    a, b = _make(sizes, bits, pt, master, offset), _make(sizes, bits, pt, master, offset)
    there, here = b, b.twin()
    for t in range(1, 6):
        for o in (a, b):
            for k, g in enumerate(o.grads):
                g.copy_(torch.from_numpy((np.random.default_rng(100 * t + k).standard_normal(g.numel()) * 0.01).astype(np.float32)))
            if t == bad_at:
                o.grads[1][2] = INF if t == 1 else float("nan")
        for x in _held(here):  # garbage, as in new memory
            _bits(x).fill_(-1 if x.dtype is not torch.uint8 else 255)
        before = [x.clone() for x in _held(there)]
        a.step(max_norm=0.5)
        there.step(max_norm=0.5, into=here)
        assert _same(before, _held(there))
        assert _same(_held(here), before if t == bad_at else _held(a)), t
        assert _same(_held(here), _held(a)), t
        assert int(a.steps) == int(b.steps) == t - (t >= bad_at)
        there, here = here, there


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("captured", [False, True])
def test_a_norm_is_for_one_step(bits, captured):
    # b takes the same steps with every factor given by hand. steps: (max_norm, bad gradient, clip set before)
    steps = [(None, False, None), (0.01, False, None), (None, False, None), (0.01, True, None), (None, False, None), (None, False, 0.25),
             (0.02, False, None), (0.03, True, 2.0), (None, False, None), (None, False, None)]
    a, b = (_make((5000, 257, 3), bits, F32, False, clip=0.5) for _ in range(2))
    own, taken, graphs = 0.5, 0, {}
    for max_norm, bad, clip in steps:
        for o in (a, b):
            for g in o.grads:
                g.copy_(torch.from_numpy((np.random.default_rng(g.numel() + taken).standard_normal(g.numel()) * 0.01).astype(np.float32)))
            if bad:
                o.grads[0][77] = float("nan")
        if clip is not None:
            a.clip = own = clip
        if not captured:
            a.step(max_norm=max_norm)
        else:
            if max_norm not in graphs:
                graphs[max_norm], side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
                torch.cuda.synchronize()
                with torch.cuda.stream(side), torch.cuda.graph(graphs[max_norm], stream=side):
                    a.step(max_norm=max_norm)
            graphs[max_norm].replay()
        torch.cuda.synchronize()
        if not bad:
            norm = np.sqrt(sum(float((g.double() ** 2).sum()) for g in b.grads))
            factor = float(a.clip)
            assert factor == own if max_norm is None else abs(factor * (norm + 1e-6) / max_norm - 1) < 1e-6 and factor < 0.1
            b.clip = factor
            b.step()
            taken += 1
        assert int(a.steps) == int(b.steps) == taken
        assert _same(_held(a), _held(b))


def test_a_norm_taken_by_hand_is_the_next_steps():
    a, b = (_make((300, 5), 32, F32, False) for _ in range(2))
    a.grad_norm(0.01)
    a.grad_norm(0.02)  # the later one counts
    b.clip = float(a.clip)
    a.step()
    b.step()
    assert _same(_held(a), _held(b))
    b.clip = 1.0
    a.step()
    b.step()
    assert _same(_held(a), _held(b)) and float(a.clip) == 1.0
    a.grads[0][1] = INF
    a.grad_norm(0.01)
    before = [t.clone() for t in _held(a)]
    a.step()
    assert _same(before, _held(a)) and int(a.steps) == 2
    a.grads[0][1] = b.grads[0][1]
    a.step()
    b.step()
    assert _same(_held(a), _held(b)) and int(a.steps) == 3
    a.grad_norm(0.01)
    a.clip = 0.125  # set after the norm: replaces its factor
    b.clip = 0.125
    for _ in range(2):
        a.step()
        b.step()
        assert _same(_held(a), _held(b))


def test_a_ctl_without_once_keeps_a_norm_for_every_call_until_the_next():
    # several calls under one norm, as the C interface allows
    a, b = (_make((300, 5), 32, F32, False) for _ in range(2))
    a.ctl[7] = 0
    a.grad_norm(0.01)
    b.clip = float(a.clip)
    for _ in range(2):
        a.step()
        b.step()
    assert _same(_held(a), _held(b)) and float(a.clip) == float(b.clip) < 1
    a.grads[0][1] = INF
    a.grad_norm(0.01)
    for _ in range(2):
        a.step()
    assert _same(_held(a), _held(b)) and int(a.steps) == 2


def test_a_skip_of_the_callers_stays():
    a = _make((300, 5), 32, F32, False)
    before = [t.clone() for t in _held(a)]
    a.ctl[3] = 1
    for _ in range(2):
        a.step()
    assert _same(before, _held(a)) and int(a.steps) == 0
    a.ctl[3] = 0
    a.step()
    assert not _same(before, _held(a)) and int(a.steps) == 1


def test_a_twin_shares_the_norm_and_the_factor():
    a, b = (_make((300, 5), 8, F32, False, clip=0.5) for _ in range(2))
    twin = a.twin()
    a.step(max_norm=0.01, into=twin)
    b.step(max_norm=0.01)
    twin.step(into=a)
    b.step()
    assert _same(_held(a), _held(b)) and float(a.clip) == float(twin.clip) == 0.5


def test_a_step_that_is_refused_takes_no_norm_and_no_other_number():
    a, other = _make((300, 5), 32, F32, False), _make((300, 5), 32, F32, False)
    before = [t.clone() for t in _held(a)] + [a.ctl.clone()]
    for kw in (dict(into=other), dict(number=-1), dict(number=2 ** 31), dict(number=2 ** 32), dict(number=2 ** 32 + 5), dict(number=-2 ** 32 + 5)):
        with pytest.raises(bs.BsError) as e:
            a.step(max_norm=0.01, **kw)
        assert e.value.code == bs.E_ARG
    assert _same(before, _held(a) + [a.ctl])
    a.step(number=2 ** 31 - 1)
    assert int(a.steps) == 2 ** 31 - 1


def test_a_step_keeps_its_number_whatever_other_threads_step(monkeypatch):
    # another thread's step between a call's own preparation and its launch
    a, b = (_make((300, 5), 8, F32, False) for _ in range(2))
    launch, others = bs._on, [9, 0, 7]

    def on(index, what, fn, *args, **kw):
        if others:
            a.step(number=others.pop())
        return launch(index, what, fn, *args, **kw)
    monkeypatch.setattr(bs, "_on", on)
    a.step(number=5)
    monkeypatch.setattr(bs, "_on", launch)
    for number in (9, 0, 7, 5):  # the innermost is launched first
        b.step(number=number)
    assert int(a.steps) == 5 and _same(_held(a), _held(b))
