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
