"""Weight decay of weights held in 32 bits (parameters, or master copies of BF16 ones) where it is small.

With no gradient the step is p (1 - lr decay): lr decay is a product of two FP32 numbers, rounded to 2^-24 of
itself, and the new weight is rounded to nearest: half a step of FP32 at its size, and nothing more that could
be seen. In 8 and in 32 bits, in whole aligned groups and in the others.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

bs = pytest.importorskip("lossless_entropy_coding_interleaved_b200")
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("master", [False, True])
@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("lr,decay", [(1e-5, 0.01), (1e-5, 0.0047), (3e-6, 0.1), (1e-3, 0.1), (1e-3, 0.0)])
def test_a_small_decay_is_not_rounded(bits, master, offset, lr, decay):
    n = 5000
    rng = np.random.default_rng(1)
    w = (rng.standard_normal(n) * 10.0 ** rng.uniform(-3, 3, n)).astype(np.float32)
    p = torch.zeros(n + 8, device="cuda")[offset:offset + n].copy_(torch.from_numpy(w))
    q = torch.zeros(n + 8, dtype=BF, device="cuda")[offset:offset + n].copy_(p) if master else p
    g = torch.zeros(n + 8, dtype=BF, device="cuda")[offset:offset + n]
    opt = bs.AdamW([q], [g], lr=lr, weight_decay=decay, bits=bits, masters=[p] if master else None)
    want = w.astype(np.float64)
    ld = float(np.float32(lr)) * float(np.float32(decay))
    for _ in range(3):
        before = p.double().cpu().numpy()
        opt.step()
        want = before * (1 - ld)
        got = p.cpu().numpy()
        tol = np.spacing(np.maximum(np.abs(got), np.abs(before).astype(np.float32))).astype(np.float64) / 2 + 2.0 ** -23 * ld * np.abs(before)
        bad = np.flatnonzero(np.abs(got - want) > tol)
        assert bad.size == 0, (bad.size, before[bad[:3]], got[bad[:3]], want[bad[:3]])
        if master:
            assert torch.equal(q, p.to(BF))


@pytest.mark.parametrize("pt", [F32, BF])
@pytest.mark.parametrize("decay", [0.0, 0.1])
def test_infinite_weights_stay_infinite(pt, decay):
    p = torch.ones(600, dtype=pt, device="cuda")
    p[::7], p[3::7], p[5::7] = float("-inf"), float("inf"), float("nan")
    keep = p.clone()
    bs.AdamW([p], [torch.full((600,), 0.5, device="cuda")], lr=1e-3, weight_decay=decay).step()
    odd = ~torch.isfinite(keep)
    assert torch.equal(torch.isnan(p), torch.isnan(keep)) and torch.equal(p[odd].nan_to_num(nan=5.0), keep[odd].nan_to_num(nan=5.0))
    # the others: m / sqrt(v) is 1, so 1 - 1e-3 (1 + decay) within 24 roundings of the step and two of the weight (as
    # in test_gpu_adamw.py), eps 2e-8 of the step; in BF16 that is 1, whose lower neighbour is 2^-8 away
    rest = p[~odd].double()
    if pt is BF:
        assert torch.all(rest == 1)
    else:
        assert torch.all((rest - (1 - 1e-3 * (1 + decay))).abs() <= 2.0 ** -24 * (24e-3 + 2) + 2e-11)
