"""The norm's rounding: 8 squares of a lane are added in FP32 (each addition a fused one: 8 roundings), everything
from there on in 64 bits. So the sum of squares is off by 8 roundings of 2^-24 at most, its root by half of that,
and the result is rounded once: 5 x 2^-24. A longer chain in FP32 would show."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

bs = pytest.importorskip("lossless_entropy_coding_interleaved_b200")
BF, F32, U = torch.bfloat16, torch.float32, 2.0 ** -24


@pytest.mark.parametrize("gt", [F32, BF])
@pytest.mark.parametrize("sizes,offset", [([1], 0), ([8], 1), ([5000, 3], 1), ([1 << 22, 777], 0), ([513] * 900, 0)])
@pytest.mark.parametrize("kind", ["normal", "alike", "one large"])
def test_the_norm_is_five_roundings_off_at_most(gt, sizes, offset, kind):
    rng = np.random.default_rng(sum(sizes))
    gs = []
    for n in sizes:
        v = rng.standard_normal(n) * 0.01 if kind == "normal" else np.full(n, 1 / 3)
        if kind == "one large":
            v[::97] = 1000 / 3
        gs.append(torch.zeros(n + 8, dtype=gt, device="cuda")[offset:offset + n].copy_(torch.from_numpy(v.astype(np.float32))))
    opt = bs.AdamW([torch.zeros(n, device="cuda") for n in sizes], gs)
    got = float(opt.grad_norm(0.5))
    want = float(np.sqrt(sum(np.dot(v, v) for v in (g.double().cpu().numpy() for g in gs))))
    assert abs(got - want) <= 5 * U * want
    # min(1, max_norm / (norm + 1e-6)) of the norm before its own rounding, rounded once
    clip = min(1.0, 0.5 / (want + 1e-6))
    assert abs(float(opt.clip) - clip) <= 5 * U * clip
