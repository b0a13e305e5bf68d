"""fw_gemv and fw_gemm with adapters that are refused: nothing has been written when the error comes."""
import pytest
import torch

pytestmark = pytest.mark.gpu

bs = pytest.importorskip("lossless_entropy_coding_interleaved_b200")
BF = torch.bfloat16


@pytest.mark.parametrize("product,tokens,rows", [("fw_gemv", 4, 128), ("fw_gemv", 1, 100), ("fw_gemm", 40, 128)])
def test_nothing_is_written_where_the_adapters_are_refused(product, tokens, rows):
    product, cols, n, r = getattr(bs, product), 256, 3, 16
    w = torch.randn(rows, cols, device="cuda").to(BF)
    fw, info = bs.fw_transcode(w.view(torch.int16).reshape(-1))
    x, err = torch.randn(tokens, cols, device="cuda").to(BF), torch.zeros(1, dtype=torch.int32, device="cuda")
    buf = torch.full((tokens * rows + 8,), 7.0, device="cuda")
    y, shifted = buf[:tokens * rows].view(tokens, rows), buf[1:1 + tokens * rows].view(tokens, rows)
    make = lambda rows, cols, k=1: bs.LoraAdapters([torch.zeros(n, r, cols, dtype=BF, device="cuda")] * k, [torch.zeros(n, rows, r, dtype=BF, device="cuda")] * k)  # noqa: E731
    good, plan = make(rows, cols), bs.LoraPlan(tokens, n)
    call = lambda y, *adapters, products=1: product([(fw, info, rows, cols, x, y)] * products, err, adapters=adapters)  # noqa: E731
    bad = [(y, make(rows + 8, cols), plan), (y, make(rows, cols + 8), plan), (y, make(rows, cols, 2), plan), (y, good, bs.LoraPlan(tokens + 1, n)),
           (y, good, bs.LoraPlan(tokens, n + 1)), (y, good, plan, [torch.zeros(16, dtype=torch.uint8, device="cuda")]),
           (y, good, plan, [good.state(tokens)[0][1:].new_zeros(good.state(tokens)[0].numel() + 16)[1:]]), (shifted, good, plan)]
    if rows % 8:
        bad.append((y, good, plan))
    for args in bad:
        with pytest.raises(bs.BsError) as e:
            call(*args)
        assert e.value.code in (bs.E_ARG, bs.E_SIZE)
        assert torch.all(buf == 7.0)
    with pytest.raises(bs.BsError):  # two products, one y
        call(y, make(rows, cols, 2), plan, products=2)
    assert torch.all(buf == 7.0) and int(err) == 0
    if rows % 8 == 0:
        call(y, good, plan)
        assert not torch.any(buf[:tokens * rows] == 7.0) and int(err) == 0 and int(plan.err) == 0
