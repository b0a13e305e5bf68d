"""Which buffers a twin may have: new ones, or whole ones of its handle, but none that overlap in part."""
import pytest
import torch

pytestmark = pytest.mark.gpu

bs = pytest.importorskip("lossless_entropy_coding_interleaved_b200")


def _handle(bits, buf=None):
    p = [torch.ones(300, device="cuda") if buf is None else buf[:300], torch.ones(1000, device="cuda")]
    return bs.AdamW(p, [torch.ones(300, device="cuda"), torch.ones(1000, device="cuda")], lr=0.1, bits=bits, masters=[t.clone() for t in p])


@pytest.mark.parametrize("bits", [8, 32])
def test_a_twin_that_overlaps_its_handle_in_part_is_refused(bits):
    buf = torch.ones(2000, device="cuda")
    a = _handle(bits, buf)
    new = lambda n: torch.zeros(n, device="cuda")  # noqa: E731
    one = a.exp_avg[1]
    bad = [dict(params=[buf[100:400], new(1000)]), dict(params=[a.params[1][:300], new(1000)]), dict(masters=[buf[299:599], new(1000)]),
           dict(params=[a.masters[0], new(1000)]), dict(masters=[a.params[0], new(1000)])]
    if bits == 32:
        bad += [dict(states=([one[:300], new(1000)], [new(300), new(1000)])), dict(states=(list(a.exp_avg_sq), [new(300), new(1000)]))]
    else:
        codes, scales = lambda n: torch.zeros(n, dtype=torch.uint8, device="cuda"), lambda: [new(2), new(4)]  # noqa: E731
        bad += [dict(states=(([one[4:304], codes(1000)], scales()), ([codes(300), codes(1000)], scales()))),
                dict(states=(([codes(300), codes(1000)], a.exp_avg_sq_scale), ([codes(300), codes(1000)], scales())))]
    for kw in bad:
        with pytest.raises(bs.BsError) as e:
            a.twin(**kw)
        assert e.value.code == bs.E_ARG, kw
    b = a.twin()
    with pytest.raises(bs.BsError):  # nor a twin's twin the first handle
        b.twin(params=[buf[100:400], new(1000)])
    a.step(into=b)  # what was refused left nothing behind
    assert torch.equal(buf, torch.ones_like(buf)) and not torch.equal(b.params[1], a.params[1])


@pytest.mark.parametrize("bits", [8, 32])
def test_a_twin_may_share_whole_buffers(bits):
    a, c = _handle(bits), _handle(bits)
    b = a.twin(params=a.params)
    for _ in range(3):
        a.step(into=b)
        c.step()
        a, b = b, a
        assert all(torch.equal(x, y) for x, y in zip(a.params + a.masters + a.exp_avg, c.params + c.masters + c.exp_avg))


def test_memory_of_a_twin_that_is_gone_may_be_used_again():
    a = _handle(32)
    b = a.twin()
    old = [t.untyped_storage() for t in b.params]
    del b
    t = torch.empty(0, device="cuda")
    p = [t.new_empty(0).set_(s, 1, (n,)) for s, n in zip(old, (299, 999))]
    q = [torch.cat([v, v.new_zeros(1)]) for v in p]
    a.twin(params=q)
    x = torch.empty(0, device="cuda").set_(old[1], 0, (300,))
    a.twin(params=[x, torch.zeros(1000, device="cuda")])
