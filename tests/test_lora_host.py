"""CPU checks of the adapters' entry points: sizes, and refusals before any launch."""
import ctypes
import os
import re

import pytest

bs = pytest.importorskip("lossless_entropy_coding_interleaved_b200")
L = bs.lib


def _item(**kw):
    it = bs.LoraItem(d_a=256, d_b=512, rows=64, cols=128, d_x=1024, x_stride=128, d_h=2048, d_y=4096, y_stride=64,
                     d_dy=8192, dy_stride=64, d_g=16384, d_da=32768, d_db=65536)
    for k, v in kw.items():
        setattr(it, k, v)
    return it


def _batch(**kw):
    b = bs.LoraBatch(10, 4, 16, 0, None, None, 256, 1 << 20, None)
    for k, v in kw.items():
        setattr(b, k, v)
    return b


def _forward(items, batch=None):
    arr = (bs.LoraItem * max(1, len(items)))(*items)
    return L.bs_lora_forward(len(items), arr, ctypes.byref(batch or _batch()), None)


def _backward(items, batch=None, flags=0):
    arr = (bs.LoraItem * max(1, len(items)))(*items)
    return L.bs_lora_backward(len(items), arr, ctypes.byref(batch or _batch()), flags, None)


def test_sizes():
    assert L.bs_lora_plan_bytes(0, 1) > 0 and L.bs_lora_plan_bytes(1 << 20, 8192) > 4 << 20
    for t, n in (((1 << 20) + 1, 1), (5, 0), (5, 8193)):
        assert L.bs_lora_plan_bytes(t, n) == 0
    assert [L.bs_lora_state_bytes(10, r) for r in (8, 16, 24, 32, 40, 64, 72, 128)] == [60 * p for p in (16, 16, 32, 32, 64, 64, 128, 128)]
    assert L.bs_lora_state_bytes(0, 8) > 0
    for t, r in (((1 << 20) + 1, 8), (5, 0), (5, 4), (5, 12), (5, 136)):
        assert L.bs_lora_state_bytes(t, r) == 0


def test_plan_refusals_before_any_launch():
    need = L.bs_lora_plan_bytes(10, 4)
    plan = lambda idx=256, t=10, n=4, p=256, b=need, e=None: L.bs_lora_plan(idx, t, n, p, b, e, None)  # noqa: E731
    assert plan(idx=None) == bs.E_ARG and plan(idx=258) == bs.E_ARG and plan(p=None) == bs.E_ARG and plan(p=264) == bs.E_ARG
    assert plan(n=0) == bs.E_ARG and plan(t=(1 << 20) + 1) == bs.E_ARG and plan(e=2) == bs.E_ARG and plan(b=need - 1) == bs.E_SIZE


def test_batch_refusals_before_any_launch():
    for b in (_batch(tokens=(1 << 20) + 1), _batch(n_adapters=0), _batch(n_adapters=8193), _batch(rank_max=0), _batch(rank_max=12),
              _batch(rank_max=136), _batch(reserved=1), _batch(d_plan=None), _batch(d_plan=8), _batch(d_ranks=2), _batch(d_scales=1), _batch(d_err=2),
              _batch(plan_bytes=L.bs_lora_plan_bytes(10, 4) - 1)):
        assert _forward([_item()], b) == bs.E_ARG and _backward([_item()], b) == bs.E_ARG
    assert L.bs_lora_forward(1, None, ctypes.byref(_batch()), None) == bs.E_ARG
    assert L.bs_lora_forward(-1, ctypes.byref(_item()), ctypes.byref(_batch()), None) == bs.E_ARG
    assert L.bs_lora_backward(0, None, None, 0, None) == bs.E_ARG


def test_item_refusals_before_any_launch():
    common = [dict(d_a=None), dict(d_a=264), dict(d_b=None), dict(d_b=520), dict(rows=0), dict(rows=60), dict(cols=4), dict(cols=130),
              dict(rows=(1 << 24) + 8), dict(type=2), dict(reserved=1), dict(d_x=None), dict(d_x=1026), dict(x_stride=120),
              dict(x_stride=132), dict(d_h=None), dict(d_h=2056)]
    for kw in common + [dict(d_y=4100), dict(y_stride=56), dict(y_stride=66), dict(type=1, y_stride=68), dict(d_base=4100, base_stride=64),
                        dict(d_base=4096, base_stride=60), dict(d_y=None, d_base=4096, base_stride=64)]:
        assert _forward([_item(**kw)]) == bs.E_ARG, kw
    for kw in common + [dict(d_dy=None), dict(d_dy=8194), dict(dy_stride=56), dict(dy_stride=68), dict(d_g=None), dict(d_g=8),
                        dict(d_da=None), dict(d_db=None), dict(d_da=32772), dict(d_dx=4104, dx_stride=128), dict(d_dx=4096, dx_stride=64),
                        dict(d_dx=4096, dx_stride=130), dict(d_dx_base=4096, dx_base_stride=128)]:
        assert _backward([_item(**kw)]) == bs.E_ARG, kw
    assert _backward([_item()], flags=2) == bs.E_ARG


def test_two_items_of_one_call_may_not_write_the_same_memory():
    other = dict(d_h=1 << 20, d_y=1 << 21, d_g=1 << 22, d_da=1 << 23, d_db=1 << 24)
    for k in ("d_h", "d_y"):
        assert _forward([_item(), _item(**{**other, k: getattr(_item(), k)})]) == bs.E_ARG, k
    for k in ("d_g", "d_da", "d_db"):
        assert _backward([_item(), _item(**{**other, k: getattr(_item(), k)})]) == bs.E_ARG, k
    # one dx for two items has to be described alike
    dx = dict(d_dx=1 << 25, dx_stride=128)
    for kw in (dict(dx_stride=136), dict(type=1), dict(d_dx_base=1 << 26, dx_base_stride=128)):
        assert _backward([_item(**dx), _item(**{**other, **dx, **kw})]) == bs.E_ARG, kw


def test_what_a_call_writes_may_not_be_what_it_reads():
    square = dict(rows=128, y_stride=128, dy_stride=128, type=1)
    for kw in (dict(d_y=1024), dict(d_base=4096, base_stride=136)):
        assert _forward([_item(**{**square, **kw})]) == bs.E_ARG, kw
    other = dict(d_h=1 << 20, d_y=1 << 21, d_g=1 << 22, d_da=1 << 23, d_db=1 << 24, d_x=1 << 27, d_dy=1 << 28)
    for kw in (dict(d_x=4096), dict(d_base=4096, base_stride=64)):
        assert _forward([_item(), _item(**{**other, **kw})]) == bs.E_ARG, kw
    dx = dict(dx_stride=128, type=1)
    for kw in (dict(d_dx=1024), dict(d_dx=8192), dict(d_dx=1 << 25, d_dx_base=1 << 25, dx_base_stride=136), dict(d_g=2048)):
        assert _backward([_item(**{**square, **dx, **kw})]) == bs.E_ARG, kw
    for kw in (dict(d_x=1 << 25), dict(d_dy=1 << 25), dict(d_h=16384)):
        assert _backward([_item(**dx, d_dx=1 << 25), _item(**{**other, **kw})]) == bs.E_ARG, kw


def _source(name):
    src = open(os.path.join(os.path.dirname(bs.__file__), "csrc", name)).read()
    return re.sub(r"//[^\n]*", "", src)


@pytest.mark.parametrize("name", ["bs_lora.cuh", "bs_lora_tc.cuh", "bs_lora.cu", "bs_lora_few.cu", "bs_fw_gemv.cu"])
def test_kernels_that_start_beside_the_one_before_read_nothing_as_constant(name):
    # ld.global.nc is undefined for data that is written while the kernel runs, and a programmatic dependent
    # launch runs from before the end of the kernel that may write its x, its index or its weights
    assert not re.search(r"__ldg|ld\.global(\.\w+)*\.nc|__ldlu|__ldcs\b", _source(name))


def test_kernels_let_the_next_one_go_only_once_they_hold_their_tensor_memory():
    # else a CTA of the next kernel could take the tensor memory that one of this kernel still waits for, and
    # wait for this kernel itself: in every kernel the release stands behind the barrier that follows the
    # allocation, for all threads, and nowhere else
    kernels = [k for k in re.split(r"(?=__global__)", _source("bs_lora.cu") + _source("bs_lora_few.cu")) if k.startswith("__global__")]
    assert len(kernels) == 5
    taking = [k for k in kernels if "tmem_alloc(" in k]
    assert len(taking) == 3
    for k in taking:
        assert k.count("next_kernel_may_start();") == 1 and "launch_dependents" not in k
        before = k[:k.index("next_kernel_may_start();")]
        assert before.index("tmem_alloc(") < before.index("kernels_before_done();") < before.rindex("__syncthreads();")
        assert re.search(r"__syncthreads\(\);\s*fence_after\(\);\s*const uint32_t tmem = s_tmem;\s*(if \(!p\.beside_expand\) )?$", before)
    assert all("launch_dependents" not in _source(f) for f in ("bs_lora.cu", "bs_lora_few.cu", "bs_lora_tc.cuh"))


class _Shared(bs.LoraAdapters):
    """Adapters without tensors whose last batch's size another thread replaces after every look at it."""
    others = ()

    def __init__(self, rank_max, last):
        self.n, self.rank_max, self._n, self._index, self._array = 4, rank_max, 1, -1, bs.LoraItem * 1
        self._ranks_at = self._scales_at = None
        self.last = last

    @property
    def _need(self):
        now, self.last = self.last, self.other
        return now

    @_need.setter
    def _need(self, v):
        self.last = self.other


class _Plan:
    n_adapters, _index, _args = 4, -1, (0, 4, 256, 1 << 20, 0)

    def __init__(self, tokens):
        self.tokens = tokens


@pytest.mark.parametrize("last", [5, 9, 300])
@pytest.mark.parametrize("other", [1, 1000])
def test_a_state_is_held_against_its_own_batch_whatever_other_threads_serve(last, other):
    import torch
    size = lambda t: (t, L.bs_lora_state_bytes(t, 16))  # noqa: E731
    who = _Shared(16, size(last))
    who.other = size(other)
    state = lambda t: [torch.zeros(size(t)[1], dtype=torch.uint8)]  # noqa: E731
    who._begin(_Plan(9), (), state(9))
    who.last = size(last)
    with pytest.raises(bs.BsError) as e:
        who._begin(_Plan(9), (), [state(9)[0][:-1]])
    assert e.value.code == bs.E_SIZE


def test_a_dx_may_not_be_the_base_of_another():
    dx = dict(dx_stride=128, type=1)
    other = dict(d_h=1 << 20, d_y=1 << 21, d_g=1 << 22, d_da=1 << 23, d_db=1 << 24, d_x=1 << 27, d_dy=1 << 28, dx_base_stride=128, **dx)
    for d_dx in (1 << 26, None):
        items = [_item(**dx, d_dx=1 << 25), _item(**other, d_dx=d_dx, d_dx_base=1 << 25)]
        assert _backward(items) == bs.E_ARG and _backward(items[::-1]) == bs.E_ARG


def test_the_check_answers_what_the_call_would():
    check = lambda items, batch=None: L.bs_lora_forward_check(len(items), (bs.LoraItem * max(1, len(items)))(*items), ctypes.byref(batch or _batch()))  # noqa: E731
    assert check([_item()]) == check([]) == check([_item(d_base=4096, base_stride=64)]) == bs.OK
    for kw in (dict(d_y=4100), dict(rows=60), dict(x_stride=120), dict(d_x=4096), dict(d_h=2056)):
        assert check([_item(**kw)]) == _forward([_item(**kw)]) == bs.E_ARG, kw
    assert check([_item()], _batch(rank_max=12)) == bs.E_ARG and check([_item(), _item()]) == bs.E_ARG
    assert L.bs_lora_forward_check(-1, None, ctypes.byref(_batch())) == bs.E_ARG and L.bs_lora_forward_check(1, None, None) == bs.E_ARG


def test_what_an_sm_holds_of_clustered_kernels_finds_its_tensor_memory():
    # checked when the library is compiled; here: that it still is, of every kernel that is launched as a cluster and
    # takes tensor memory, by the sizes that the launches use
    src = _source("bs_lora.cu")
    assert "static_assert(most_columns(0, kSmShared) <= 512" in src
    table = src[src.index("kClustered[] = {"):src.index("constexpr uint32_t most_columns")]
    for r in (16, 32, 64, 128):
        for wt in ("false", "true"):
            assert f"{{shrink_tmem<{r}>, shrink_smem<{r}, {wt}>()}}" in table
        assert f"{{outer_tmem<{r}>, outer_smem<{r}>()}}" in table
        assert f"launch<lora_shrink_kernel<{r}, WT>, shrink_threads<{r}>>(grid, shrink_smem<{r}, WT>(), p.split" in src
        assert f"launch<lora_outer_kernel<{r}>, outer_threads<{r}>>(grid, outer_smem<{r}>(), p.split" in src
    assert src.count("constexpr uint32_t kTmem = shrink_tmem<R>") == src.count("constexpr uint32_t kTmem = outer_tmem<R>") == 1
    assert re.findall(r"lora_expand_kernel<[^;]*>\(grid, smem, (\d)", src) == ["1", "1"]  # no cluster
