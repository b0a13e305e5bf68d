"""CPU checks of the AdamW entry points: refusals before any launch, and the plain formula the GPU
tests compare with (tests/adamw_plain.py) against the 8-bit formats' definitions."""
import ctypes

import numpy as np
import pytest

import adamw_plain as A

bs = pytest.importorskip("lossless_entropy_coding_interleaved_b200")


def _item(**kw):
    it = bs.AdamWItem(d_param=256, d_grad=512, d_m=1024, d_v=2048, d_m_scale=4096, d_v_scale=8192, n=100)
    for k, v in kw.items():
        setattr(it, k, v)
    return it


def _prm(**kw):
    p = bs.AdamWParams(0.9, 0.999, 1e-8, 32, 0, 0)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def _step(item, prm=None, ctl=256, n=1, to=None):
    return bs.lib.bs_adamw(n, ctypes.byref(item) if item is not None else None, ctypes.byref(to) if to is not None else None,
                           ctypes.byref(prm) if prm is not None else None, ctl, None)


def test_step_refusals_before_any_launch():
    ok = _prm()
    for it in (_item(d_param=None), _item(d_grad=None), _item(d_m=None), _item(d_v=None), _item(d_param=258), _item(d_grad=513),
               _item(d_m=1026), _item(d_v=2047), _item(d_master=2), _item(param_type=2), _item(grad_type=7),
               _item(weight_decay=-0.5), _item(weight_decay=float("inf")), _item(weight_decay=float("nan"))):
        assert _step(it, ok) == bs.E_ARG
    assert _step(_item(n=(1 << 34) + 1), ok) == bs.E_SIZE
    assert _step(_item(), None) == bs.E_ARG and _step(_item(), ok, ctl=None) == bs.E_ARG and _step(_item(), ok, ctl=8) == bs.E_ARG
    assert _step(None, ok) == bs.E_ARG and _step(_item(), ok, n=-1) == bs.E_ARG
    for p in (_prm(bits=16), _prm(bits=0), _prm(step=1 << 31), _prm(beta1=1.0), _prm(beta2=1.5), _prm(beta1=-0.1),
              _prm(beta2=float("nan")), _prm(eps=-1e-8), _prm(eps=0.0), _prm(eps=float("inf"))):
        assert _step(_item(), p) == bs.E_ARG
    for it in (_item(d_m_scale=None), _item(d_v_scale=None), _item(d_m_scale=2), _item(d_v_scale=3)):
        assert _step(it, _prm(bits=8)) == bs.E_ARG


def test_norm_and_read_refusals_before_any_launch():
    it = _item()
    need = bs.lib.bs_grad_norm_scratch_bytes(1, ctypes.byref(it))
    assert need >= 8 and bs.lib.bs_grad_norm_scratch_bytes(1, ctypes.byref(_item(d_grad=None))) == 0
    norm = lambda item=it, mx=1.0, ctl=256, sc=256, nb=need: bs.lib.bs_grad_norm(1, ctypes.byref(item), mx, ctl, sc, nb, None)  # noqa: E731
    assert norm(nb=need - 1) == bs.E_SIZE
    assert norm(mx=0.0) == bs.E_ARG and norm(mx=-1.0) == bs.E_ARG and norm(mx=float("nan")) == bs.E_ARG
    assert norm(ctl=None) == bs.E_ARG and norm(sc=None) == bs.E_ARG and norm(item=_item(d_grad=3)) == bs.E_ARG
    out = (ctypes.c_void_p * 1)(256)
    none = (ctypes.c_void_p * 1)(None)
    read = lambda a, b, item=it: bs.lib.bs_adamw_read_states(1, ctypes.byref(item), a, b, None)  # noqa: E731
    assert read(none, out) == bs.E_ARG and read(out, none) == bs.E_ARG and read(None, out) == bs.E_ARG
    assert read(out, out, _item(d_m_scale=None)) == bs.E_ARG
    assert bs.lib.bs_adamw_read_states(1, ctypes.byref(_item(n=0)), none, none, None) == bs.OK


def test_plain_codes_round_up_in_proportion():
    # every code's own value keeps its code whatever the random bits; a value a quarter of the way
    # to the next code goes up for a quarter of them
    for kind, table, top, most in (("m", A.E4M3, 448.0, 0x7E), ("v", A.U53, 61440.0, 0xF7)):
        x = table[1:most + 1].astype(np.float32)
        x = np.concatenate([x, np.full(-x.size % 256, top, np.float32)])
        x.reshape(-1, 256)[:, -1] = top if kind == "m" else x.reshape(-1, 256)[:, -1]
        x[-1] = top
        for u in (0, 65535):
            codes, scales = A.encode(x, np.full(x.size, u), kind)
            assert np.array_equal(table[codes & (0x7F if kind == "m" else 0xFF)].astype(np.float32), x) and np.all(scales == 1)
        y = np.full(65536, np.float32(table[40] + 0.25 * (table[41] - table[40])))
        y = y.reshape(-1, 256)
        y[:, 0] = top
        codes, _ = A.encode(y.reshape(-1), np.tile(np.arange(256) * 256 + 255, 256), kind)
        up = (codes.reshape(-1, 256)[:, 1:] == 41).mean()
        assert set(np.unique(codes.reshape(-1, 256)[:, 1:])) == {40, 41} and abs(up - 0.25) < 0.01


def test_plain_random_bits_are_splitmix64():
    # the first output of splitmix64 seeded with 0 is published: 0xE220A8397B1DCDAF
    z = A._mix(np.array([0x9E3779B97F4A7C15], np.uint64))
    assert int(z[0]) == 0xE220A8397B1DCDAF
    um, uv = A.random_bits(1, 2, 3, 1 << 16)
    assert abs(um.mean() - 32767.5) < 6 * 18919 / 256 and abs(uv.mean() - 32767.5) < 6 * 18919 / 256


def test_a_step_into_other_buffers_is_checked_alike():
    for to in (_item(n=99), _item(param_type=1), _item(d_master=64), _item(d_param=None), _item(d_m=None), _item(d_v=2049)):
        assert _step(_item(), _prm(), to=to) == bs.E_ARG
    assert _step(_item(), _prm(bits=8), to=_item(d_v_scale=None)) == bs.E_ARG
    assert _step(_item(d_master=64), _prm(), to=_item()) == bs.E_ARG
