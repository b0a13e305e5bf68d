"""Python binding of libbs, the sm_100a decoder for BF16RANS containers.

The binding only marshals arguments. Every step of the decode runs in libbs's CUDA
kernels (csrc/bs_kernels.cu), and its host planner is csrc/bs_plan.cpp. PyTorch
supplies device memory and streams. There is no CPU fallback: importing this module
without a built libbs.so raises, and so does planning without a CUDA device.

The method is the one in the paragraph after the accounting table of the
"Qwen3.8-27B-BF16-NVLC-Lossless" model card:
  - each BF16 word is split into sign, exponent and fraction;
  - the sign+exponent symbol is rANS-decoded with a per-tensor model;
  - that symbol selects the 7-bit fraction's distribution;
  - the fields are recombined bitwise.
The byte layout is the BF16RANS container, version 2.
"""
from __future__ import annotations

import array
import bisect
import ctypes
import os
import struct
import weakref

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbs.so")

OK, E_ARG, E_FORMAT, E_VERSION, E_SIZE, E_CUDA, E_CORRUPT, E_NOMEM, E_UNSUPPORTED = range(9)
FW_LAYOUTS_RESIDENT = 1  # bs_fw_gemv flag: no work in flight writes the layouts
KIND_RANS, KIND_STORED, KIND_RAW, KIND_JOINT = 0, 1, 2, 3


class BsError(RuntimeError):
    def __init__(self, code: int, what: str, msg: str = "", first_bad: int = -1):
        super().__init__(f"libbs {what}: {msg or code} (status {code})")
        self.code = code
        self.first_bad = first_bad


class _Range(ctypes.Structure):
    _fields_ = [("idx", ctypes.c_int32), ("reserved", ctypes.c_uint32), ("begin", ctypes.c_uint64),
                ("count", ctypes.c_uint64), ("d_out", ctypes.c_void_p), ("out_bytes", ctypes.c_size_t)]


class _Info(ctypes.Structure):
    _fields_ = [("n_elems", ctypes.c_uint64), ("out_bytes", ctypes.c_uint64), ("coded_bytes", ctypes.c_uint64),
                ("n_chunks", ctypes.c_uint64), ("checksum", ctypes.c_uint64), ("shape", ctypes.c_uint64 * 8),
                ("kind", ctypes.c_uint32), ("ndim", ctypes.c_uint32), ("ns", ctypes.c_uint32),
                ("nh", ctypes.c_uint32), ("n_routes", ctypes.c_uint32), ("log2_chunk", ctypes.c_uint32),
                ("name", ctypes.c_void_p), ("name_bytes", ctypes.c_uint32), ("nib_mode", ctypes.c_uint32)]


class _EncItem(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_uint32), ("ndim", ctypes.c_uint32), ("shape", ctypes.c_uint64 * 8),
                ("n_elems", ctypes.c_uint64), ("d_data", ctypes.c_void_p), ("name", ctypes.c_char_p),
                ("name_bytes", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


class _StreamStats(ctypes.Structure):
    _fields_ = [(k, ctypes.c_uint64) for k in ("loads", "hits", "evictions", "h2d_bytes", "decoded_bytes",
                                                "resident_groups", "cache_bytes", "cache_bytes_used",
                                                "stage_bytes")]


class _EncParams(ctypes.Structure):
    _fields_ = [(k, ctypes.c_uint32) for k in ("log2_chunk", "ns", "nh", "max_routes", "force_rans", "model", "nj")]


class FwInfo(ctypes.Structure):
    """bs_fw_info: the header of a fixed-width lane layout (4-bit codes, 7-bit fractions, exceptions)."""
    _fields_ = [("n_elems", ctypes.c_uint64), ("n_tiles", ctypes.c_uint64), ("n_exc", ctypes.c_uint64),
                ("total_bytes", ctypes.c_uint64), ("table", ctypes.c_uint16 * 16)]

    def __repr__(self):
        return (f"FwInfo(n_elems={self.n_elems}, n_tiles={self.n_tiles}, n_exc={self.n_exc}, "
                f"total_bytes={self.total_bytes}, table={list(self.table)})")


class FwGemvItem(ctypes.Structure):
    """bs_fw_gemv_item: one product y = W x (W in the FW layout)."""
    _fields_ = [("d_fw", ctypes.c_void_p), ("info", FwInfo), ("rows", ctypes.c_uint32), ("cols", ctypes.c_uint32),
                ("d_x", ctypes.c_void_p), ("d_y", ctypes.c_void_p)]


class LoraItem(ctypes.Structure):
    """bs_lora_item: one projection's adapters, inputs and outputs."""
    _fields_ = [("d_a", ctypes.c_void_p), ("d_b", ctypes.c_void_p), ("rows", ctypes.c_uint32), ("cols", ctypes.c_uint32),
                ("type", ctypes.c_uint32), ("reserved", ctypes.c_uint32), ("d_x", ctypes.c_void_p), ("x_stride", ctypes.c_uint64),
                ("d_h", ctypes.c_void_p), ("d_base", ctypes.c_void_p), ("base_stride", ctypes.c_uint64),
                ("d_y", ctypes.c_void_p), ("y_stride", ctypes.c_uint64), ("d_dy", ctypes.c_void_p), ("dy_stride", ctypes.c_uint64),
                ("d_g", ctypes.c_void_p), ("d_dx_base", ctypes.c_void_p), ("dx_base_stride", ctypes.c_uint64),
                ("d_dx", ctypes.c_void_p), ("dx_stride", ctypes.c_uint64), ("d_da", ctypes.c_void_p), ("d_db", ctypes.c_void_p)]


class LoraBatch(ctypes.Structure):
    """bs_lora_batch: the batch that the items of one call share."""
    _fields_ = [("tokens", ctypes.c_uint32), ("n_adapters", ctypes.c_uint32), ("rank_max", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32), ("d_ranks", ctypes.c_void_p), ("d_scales", ctypes.c_void_p),
                ("d_plan", ctypes.c_void_p), ("plan_bytes", ctypes.c_size_t), ("d_err", ctypes.c_void_p)]


class AdamWItem(ctypes.Structure):
    """bs_adamw_item: one tensor of an AdamW step."""
    _fields_ = ([(k, ctypes.c_void_p) for k in ("d_param", "d_grad", "d_master", "d_m", "d_v", "d_m_scale", "d_v_scale")] +
                [("n", ctypes.c_uint64), ("param_type", ctypes.c_uint32), ("grad_type", ctypes.c_uint32),
                 ("weight_decay", ctypes.c_float), ("reserved", ctypes.c_uint32)])


class AdamWParams(ctypes.Structure):
    _fields_ = [("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("eps", ctypes.c_double),
                ("bits", ctypes.c_uint32), ("step", ctypes.c_uint32), ("seed", ctypes.c_uint64)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libbs.so is not built ({LIB_PATH}); run "
                          f"`python lossless_entropy_coding_interleaved_b200/build.py`")
    L = ctypes.CDLL(LIB_PATH)
    P, i32, u64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint64, ctypes.c_size_t
    L.bs_plan_workspace_bytes.argtypes = [P, sz]
    L.bs_plan_workspace_bytes.restype = sz
    L.bs_plan.argtypes = [P, sz, P, P, sz, P, ctypes.POINTER(P)]
    L.bs_plan_destroy.argtypes = [P]
    L.bs_plan_destroy.restype = None
    L.bs_tensor_count.argtypes = [P, ctypes.POINTER(i32)]
    L.bs_tensor_info_get.argtypes = [P, i32, ctypes.POINTER(_Info)]
    L.bs_decode_tensor.argtypes = [P, i32, P, sz, P]
    L.bs_decode_batch.argtypes = [P, P, P, P, i32, P]
    L.bs_decode_ranges.argtypes = [P, ctypes.POINTER(_Range), i32, P]
    L.bs_decode_geometry.argtypes = [P, i32, ctypes.POINTER(ctypes.c_uint32), ctypes.POINTER(ctypes.c_uint32)]
    L.bs_verify_tensor.argtypes = [P, i32, P, sz, P, P, ctypes.POINTER(u64)]
    L.bs_check.argtypes = [P, P, ctypes.POINTER(ctypes.c_int64)]
    L.bs_status_str.argtypes = [ctypes.c_int]
    L.bs_status_str.restype = ctypes.c_char_p
    L.bs_last_cuda_error.argtypes = []
    L.bs_decode_tensor_noalloc.argtypes = [P, sz, P, i32, P, sz, P]
    L.bs_decode_tensor_noalloc.restype = ctypes.c_int
    L.bs_launch_counter.argtypes = []
    L.bs_launch_counter.restype = u64
    L.bs_plan_workspace_bytes_device.argtypes = [P, sz, P]
    L.bs_plan_workspace_bytes_device.restype = sz
    L.bs_encoder_create.argtypes = [ctypes.POINTER(_EncItem), i32, ctypes.POINTER(_EncParams), ctypes.POINTER(P)]
    L.bs_encoder_scratch_bytes.argtypes = [P, ctypes.POINTER(sz)]
    L.bs_encoder_run.argtypes = [P, P, sz, P, ctypes.POINTER(sz)]
    L.bs_encoder_emit.argtypes = [P, P, P, sz, P, P]
    L.bs_encoder_destroy.argtypes = [P]
    L.bs_encoder_destroy.restype = None
    L.bs_streamer_workspace_bytes.argtypes = [P, sz]
    L.bs_streamer_workspace_bytes.restype = sz
    L.bs_streamer_min_arena_bytes.argtypes = [P, sz, P]
    L.bs_streamer_min_arena_bytes.restype = sz
    L.bs_streamer_create.argtypes = [P, sz, P, P, sz, P, sz, P, ctypes.POINTER(P)]
    L.bs_streamer_group_count.argtypes = [P, ctypes.POINTER(i32)]
    L.bs_streamer_tensor_info_get.argtypes = [P, i32, ctypes.POINTER(_Info)]
    L.bs_streamer_prefetch.argtypes = [P, i32, P]
    L.bs_streamer_acquire.argtypes = [P, i32, P, i32, P]
    L.bs_streamer_release.argtypes = [P, i32, P]
    L.bs_streamer_get_stats.argtypes = [P, ctypes.POINTER(_StreamStats)]
    L.bs_streamer_check.argtypes = [P, P, ctypes.POINTER(ctypes.c_int64)]
    L.bs_streamer_destroy.argtypes = [P]
    L.bs_streamer_destroy.restype = None
    L.bs_fw_scratch_bytes.argtypes = [u64]
    L.bs_fw_scratch_bytes.restype = sz
    L.bs_fw_measure.argtypes = [P, u64, P, sz, P, ctypes.POINTER(FwInfo)]
    L.bs_fw_write.argtypes = [P, u64, P, sz, ctypes.POINTER(FwInfo), P, sz, P]
    L.bs_fw_parse.argtypes = [P, sz, sz, ctypes.POINTER(FwInfo)]
    L.bs_fw_decode.argtypes = [i32, P, P, P, P, P, P]
    L.bs_fw_gemv.argtypes = [i32, ctypes.POINTER(FwGemvItem), ctypes.c_uint32, ctypes.c_uint32, P, P]
    L.bs_fw_gemm.argtypes = [i32, ctypes.POINTER(FwGemvItem), ctypes.c_uint32, P, P]
    LI, LB = ctypes.POINTER(LoraItem), ctypes.POINTER(LoraBatch)
    u32 = ctypes.c_uint32
    L.bs_lora_plan_bytes.argtypes = [u32, u32]
    L.bs_lora_plan_bytes.restype = sz
    L.bs_lora_state_bytes.argtypes = [u32, u32]
    L.bs_lora_state_bytes.restype = sz
    L.bs_lora_plan.argtypes = [P, u32, u32, P, sz, P, P]
    L.bs_lora_forward.argtypes = [i32, LI, LB, P]
    L.bs_lora_forward_check.argtypes = [i32, LI, LB]
    L.bs_lora_backward.argtypes = [i32, LI, LB, u32, P]
    for fn in ("bs_lora_plan", "bs_lora_forward", "bs_lora_forward_check", "bs_lora_backward"):
        getattr(L, fn).restype = ctypes.c_int
    IT = ctypes.POINTER(AdamWItem)
    L.bs_grad_norm_scratch_bytes.argtypes = [i32, IT]
    L.bs_grad_norm_scratch_bytes.restype = sz
    L.bs_grad_norm.argtypes = [i32, IT, ctypes.c_float, P, P, sz, P]
    L.bs_adamw.argtypes = [i32, IT, IT, ctypes.POINTER(AdamWParams), P, P]
    L.bs_adamw_read_states.argtypes = [i32, IT, P, P, P]
    for fn in ("bs_grad_norm", "bs_adamw", "bs_adamw_read_states"):
        getattr(L, fn).restype = ctypes.c_int
    for fn in ("bs_fw_measure", "bs_fw_write", "bs_fw_parse", "bs_fw_decode", "bs_fw_gemv", "bs_fw_gemm"):
        getattr(L, fn).restype = ctypes.c_int
    for fn in ("bs_streamer_create", "bs_streamer_group_count", "bs_streamer_tensor_info_get", "bs_streamer_prefetch", "bs_streamer_acquire",
               "bs_streamer_release", "bs_streamer_get_stats", "bs_streamer_check"):
        getattr(L, fn).restype = ctypes.c_int
    for fn in ("bs_plan", "bs_tensor_count", "bs_tensor_info_get", "bs_decode_tensor", "bs_decode_batch",
               "bs_decode_ranges", "bs_decode_geometry", "bs_verify_tensor", "bs_check", "bs_last_cuda_error", "bs_encoder_create", "bs_encoder_scratch_bytes",
               "bs_encoder_run", "bs_encoder_emit"):
        getattr(L, fn).restype = ctypes.c_int
    return L


lib = _load()

#: every symbol include/bs.h declares
EXPORTS = ("bs_plan_workspace_bytes", "bs_plan_workspace_bytes_device", "bs_plan", "bs_plan_destroy",
           "bs_tensor_count", "bs_tensor_info_get", "bs_decode_tensor", "bs_decode_batch", "bs_decode_ranges",
           "bs_decode_geometry",
           "bs_verify_tensor",
           "bs_check", "bs_encoder_create", "bs_encoder_scratch_bytes", "bs_encoder_run", "bs_encoder_emit",
           "bs_encoder_destroy", "bs_status_str", "bs_last_cuda_error", "bs_launch_counter",
           "bs_decode_tensor_noalloc", "bs_streamer_workspace_bytes", "bs_streamer_min_arena_bytes",
           "bs_streamer_create", "bs_streamer_group_count", "bs_streamer_tensor_info_get", "bs_streamer_prefetch",
           "bs_streamer_acquire",
           "bs_streamer_release", "bs_streamer_get_stats", "bs_streamer_check", "bs_streamer_destroy",
           "bs_fw_scratch_bytes", "bs_fw_measure", "bs_fw_write", "bs_fw_parse", "bs_fw_decode", "bs_fw_gemv",
           "bs_fw_gemm", "bs_lora_plan_bytes", "bs_lora_state_bytes", "bs_lora_plan", "bs_lora_forward", "bs_lora_forward_check", "bs_lora_backward",
           "bs_grad_norm_scratch_bytes", "bs_grad_norm", "bs_adamw", "bs_adamw_read_states")


def decode_noalloc(container, d_container: torch.Tensor, idx: int, out: torch.Tensor, stream=None) -> torch.Tensor:
    """bs_decode_tensor_noalloc: decode tensor idx into out using libbs's static device
    array instead of a workspace. For callers that cannot allocate device memory. It
    synchronises the stream, and calls that overlap on the GPU race on the shared array."""
    h = _host_bytes(container)
    _check(lib.bs_decode_tensor_noalloc(h.ctypes.data, h.size, d_container.data_ptr(), idx, out.data_ptr(),
                                        out.numel() * out.element_size(), _stream(stream)), "decode_tensor_noalloc")
    return out


def launch_counter() -> int:
    """Kernel launches libbs has made in this process."""
    return int(lib.bs_launch_counter())


def _check(st: int, what: str):
    if st != OK:
        msg = lib.bs_status_str(st).decode()
        if st == E_CUDA:
            msg += f" (cudaError {lib.bs_last_cuda_error()})"
        raise BsError(st, what, msg)


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _on(index: int, what: str, fn, *args, stream=None):
    """fn(*args, stream) with device `index` current; the stream is that device's current one by default."""
    if torch.cuda.current_device() != index:
        with torch.cuda.device(index):
            return _on(index, what, fn, *args, stream=stream)
    if stream is not None:
        st = _stream(stream)
    else:
        st = _raw_stream(index) if _raw_stream is not None else torch.cuda.current_stream(index).cuda_stream
    r = fn(*args, st)
    if r != OK:
        _check(r, what)


def _made_on(stream, index: int, make):
    """make()'s new tensors, belonging to the stream that a call is enqueued on: their memory goes back to
    that stream's later work when they are freed, not to another's that may run before the call."""
    if stream is None:
        return make()
    with torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(_stream(stream), device=index)):
        return make()


def _host_bytes(container) -> np.ndarray:
    if isinstance(container, np.ndarray):
        a = np.ascontiguousarray(container.reshape(-1).view(np.uint8))
    else:
        a = np.frombuffer(container, dtype=np.uint8)
    return a


def _info_dict(ti: _Info) -> dict:
    d = {k: getattr(ti, k) for k, _ in _Info._fields_ if k not in ("shape", "name", "name_bytes")}
    d["shape"] = tuple(ti.shape[i] for i in range(ti.ndim))
    d["name"] = ctypes.string_at(ti.name, ti.name_bytes).decode() if ti.name_bytes else ""
    return d


def _container_names(h: np.ndarray) -> list:
    """Tensor names in directory order, read from a container that already passed
    validation (header: n_tensors at byte 16, dir_offset at 24, names_offset at 32; directory:
    144-byte entries with name_offset at 8 and name_bytes at 12)."""
    hdr = h[:64].tobytes()
    nt = int.from_bytes(hdr[16:20], "little")
    d0, n0 = int.from_bytes(hdr[24:32], "little"), int.from_bytes(hdr[32:40], "little")
    names = []
    for k in range(nt):
        e = h[d0 + 144 * k: d0 + 144 * k + 16].tobytes()
        off, nb = int.from_bytes(e[8:12], "little"), int.from_bytes(e[12:16], "little")
        names.append(h[n0 + off: n0 + off + nb].tobytes().decode())
    return names


def workspace_bytes(container) -> int:
    h = _host_bytes(container)
    n = lib.bs_plan_workspace_bytes(h.ctypes.data, h.size)
    if n == 0:
        raise BsError(E_FORMAT, "workspace_bytes", "container fails validation")
    return n


def encode(tensors, log2_chunk: int = 16, ns: int = 11, nh: int = 5, max_routes: int = 15,
           force_rans: bool = False, host_copy: bool = False, stream=None, model: str = "factored", nj: int = 13):
    """Encode device tensors into a container on the device (bs_encoder_*).

    tensors: sequence of (name, tensor) pairs; int16/bfloat16 CUDA tensors are BF16
    words and uint8 CUDA tensors are opaque byte spans. model "factored" codes BF16 tensors
    as kind RANS (ns, nh, routes), "joint" as kind JOINT (one table of precision nj; faster
    to decode). Returns (d_container, h_container),
    a uint8 CUDA tensor and, when host_copy, a uint8 numpy copy (else None).
    """
    keep = []
    items = (_EncItem * max(1, len(tensors)))()
    dev = None
    for k, (name, t) in enumerate(tensors):
        assert t.is_cuda and t.is_contiguous()
        dev = t.device
        if t.dtype == torch.bfloat16:
            t = t.view(torch.int16)
        assert t.dtype in (torch.int16, torch.uint8), t.dtype
        nb = name.encode()
        keep += [t, nb]
        it = items[k]
        it.kind = 0 if t.dtype == torch.int16 else 2
        it.ndim = t.dim()
        for d, v in enumerate(t.shape):
            it.shape[d] = v
        it.n_elems = t.numel()
        it.d_data = t.data_ptr() if t.numel() else None
        it.name = nb
        it.name_bytes = len(nb)
    if dev is None:
        dev = torch.device("cuda")
    assert model in ("factored", "joint")
    prm = _EncParams(log2_chunk, ns, nh, max_routes, 1 if force_rans else 0, 1 if model == "joint" else 0, nj)
    enc = ctypes.c_void_p()
    _check(lib.bs_encoder_create(items, len(tensors), ctypes.byref(prm), ctypes.byref(enc)), "encoder_create")
    try:
        sc = ctypes.c_size_t()
        _check(lib.bs_encoder_scratch_bytes(enc, ctypes.byref(sc)), "encoder_scratch_bytes")
        scratch = torch.empty(max(sc.value, 256), dtype=torch.uint8, device=dev)
        total = ctypes.c_size_t()
        st = _stream(stream)
        with torch.cuda.device(dev):
            _check(lib.bs_encoder_run(enc, scratch.data_ptr(), scratch.numel(), st, ctypes.byref(total)),
                   "encoder_run")
            d_container = torch.empty(total.value, dtype=torch.uint8, device=dev)
            h = np.empty(total.value, dtype=np.uint8) if host_copy else None
            _check(lib.bs_encoder_emit(enc, scratch.data_ptr(), d_container.data_ptr(), total.value,
                                       h.ctypes.data if host_copy else None, st), "encoder_emit")
    finally:
        lib.bs_encoder_destroy(enc)
    return d_container, h


class Plan:
    """A validated container resident in device memory, with its decode tables.

    ``container`` holds the container's bytes on the host (bytes or a uint8 numpy
    array), or is None when ``d_container`` is given: the plan then reads the metadata
    from the device. ``d_container`` is an optional uint8 CUDA tensor that already holds
    the container; without it, the host bytes are copied to ``device``.
    """

    def __init__(self, container=None, device="cuda", d_container: torch.Tensor | None = None, stream=None):
        if not torch.cuda.is_available():
            raise BsError(E_UNSUPPORTED, "plan", "no CUDA device")
        if container is None and d_container is None:
            raise BsError(E_ARG, "plan", "no container")
        self.device = torch.device(device) if d_container is None else d_container.device
        h = None if container is None else _host_bytes(container)
        if d_container is None:
            d_container = torch.from_numpy(h.copy()).to(self.device)
        assert d_container.dtype == torch.uint8 and d_container.is_cuda
        assert h is None or d_container.numel() == h.size
        self.d_container = d_container
        self.container_bytes = d_container.numel()
        st = _stream(stream)
        with torch.cuda.device(self.device):
            if h is not None:
                ws = workspace_bytes(h)
            else:
                ws = lib.bs_plan_workspace_bytes_device(d_container.data_ptr(), d_container.numel(), st)
                if ws == 0:
                    raise BsError(E_FORMAT, "workspace_bytes", "container fails validation")
            self.workspace = torch.empty(ws, dtype=torch.uint8, device=self.device)
            self._scratch = torch.zeros(2, dtype=torch.int64, device=self.device)
            ptr = ctypes.c_void_p()
            _check(lib.bs_plan(None if h is None else h.ctypes.data, self.container_bytes, d_container.data_ptr(),
                               self.workspace.data_ptr(), ws, st, ctypes.byref(ptr)), "plan")
        self._p = ptr
        n = ctypes.c_int32()
        _check(lib.bs_tensor_count(self._p, ctypes.byref(n)), "tensor_count")
        self.n_tensors = n.value
        self._info = [self._get_info(k) for k in range(self.n_tensors)]
        self.names = [i["name"] for i in self._info]

    def __del__(self):
        p = getattr(self, "_p", None)
        if p and lib is not None:
            lib.bs_plan_destroy(p)
            self._p = None

    def _get_info(self, idx: int) -> dict:
        ti = _Info()
        _check(lib.bs_tensor_info_get(self._p, idx, ctypes.byref(ti)), "tensor_info")
        return _info_dict(ti)

    def info(self, idx: int) -> dict:
        return dict(self._info[idx])

    def empty_output(self, idx: int) -> torch.Tensor:
        """A device buffer of the right size and dtype for tensor idx: int16 words viewable
        as bfloat16, or uint8 for RAW."""
        i = self._info[idx]
        if i["kind"] == KIND_RAW:
            return torch.empty(i["n_elems"], dtype=torch.uint8, device=self.device)
        return torch.empty(i["shape"] if i["shape"] else (), dtype=torch.int16, device=self.device)

    def decode(self, idx: int, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        if out is None:
            out = self.empty_output(idx)
        _check(lib.bs_decode_tensor(self._p, idx, out.data_ptr(), out.numel() * out.element_size(),
                                    _stream(stream)), "decode_tensor")
        return out

    def decode_batch(self, idxs, outs=None, stream=None):
        idxs = list(idxs)
        if outs is None:
            outs = [self.empty_output(k) for k in idxs]
        n = len(idxs)
        ia = (ctypes.c_int32 * max(n, 1))(*idxs)
        pa = (ctypes.c_void_p * max(n, 1))(*[o.data_ptr() for o in outs])
        ba = (ctypes.c_size_t * max(n, 1))(*[o.numel() * o.element_size() for o in outs])
        _check(lib.bs_decode_batch(self._p, ia, pa, ba, n, _stream(stream)), "decode_batch")
        return outs

    def decode_ranges(self, ranges, stream=None):
        """bs_decode_ranges: ranges is a sequence of (idx, begin, count, out). Elements
        [begin, begin + count) of tensor idx (bytes for RAW) are decoded into out; for coded
        kinds the range covers whole chunks (it may end at the tensor's end)."""
        ranges = list(ranges)
        n = len(ranges)
        ra = (_Range * max(n, 1))()
        for k, (idx, begin, count, out) in enumerate(ranges):
            ra[k].idx, ra[k].reserved, ra[k].begin, ra[k].count = idx, 0, begin, count
            ra[k].d_out = out.data_ptr() if out.numel() else None
            ra[k].out_bytes = out.numel() * out.element_size()
        _check(lib.bs_decode_ranges(self._p, ra, n, _stream(stream)), "decode_ranges")
        return [r[3] for r in ranges]

    def decode_geometry(self, idx: int):
        """bs_decode_geometry: (chunks one CTA of tensor idx's decode takes, CTAs per wave)."""
        cpc, wave = ctypes.c_uint32(), ctypes.c_uint32()
        _check(lib.bs_decode_geometry(self._p, idx, ctypes.byref(cpc), ctypes.byref(wave)), "decode_geometry")
        return cpc.value, wave.value

    def to_fw(self, idx: int, scratch: torch.Tensor | None = None, stream=None):
        """The fixed-width lane layout of BF16 tensor idx, built on the
        device from the container, as the runtime of the NVLC card derives its streams from
        the rANS files at start-up. The tensor is decoded (bs_decode_tensor) into `scratch`
        (or a temporary), checked (bs_check), then transcoded (bs_fw_measure, bs_fw_write).
        Returns (layout, FwInfo). Synchronises the stream."""
        i = self._info[idx]
        if i["kind"] == KIND_RAW:
            raise BsError(E_ARG, "to_fw", "a RAW tensor has no BF16 words")
        n = i["n_elems"]
        if scratch is None or scratch.numel() < n:
            scratch = torch.empty(max(n, 1), dtype=torch.int16, device=self.device)
        words = scratch.view(-1)[:n]
        self.decode(idx, words, stream=stream)
        self.check(stream=stream)
        return fw_transcode(words, stream=stream)

    def verify(self, idx: int, out: torch.Tensor, stream=None) -> int:
        """Checksum of a decoded tensor computed on the device; raises BsError(E_CORRUPT)
        if it differs from the stored one. Synchronises the stream."""
        got = ctypes.c_uint64()
        st = lib.bs_verify_tensor(self._p, idx, out.data_ptr(), out.numel() * out.element_size(),
                                  self._scratch.data_ptr(), _stream(stream), ctypes.byref(got))
        _check(st, "verify_tensor")
        return got.value

    def check(self, stream=None) -> int:
        """Synchronise and read the device error word: -1 if clean, else raises BsError with
        first_bad = (tensor << 40) | chunk."""
        fb = ctypes.c_int64()
        st = lib.bs_check(self._p, _stream(stream), ctypes.byref(fb))
        if st == E_CORRUPT:
            raise BsError(st, "check", "corrupt chunk", first_bad=fb.value)
        _check(st, "check")
        return fb.value


def _group_list(groups, names) -> list:
    if callable(groups):
        keys = {}
        groups = [keys.setdefault(groups(n), len(keys)) for n in names]
    groups = [int(g) for g in groups]
    if len(groups) != len(names):
        raise BsError(E_ARG, "streamer", "one group number per tensor")
    return groups


def streamer_min_arena_bytes(container, groups) -> int:
    """bs_streamer_min_arena_bytes: the smallest device budget for this grouping (two
    staging slots plus the largest decoded group)."""
    h = container.numpy() if isinstance(container, torch.Tensor) else _host_bytes(container)
    if lib.bs_streamer_workspace_bytes(h.ctypes.data, h.size) == 0:
        raise BsError(E_FORMAT, "streamer", "container fails validation")
    g = _group_list(groups, _container_names(h))
    ga = (ctypes.c_int32 * max(1, len(g)))(*g)
    n = lib.bs_streamer_min_arena_bytes(h.ctypes.data, h.size, ga)
    if n == 0:
        raise BsError(E_ARG, "streamer", "invalid grouping")
    return n


class Streamer:
    """Layer streaming (bs_streamer_*): decode groups of tensors on demand from a container
    in host memory into a device cache of ``arena_bytes`` with least-recently-used eviction.

    ``groups`` gives each tensor's group number in directory order: a list of ints, or a
    callable name -> hashable key, whose distinct keys are numbered in order of first use.
    The host bytes are copied once into page-locked memory, so the host-to-device copies
    can overlap other work; a page-locked uint8 CPU tensor is used in place instead. ``arena_bytes`` is the whole device budget: two staging slots
    plus the cache (at least ``min_arena_bytes``).
    """

    def __init__(self, container, groups, arena_bytes: int | None = None, device="cuda", stream=None):
        if not torch.cuda.is_available():
            raise BsError(E_UNSUPPORTED, "streamer", "no CUDA device")
        self.device = torch.device(device)
        if isinstance(container, torch.Tensor) and container.dtype == torch.uint8 and container.is_pinned():
            self.host = container.reshape(-1)          # used in place: it must stay unchanged
        else:
            h = _host_bytes(container)
            self.host = torch.empty(h.size, dtype=torch.uint8, pin_memory=True)
            self.host.numpy()[:] = h
        hp, hn = self.host.data_ptr(), self.host.numel()
        ws = lib.bs_streamer_workspace_bytes(hp, hn)
        if ws == 0:
            raise BsError(E_FORMAT, "streamer", "container fails validation")
        self.names = _container_names(self.host.numpy())
        groups = _group_list(groups, self.names)
        self._groups = (ctypes.c_int32 * max(1, len(groups)))(*groups)
        self.min_arena_bytes = lib.bs_streamer_min_arena_bytes(hp, hn, self._groups)
        if self.min_arena_bytes == 0:
            raise BsError(E_ARG, "streamer", "invalid grouping")
        if arena_bytes is None:
            arena_bytes = self.min_arena_bytes
        with torch.cuda.device(self.device):
            self.workspace = torch.empty(ws, dtype=torch.uint8, device=self.device)
            self.arena = torch.empty(arena_bytes, dtype=torch.uint8, device=self.device)
            ptr = ctypes.c_void_p()
            _check(lib.bs_streamer_create(hp, hn, self._groups, self.workspace.data_ptr(), ws,
                                          self.arena.data_ptr(), arena_bytes, _stream(stream), ctypes.byref(ptr)),
                   "streamer_create")
        self._s = ptr
        n = ctypes.c_int32()
        _check(lib.bs_streamer_group_count(self._s, ctypes.byref(n)), "streamer_group_count")
        self.n_groups = n.value
        self.members = [[k for k, g in enumerate(groups) if g == j] for j in range(self.n_groups)]
        self._info = []
        for k in range(len(self.names)):
            ti = _Info()
            _check(lib.bs_streamer_tensor_info_get(self._s, k, ctypes.byref(ti)), "streamer_tensor_info")
            self._info.append(_info_dict(ti))

    def info(self, idx: int) -> dict:
        return dict(self._info[idx])

    def __del__(self):
        s = getattr(self, "_s", None)
        if s and lib is not None:
            torch.cuda.synchronize(self.device)
            lib.bs_streamer_destroy(s)
            self._s = None

    def prefetch(self, group: int, stream=None):
        _check(lib.bs_streamer_prefetch(self._s, group, _stream(stream)), "streamer_prefetch")

    def acquire(self, group: int, stream=None) -> list:
        """Pin the group and return its tensors as views into the arena (int16 words shaped
        like the originals, uint8 for RAW), valid until release."""
        m = self.members[group] if 0 <= group < self.n_groups else []
        ptrs = (ctypes.c_void_p * max(1, len(m)))()
        _check(lib.bs_streamer_acquire(self._s, group, ptrs, len(m), _stream(stream)), "streamer_acquire")
        base = self.arena.data_ptr()
        out = []
        for k, p in zip(m, ptrs):
            i = self._info[k]
            off = (p or base) - base
            if i["kind"] == KIND_RAW:
                out.append(self.arena[off:off + i["n_elems"]])
            else:
                v = self.arena[off:off + 2 * i["n_elems"]].view(torch.int16)
                out.append(v.view(i["shape"]) if i["shape"] else v.view(()))
        return out

    def release(self, group: int, stream=None):
        _check(lib.bs_streamer_release(self._s, group, _stream(stream)), "streamer_release")

    def stats(self) -> dict:
        st = _StreamStats()
        _check(lib.bs_streamer_get_stats(self._s, ctypes.byref(st)), "streamer_stats")
        return {k: getattr(st, k) for k, _ in _StreamStats._fields_}

    def check(self, stream=None) -> int:
        fb = ctypes.c_int64()
        st = lib.bs_streamer_check(self._s, _stream(stream), ctypes.byref(fb))
        if st == E_CORRUPT:
            raise BsError(st, "streamer_check", "corrupt chunk", first_bad=fb.value)
        _check(st, "streamer_check")
        return fb.value


# ------------------------------------------------------------ fixed-width lane layout
def _words(t: torch.Tensor) -> torch.Tensor:
    assert t.is_cuda and t.is_contiguous() and t.element_size() == 2, "BF16 words: a contiguous 2-byte CUDA tensor"
    return t


def fw_scratch_bytes(n_elems: int) -> int:
    return int(lib.bs_fw_scratch_bytes(n_elems))


def fw_transcode(words: torch.Tensor, stream=None) -> tuple[torch.Tensor, FwInfo]:
    """Build the fixed-width lane layout of BF16 words on their device (bs_fw_measure, then
    bs_fw_write). Returns (layout as a uint8 CUDA tensor, its FwInfo). Synchronises the stream."""
    w = _words(words)
    n = w.numel()
    scratch = torch.empty(max(fw_scratch_bytes(n), 256), dtype=torch.uint8, device=w.device)
    info = FwInfo()
    st = _stream(stream)
    with torch.cuda.device(w.device):
        _check(lib.bs_fw_measure(w.data_ptr() if n else None, n, scratch.data_ptr(), scratch.numel(), st,
                                 ctypes.byref(info)), "fw_measure")
        fw = torch.empty(info.total_bytes, dtype=torch.uint8, device=w.device)
        _check(lib.bs_fw_write(w.data_ptr() if n else None, n, scratch.data_ptr(), scratch.numel(),
                               ctypes.byref(info), fw.data_ptr(), fw.numel(), st), "fw_write")
    return fw, info


def fw_parse(head, fw_bytes: int) -> FwInfo:
    """bs_fw_parse of a host copy of a layout's first 96 bytes (or more)."""
    h = _host_bytes(head)
    info = FwInfo()
    _check(lib.bs_fw_parse(h.ctypes.data, h.size, fw_bytes, ctypes.byref(info)), "fw_parse")
    return info


def fw_decode(fws, infos, outs, err: torch.Tensor, stream=None):
    """bs_fw_decode: decode layouts fws[k] (uint8 CUDA tensors, headers infos[k]) into outs[k]
    (2-byte CUDA tensors of n_elems). err: a zeroed int32 CUDA tensor of one element that
    receives the error flags. Enqueued on the stream."""
    n = len(fws)
    assert len(infos) == n and len(outs) == n
    P = ctypes.c_void_p
    p_fw = (P * max(n, 1))(*[f.data_ptr() for f in fws])
    p_out = (P * max(n, 1))(*[_words(o).data_ptr() if o.numel() else None for o in outs])
    sizes = (ctypes.c_size_t * max(n, 1))(*[o.numel() * 2 for o in outs])
    inf = (FwInfo * max(n, 1))(*infos)
    assert err.is_cuda and err.dtype == torch.int32 and err.numel() >= 1
    with torch.cuda.device(err.device):
        _check(lib.bs_fw_decode(n, p_fw, inf, p_out, sizes, err.data_ptr(), _stream(stream)), "fw_decode")
    return outs


def _fw_products(products, max_batch):
    n = len(products)
    arr = (FwGemvItem * max(n, 1))()
    batch = None
    for k, (fw, info, rows, cols, x, y) in enumerate(products):
        b = 1 if x.dim() == 1 else x.shape[0]
        assert batch in (None, b), "every product of one call has the same batch"
        batch = b
        assert max_batch is None or b <= max_batch
        assert x.is_cuda and x.is_contiguous() and x.element_size() == 2 and x.numel() == b * cols
        assert y.is_cuda and y.is_contiguous() and y.dtype == torch.float32 and y.numel() == b * rows
        arr[k].d_fw = fw.data_ptr()
        arr[k].info = info
        arr[k].rows, arr[k].cols = rows, cols
        arr[k].d_x = x.data_ptr()
        arr[k].d_y = y.data_ptr()
    return n, arr, batch or 1


def _with_adapters(products, adapters, stream):
    """What adds each token's adapter to the products' outputs, to be called once they are enqueued: adapters is
    (LoraAdapters, LoraPlan) or (LoraAdapters, LoraPlan, state), the adapters' projections being the products
    in order. Whatever is to be refused of them is refused here, before anything is enqueued."""
    if adapters is None:
        return lambda: None
    who, plan = adapters[:2]
    two = lambda t: t.view(1, -1) if t.dim() == 1 else t  # noqa: E731
    args = who._forward_args(plan, [two(p[4].view(torch.bfloat16)) for p in products], [two(p[5]) for p in products], None,
                             adapters[2] if len(adapters) > 2 else None, stream)
    _check(lib.bs_lora_forward_check(*args[:3]), "lora_forward")
    return lambda: _on(who._index, "lora_forward", lib.bs_lora_forward, *args[:3], stream=stream)


def fw_gemm(products, err: torch.Tensor, stream=None, adapters=None):
    """bs_fw_gemm: as fw_gemv, on the tensor cores, for any batch (rows a multiple of 128):
    products is a sequence of (fw, info, rows, cols, x [batch, cols] BF16, y [batch, rows] float32).
    err: a zeroed int32 CUDA tensor of one element. adapters: as fw_gemv's. Enqueued on the stream."""
    n, arr, batch = _fw_products(products, None)
    assert err.is_cuda and err.dtype == torch.int32 and err.numel() >= 1
    add = _with_adapters(products, adapters, stream)
    with torch.cuda.device(err.device):
        _check(lib.bs_fw_gemm(n, arr, batch, err.data_ptr(), _stream(stream)), "fw_gemm")
    add()
    return [p[5] for p in products]


def fw_gemv(products, err: torch.Tensor, stream=None, layouts_resident: bool = False, adapters=None):
    """bs_fw_gemv: products is a sequence of (fw, info, rows, cols, x, y) with fw the layout of
    W (rows x cols), x a BF16 CUDA tensor [batch, cols] (or [cols]) and y a float32 CUDA
    tensor [batch, rows] (or [rows]); every x has the same batch (1..8). err: a zeroed int32
    CUDA tensor of one element. Enqueued on the stream. layouts_resident: BS_FW_LAYOUTS_RESIDENT,
    a statement that no work in flight on the stream writes the layouts (resident weights), so
    that their copies may start before the preceding kernel has finished. adapters: low-rank adapters
    beside the products, (LoraAdapters, LoraPlan) or (LoraAdapters, LoraPlan, state), whose projections
    are the products in order and whose tokens are the batch; their part is added to every y
    (bs_lora_forward), and the state that a backward pass needs is left in state."""
    n = len(products)
    arr = (FwGemvItem * max(n, 1))()
    batch = None
    for k, (fw, info, rows, cols, x, y) in enumerate(products):
        b = 1 if x.dim() == 1 else x.shape[0]
        assert batch in (None, b), "every product of one call has the same batch"
        batch = b
        assert x.is_cuda and x.is_contiguous() and x.element_size() == 2 and x.numel() == b * cols
        assert y.is_cuda and y.is_contiguous() and y.dtype == torch.float32 and y.numel() == b * rows
        arr[k].d_fw = fw.data_ptr()
        arr[k].info = info
        arr[k].rows, arr[k].cols = rows, cols
        arr[k].d_x = x.data_ptr()
        arr[k].d_y = y.data_ptr()
    assert err.is_cuda and err.dtype == torch.int32 and err.numel() >= 1
    add = _with_adapters(products, adapters, stream)
    with torch.cuda.device(err.device):
        _check(lib.bs_fw_gemv(n, arr, batch or 1, FW_LAYOUTS_RESIDENT if layouts_resident else 0, err.data_ptr(),
                              _stream(stream)), "fw_gemv")
    add()
    return [p[5] for p in products]


# ------------------------------------------------------------ low-rank adapters
_TYPES = {torch.float32: 0, torch.bfloat16: 1}
LORA_ACCUMULATE = 1
_LORA_ITEM = struct.Struct("=QQIIII16Q")  # LoraItem's fields in order
assert _LORA_ITEM.size == ctypes.sizeof(LoraItem) == 160


class LoraPlan:
    """The routing of a batch of ``tokens`` tokens to ``n_adapters`` adapters (bs_lora_plan), in
    device memory. update(idx) sets it from an int32 CUDA tensor, an adapter per token (negative:
    none; a new plan gives no token an adapter); one plan serves every projection of the batch, and may be updated for the next batch.
    ``err``, an int32 device word, gathers what the calls that use the plan report: bit 2 an index past
    the adapters, bit 1 a wait inside a kernel that ran out, bit 3 a plan of another batch (the last two
    never in a working program)."""

    def __init__(self, tokens: int, n_adapters: int, device="cuda"):
        if not torch.cuda.is_available():
            raise BsError(E_UNSUPPORTED, "lora_plan", "no CUDA device")
        nb = lib.bs_lora_plan_bytes(tokens, n_adapters) if 0 <= tokens < 2 ** 32 and 0 <= n_adapters < 2 ** 32 else 0
        if nb == 0:
            raise BsError(E_ARG, "lora_plan", "tokens up to 2^20, adapters 1..8192")
        self.tokens, self.n_adapters = tokens, n_adapters
        self.data = torch.zeros(nb, dtype=torch.uint8, device=device)
        self.err = torch.zeros(1, dtype=torch.int32, device=device)
        self.device = self.data.device
        self._index = self.data.get_device()
        self._args = (tokens, n_adapters, self.data.data_ptr(), nb, self.err.data_ptr())
        self.update(torch.full((tokens,), -1, dtype=torch.int32, device=self.device))

    def update(self, idx: torch.Tensor, stream=None) -> "LoraPlan":
        """Enqueued on the stream. An index past the adapters counts as none and sets bit 2 of ``err``."""
        if idx.dtype is not torch.int32 or not idx.is_contiguous() or idx.numel() != self.tokens or idx.get_device() != self._index:
            raise BsError(E_ARG, "lora_plan", "idx: one int32 for each token, contiguous, on the plan's device")
        _on(self._index, "lora_plan", lib.bs_lora_plan, idx.data_ptr() if self.tokens else None, *self._args, stream=stream)
        return self


class LoraAdapters:
    """The adapters of one or more projections, each a pool over ``n`` adapters:

    a[k]: bfloat16 [n, rank_max, cols_k] and b[k]: bfloat16 [n, rows_k, rank_max], contiguous; scales:
    float32 [n] or None (1); ranks: int32 [n] or None (rank_max), the rank rows that each adapter
    uses. The handle keeps the tensors and reads what stands in them at each call.

    forward(plan, xs, ys, bases, state): ys[k][t] = bases[k][t] + B_a (scale_a A_a xs[k][t]); bases
    None adds to ys in place, a None among them stands for 0; ys None leaves only the state behind.
    backward(plan, xs, dys, state, das, dbs, dxs, dx_bases, work): das and dbs (float32, as the
    pools) are written, or added to with accumulate; dxs[k] = dx_bases[k] + the adapters' part,
    where entries of dxs that are the same tensor receive the sum of their parts. dx_bases None: 0.
    xs and dys are bfloat16 [tokens, width], ys and dxs float32 or bfloat16, their bases of the same
    type; rows may be strided. Arguments of several projections are lists or tuples. Beside a coded
    projection, fw_gemv and fw_gemm take the adapters with the product (their ``adapters``).
    """

    def __init__(self, a, b, scales: torch.Tensor | None = None, ranks: torch.Tensor | None = None):
        a, b = list(a), list(b)
        bad = lambda msg: BsError(E_ARG, "lora", msg)  # noqa: E731
        if not a or len(a) != len(b):
            raise bad("one a and one b for each projection")
        self.n, self.rank_max = (a[0].shape[0], a[0].shape[1]) if a[0].dim() == 3 else (0, 0)
        self.device = a[0].device
        for x, y in zip(a, b):
            if x.dim() != 3 or y.dim() != 3 or x.shape[:2] != (self.n, self.rank_max) or y.shape[::2] != (self.n, self.rank_max):
                raise bad("a: [n, rank_max, cols], b: [n, rows, rank_max]")
            if any(t.dtype != torch.bfloat16 or not t.is_contiguous() or not t.is_cuda or t.device != self.device for t in (x, y)):
                raise bad("pools: contiguous bfloat16 CUDA tensors on one device")
        for t, dt in ((scales, torch.float32), (ranks, torch.int32)):
            if t is not None and (t.dtype != dt or t.numel() != self.n or not t.is_contiguous() or t.device != self.device):
                raise bad(f"scales float32 and ranks int32: one for each of {self.n} adapters")
        self.a, self.b, self.scales, self.ranks = a, b, scales, ranks
        self._n = len(a)
        self._index = a[0].get_device()
        self._fixed = [(x.data_ptr(), y.data_ptr(), y.shape[1], x.shape[2]) for x, y in zip(a, b)]
        self._ranks_at, self._scales_at = (t.data_ptr() if t is not None else None for t in (ranks, scales))
        self._array = LoraItem * self._n
        self._need = (-1, 0)  # the bytes of a state for the last batch's number of tokens

    def state(self, tokens: int) -> list:
        """Buffers for one batch: what forward leaves for backward, or backward's own workspace."""
        nb = lib.bs_lora_state_bytes(tokens, self.rank_max) if 0 <= tokens < 2 ** 32 else 0
        if nb == 0:
            raise BsError(E_ARG, "lora", "tokens up to 2^20, rank_max a multiple of 8 in 8..128")
        return [torch.empty(nb, dtype=torch.uint8, device=self.device) for _ in range(self._n)]

    def _rows(self, t, width, dtype, what, tokens):
        """(address, stride) of a [tokens, width] tensor of contiguous rows."""
        if t.dtype is dtype and t.shape == (tokens, width) and t.get_device() == self._index:
            if t.is_contiguous():
                return t.data_ptr(), width
            s0, s1 = t.stride()
            if s1 == 1:
                return t.data_ptr(), s0 if tokens > 1 else width
        raise BsError(E_ARG, "lora", f"{what}: [{tokens}, {width}] of {dtype}, rows contiguous, on the adapters' device")

    def _out(self, t, base, width, what, tokens):
        """(type, base, its stride, output, its stride); no output: zeros."""
        if t is None:
            return 0, 0, 0, 0, 0
        dt = t.dtype
        if dt not in _TYPES:
            raise BsError(E_ARG, "lora", f"{what}: float32 or bfloat16")
        p, s = self._rows(t, width, dt, what, tokens)
        if base is t:
            return _TYPES[dt], p, s, p, s
        if base is None:
            return _TYPES[dt], 0, 0, p, s
        bp, bs = self._rows(base, width, dt, what, tokens)
        return _TYPES[dt], bp, bs, p, s

    def _begin(self, plan, lists, states):
        if plan.n_adapters != self.n or plan._index != self._index:
            raise BsError(E_ARG, "lora", "the plan is of another set of adapters")
        n = self._n
        for v in lists:
            if len(v) != n:
                raise BsError(E_ARG, "lora", "one entry for each projection")
        known, index = self._need, self._index  # read once: another thread may serve another batch meanwhile
        if plan.tokens != known[0]:
            self._need = known = (plan.tokens, lib.bs_lora_state_bytes(plan.tokens, self.rank_max))
        need = known[1]
        for t in states:
            if t.numel() < need or t.dtype is not torch.uint8 or t.get_device() != index:
                raise BsError(E_SIZE, "lora", "a state is of another batch")
        return self._array(), LoraBatch(plan.tokens, self.n, self.rank_max, 0, self._ranks_at, self._scales_at, *plan._args[2:])

    def _forward_args(self, plan, xs, ys, bases, state, stream):
        """bs_lora_forward's arguments, and what has to outlive its call."""
        n, T = self._n, plan.tokens
        state = _made_on(stream, self._index, lambda: self.state(T)) if state is None else state
        ys = [None] * n if ys is None else ys
        bases = ys if bases is None else bases
        items, batch = self._begin(plan, (xs, ys, bases, state), state)
        pack, last = _LORA_ITEM.pack_into, None
        for k, (a, b, rows, cols) in enumerate(self._fixed):
            x = xs[k]
            if x is not last or cols != last_cols:  # q, k and v read one x
                xp, x_stride = self._rows(x, cols, torch.bfloat16, "x", T)
                last, last_cols = x, cols
            ty, bp, b_stride, y, y_stride = self._out(ys[k], bases[k], rows, "y", T)
            pack(items, 160 * k, a, b, rows, cols, ty, 0, xp, x_stride, state[k].data_ptr(), bp, b_stride, y, y_stride,
                 0, 0, 0, 0, 0, 0, 0, 0, 0)
        return n, items, ctypes.byref(batch), state, ys

    def forward(self, plan: LoraPlan, xs, ys=None, bases=None, state=None, stream=None):
        *args, _, ys = self._forward_args(plan, xs, ys, bases, state, stream)
        _on(self._index, "lora_forward", lib.bs_lora_forward, *args, stream=stream)
        return ys

    def backward(self, plan: LoraPlan, xs, dys, state, das, dbs, dxs=None, dx_bases=None, work=None, accumulate: bool = False,
                 stream=None):
        work = _made_on(stream, self._index, lambda: self.state(plan.tokens)) if work is None else work
        dxs = [None] * self._n if dxs is None else dxs
        dx_bases = [None] * self._n if dx_bases is None else dx_bases
        items, batch = self._begin(plan, (xs, dys, das, dbs, dxs, dx_bases, state, work), (*state, *work))
        T, pack, bf = plan.tokens, _LORA_ITEM.pack_into, torch.bfloat16
        for k, (a, b, rows, cols) in enumerate(self._fixed):
            for t, shape in ((das[k], self.a[k].shape), (dbs[k], self.b[k].shape)):
                if t.dtype is not torch.float32 or t.shape != shape or not t.is_contiguous() or t.get_device() != self._index:
                    raise BsError(E_ARG, "lora", "das and dbs: contiguous float32, of the pools' shapes")
            ty, base, bs_, dx, dxs_ = self._out(dxs[k], dx_bases[k], cols, "dx", T)
            pack(items, 160 * k, a, b, rows, cols, ty, 0, *self._rows(xs[k], cols, bf, "x", T), state[k].data_ptr(), 0, 0, 0, 0,
                 *self._rows(dys[k], rows, bf, "dy", T), work[k].data_ptr(), base, bs_, dx, dxs_, das[k].data_ptr(), dbs[k].data_ptr())
        _on(self._index, "lora_backward", lib.bs_lora_backward, self._n, items, ctypes.byref(batch),
            LORA_ACCUMULATE if accumulate else 0, stream=stream)
        return das, dbs, dxs


# ------------------------------------------------------------ AdamW over many tensors
ADAMW_BLOCK = 256  # elements that share a scale of the 8-bit moments


def _flat_list(ts, what: str, n: int, sizes=None, dtypes=None, device=None) -> list:
    """The list of n contiguous CUDA tensors on one device, checked."""
    ts = list(ts)
    if len(ts) != n:
        raise BsError(E_ARG, "adamw", f"{what}: one tensor for each parameter")
    for k, t in enumerate(ts):
        if not t.is_cuda or not t.is_contiguous() or (device is not None and t.device != device):
            raise BsError(E_ARG, "adamw", f"{what}[{k}]: a contiguous tensor on the parameters' device")
        if dtypes is not None and t.dtype not in dtypes:
            raise BsError(E_ARG, "adamw", f"{what}[{k}]: dtype {t.dtype}")
        if sizes is not None and t.numel() != sizes[k]:
            raise BsError(E_ARG, "adamw", f"{what}[{k}]: {t.numel()} elements, not {sizes[k]}")
    return ts


class AdamW:
    """AdamW over many tensors in one launch (bs_adamw), with the moments in 32 or in 8 bits.

    params and grads: lists of contiguous CUDA tensors (float32 or bfloat16, mixed as they come);
    the handle keeps both, and step() reads the gradients that stand in the grads' buffers then.
    masters: float32 copies of the parameters, in which the step is taken (else a bfloat16 parameter
    is rounded to nearest each step). weight_decay: a number, or one for each tensor.
    states: existing moments to go on with, (exp_avgs, exp_avg_sqs) in 32 bits, or
    ((codes, scales), (codes, scales)) in 8 bits, each a list; they are updated in place. step: the
    steps already done. clip: the factor on gradients where step() computes no norm (nor grad_norm() has
    since the last step).

    The learning rate, the factor, the step count and the norm live on the device (``ctl``): set
    ``lr`` and ``clip`` by attribute, read ``norm`` and ``steps`` as device tensors; a captured step
    sees new values. ``clip`` reads as the factor that was set, or that the last norm or step had; setting it
    replaces a norm's that no step has used yet. A norm, and the skip of a step whose norm is not finite,
    are for that one step.
    """

    def __init__(self, params, grads, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay=0.01,
                 bits: int = 32, masters=None, seed: int = 0, step: int = 0, clip: float = 1.0, states=None, _ctl=None, _family=None):
        params = list(params)
        if not torch.cuda.is_available():
            raise BsError(E_UNSUPPORTED, "adamw", "no CUDA device")
        if not params:
            raise BsError(E_ARG, "adamw", "no parameters")
        if bits not in (8, 32):
            raise BsError(E_ARG, "adamw", "bits: 8 or 32")
        n, dev = len(params), params[0].device
        sizes = [p.numel() for p in params]
        both = (torch.float32, torch.bfloat16)
        self.params = _flat_list(params, "params", n, None, both, dev)
        self.grads = _flat_list(grads, "grads", n, sizes, both, dev)
        self.masters = None if masters is None else _flat_list(masters, "masters", n, sizes, (torch.float32,), dev)
        self.device, self.bits = dev, bits
        blocks = [-(-k // ADAMW_BLOCK) for k in sizes]
        decay = list(weight_decay) if isinstance(weight_decay, (list, tuple)) else [weight_decay] * n
        if len(decay) != n:
            raise BsError(E_ARG, "adamw", "weight_decay: one for each parameter")
        if states is None:
            z = lambda dt, of: [torch.zeros(k, dtype=dt, device=dev) for k in of]  # noqa: E731
            states = ((z(torch.float32, sizes), z(torch.float32, sizes)) if bits == 32 else
                      tuple((z(torch.uint8, sizes), z(torch.float32, blocks)) for _ in range(2)))
        if not params[0].is_cuda:
            raise BsError(E_ARG, "adamw", "params: CUDA tensors")
        if bits == 32:
            self.exp_avg, self.exp_avg_sq = (_flat_list(v, "states", n, sizes, (torch.float32,), dev) for v in states)
            self.exp_avg_scale = self.exp_avg_sq_scale = None
        else:
            (m, ms), (v, vs) = states
            self.exp_avg, self.exp_avg_sq = (_flat_list(c, "states", n, sizes, (torch.uint8,), dev) for c in (m, v))
            self.exp_avg_scale, self.exp_avg_sq_scale = (_flat_list(c, "states", n, blocks, (torch.float32,), dev) for c in (ms, vs))
        # what a step writes: (first byte, behind the last, (which buffer, of which parameter))
        spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), (i, k)) for i, ts in enumerate(
            (self.params, self.masters, self.exp_avg, self.exp_avg_sq, self.exp_avg_scale, self.exp_avg_sq_scale))
            if ts is not None for k, t in enumerate(ts) if t.numel())
        if any(a[1] > b[0] for a, b in zip(spans, spans[1:])):
            raise BsError(E_ARG, "adamw", "parameters, masters and moments must not overlap")
        # a step into a twin reads one's and writes the other's: they may share a whole buffer, which is then
        # updated in place, but not overlap otherwise
        self._spans, self._family = spans, _family if _family is not None else weakref.WeakSet()
        for other in self._family:
            both = sorted(spans + other._spans)  # two runs in order: a merge
            if any(a[1] > b[0] and a != b for a, b in zip(both, both[1:])):
                raise BsError(E_ARG, "adamw", "a twin's parameters, masters and moments must not overlap its handle's")
        for g in self.grads:  # a gradient may be read by several items, but not written by any
            lo, hi = g.data_ptr(), g.data_ptr() + g.numel() * g.element_size()
            at = bisect.bisect_left(spans, (hi,))  # the first that begins at or behind the gradient's end
            if g.numel() and at and spans[at - 1][1] > lo:
                raise BsError(E_ARG, "adamw", "gradients must not overlap what the step writes")
        self._items = (AdamWItem * n)()
        ptr = lambda ts, k: ts[k].data_ptr() if ts is not None and sizes[k] else None  # noqa: E731
        for k in range(n):
            it = self._items[k]
            it.d_param, it.d_grad, it.d_master = ptr(self.params, k), ptr(self.grads, k), ptr(self.masters, k)
            it.d_m, it.d_v = ptr(self.exp_avg, k), ptr(self.exp_avg_sq, k)
            it.d_m_scale, it.d_v_scale = ptr(self.exp_avg_scale, k), ptr(self.exp_avg_sq_scale, k)
            it.n, it.param_type, it.grad_type = sizes[k], _TYPES[self.params[k].dtype], _TYPES[self.grads[k].dtype]
            it.weight_decay = decay[k]
        self._n, self._sizes, self._index = n, sizes, self.params[0].get_device()
        self._prm = self._numbered = AdamWParams(betas[0], betas[1], eps, bits, 0, seed & (2 ** 64 - 1))
        self.ctl = torch.zeros(8, dtype=torch.int32, device=dev) if _ctl is None else _ctl
        f = self.ctl.view(torch.float32)
        self._lr, self._clip, self.norm, self.steps = f[0], f[1], f[4], self.ctl[2]
        self._clips = f[1:7:5]  # clip and own_clip
        if _ctl is None:
            self.ctl[7:].fill_(1)  # once
            self.lr, self.clip = lr, clip
            self.steps.fill_(step)
        self._scratch = torch.empty(max(8, lib.bs_grad_norm_scratch_bytes(n, self._items)), dtype=torch.uint8, device=dev)
        self._at = (self.ctl.data_ptr(), self._scratch.data_ptr(), self._scratch.numel())
        self._family.add(self)

    @property
    def lr(self):
        return self._lr

    @lr.setter
    def lr(self, v):
        self._lr.fill_(v)

    @property
    def clip(self):
        return self._clip

    @clip.setter
    def clip(self, v):
        self._clips.fill_(v)

    def grad_norm(self, max_norm: float = float("inf"), stream=None) -> torch.Tensor:
        """bs_grad_norm: the norm of all gradients as a device scalar; sets the factor of the next
        step to min(1, max_norm / (norm + 1e-6)), or marks it to be left out if the norm is not finite."""
        _on(self._index, "grad_norm", lib.bs_grad_norm, self._n, self._items, max_norm, *self._at, stream=stream)
        return self.norm

    def twin(self, params=None, masters=None, states=None) -> "AdamW":
        """A second set of parameters, masters and moments (new tensors where none are given) for the
        same gradients and the same ctl, which must not overlap this handle's in part (one that is the same
        tensor is updated in place): step(into=twin) leaves this handle's as they are, to be
        coded or compared, and the twin's next step, into this one, goes on from there. A step that is
        left out (its norm was not finite) leaves the twin with this handle's values."""
        new = lambda ts, given: (None if ts is None else list(given) if given is not None else [torch.empty_like(t) for t in ts])  # noqa: E731
        if states is None:
            m, v, ms, vs = (new(ts, None) for ts in (self.exp_avg, self.exp_avg_sq, self.exp_avg_scale, self.exp_avg_sq_scale))
            states = (m, v) if self.bits == 32 else ((m, ms), (v, vs))
        return AdamW(new(self.params, params), self.grads, betas=(self._prm.beta1, self._prm.beta2), eps=self._prm.eps,
                  weight_decay=[it.weight_decay for it in self._items], bits=self.bits, masters=new(self.masters, masters),
                  seed=self._prm.seed, states=states, _ctl=self.ctl, _family=self._family)

    def step(self, max_norm: float | None = None, into: "AdamW | None" = None, number: int = 0, stream=None):
        """One step, enqueued on the stream; with max_norm, grad_norm(max_norm) first. into: a twin
        that receives the results, while this handle's tensors stay as they are. number: the step's
        number (from 1), instead of one more than the last one's."""
        if into is not None and into.ctl is not self.ctl:
            raise BsError(E_ARG, "adamw", "into: a twin of this handle")
        if not 0 <= number < 2 ** 31:
            raise BsError(E_ARG, "adamw", "number: 1 .. 2^31 - 1, or 0")
        if max_norm is not None:
            self.grad_norm(max_norm, stream)
        numbered = self._numbered  # never changed once made: another thread's call may be reading it
        if numbered.step != number:
            p = self._prm
            self._numbered = numbered = AdamWParams(p.beta1, p.beta2, p.eps, p.bits, number, p.seed)
        _on(self._index, "adamw", lib.bs_adamw, self._n, self._items, into._items if into is not None else None,
            ctypes.byref(numbered), self._at[0], stream=stream)

    def read_states(self, ms=None, vs=None, stream=None):
        """The moments as float32 lists, (exp_avgs, exp_avg_sqs). 32-bit moments are returned as they
        stand; 8-bit ones are decoded (bs_adamw_read_states) into ms and vs, or into new tensors of the stream."""
        if self.bits == 32:
            return self.exp_avg, self.exp_avg_sq
        new = lambda: [torch.empty(k, dtype=torch.float32, device=self.device) for k in self._sizes]  # noqa: E731
        ms, vs = (_made_on(stream, self._index, new) if t is None else list(t) for t in (ms, vs))
        T, n, every = torch.Tensor, self._n, [*ms, *vs]  # one look at a time at all tensors: several hundred are usual
        if len(ms) != n or len(vs) != n:
            raise BsError(E_ARG, "adamw", "read_states: one tensor for each parameter")
        if not (list(map(T.numel, every)) == self._sizes * 2 and set(map(T.dtype.__get__, every)) == {torch.float32} and
                set(map(T.get_device, every)) == {self._index} and all(map(T.is_contiguous, every))):
            raise BsError(E_ARG, "adamw", "read_states: a contiguous float32 tensor of each parameter's size")
        at = array.array("Q", map(T.data_ptr, every))
        pm = at.buffer_info()[0]
        pv = pm + 8 * n
        _on(self._index, "adamw_read_states", lib.bs_adamw_read_states, self._n, self._items, pm, pv, stream=stream)
        return ms, vs
