"""Thin Python binding of ``liblh.so`` (the C ABI declared in ``include/lh.h``).

Only argument marshalling happens here: every step of the layer runs in the library's CUDA kernels.  PyTorch
provides device memory and the current stream.  Function names match the C entry points.  Importing this module
raises when the library has not been built; there is no fallback path.
"""

from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass, fields

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "liblh.so")

LH_OK = 0
LH_ERR_INVALID_ARG = 1
LH_ERR_UNSUPPORTED = 2
LH_ERR_CUDA = 3
LH_ERR_TIMEOUT = 4
LH_ERR_WORKSPACE = 5
LH_ERR_RANGE = 6

LH_EXPAND_CHILDREN = 1


class LhParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "H", "N", "d", "L", "p", "k", "C", "flags")]


class LhCtxLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint64) for n in ("qg", "kg", "vg", "og", "lse", "idx_g", "slot", "total")]


class LhKernelTime(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 32), ("launches", ctypes.c_int32), ("ms", ctypes.c_double)]


LH_BF16 = 0
LH_FP16 = 1
LH_MAX_BUCKETS = 128


class LhAttnParams(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("B", "Hq", "Hkv", "Sq", "Skv", "d", "dtype", "causal")] +
                [(n, ctypes.c_float) for n in ("scale", "softcap")] +
                [(n, ctypes.c_int32) for n in ("buckets", "max_distance", "bidirectional")])


class LighthouseError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {error_string(status)} (status {status})")


_P = ctypes.POINTER(LhParams)
_vp = ctypes.c_void_p
_SIGS = {
    "lh_error_string": (ctypes.c_char_p, [ctypes.c_int]),
    "lh_validate": (ctypes.c_int, [_P]),
    "lh_S": (ctypes.c_int64, [_P]),
    "lh_level_size": (ctypes.c_int64, [_P, ctypes.c_int]),
    "lh_level_offset": (ctypes.c_int64, [_P, ctypes.c_int]),
    "lh_pyramid_rows": (ctypes.c_int64, [_P]),
    "lh_score_rows": (ctypes.c_int64, [_P]),
    "lh_slot_rows": (ctypes.c_int64, [_P]),
    "lh_ctx_bytes": (ctypes.c_size_t, [_P]),
    "lh_ctx_layout": (ctypes.c_int, [_P, ctypes.POINTER(LhCtxLayout)]),
    "lh_workspace_bytes": (ctypes.c_size_t, [_P]),
    "lh_pool": (ctypes.c_int, [_P, _vp, _vp, _vp]),
    "lh_score_topk": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "lh_gather": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "lh_attend": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp, _vp, _vp]),
    "lh_scatter": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp]),
    "lh_forward": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "lh_backward": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "lh_scatter_bwd": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp]),
    "lh_attend_bwd": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "lh_get_status": (ctypes.c_int, [_vp]),
    "lh_set_wait_limit_ns": (ctypes.c_int, [ctypes.c_uint64]),
    "lh_score_topk_static": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp, _vp, _vp]),
    "lh_profile_enable": (ctypes.c_int, [ctypes.c_int]),
    "lh_profile_read": (ctypes.c_int, [ctypes.POINTER(LhKernelTime), ctypes.c_int]),
    "lh_step_host_bytes": (ctypes.c_size_t, [_P, ctypes.c_int]),
    "lh_step_host": (ctypes.c_int, [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_int, _vp, ctypes.c_size_t, _vp,
                                    _vp, _vp]),
    "lh_attn_validate": (ctypes.c_int, [_vp]),
    "lh_attn_workspace_bytes": (ctypes.c_size_t, [_vp, ctypes.c_int]),
    "lh_attn_bucket_starts": (ctypes.c_int, [_vp, _vp]),
    "lh_attn_forward": (ctypes.c_int, [_vp] * 9 + [ctypes.c_size_t, _vp]),
    "lh_attn_backward": (ctypes.c_int, [_vp] * 14 + [ctypes.c_size_t, _vp]),
}


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m hierarchical_sparse_attention_avg_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load()


def library() -> ctypes.CDLL:
    return _lib


# ------------------------------------------------------------------------------------------------------------
# Parameters and host-only queries
# ------------------------------------------------------------------------------------------------------------

@dataclass(frozen=True)
class Params:
    B: int
    H: int
    N: int
    d: int
    L: int
    p: int
    k: int
    C: int
    expand: bool = False  # LH_EXPAND_CHILDREN

    def c(self) -> LhParams:
        return LhParams(self.B, self.H, self.N, self.d, self.L, self.p, self.k, self.C,
                        LH_EXPAND_CHILDREN if self.expand else 0)


def error_string(status: int) -> str:
    return _lib.lh_error_string(status).decode()


def _check(rc: int, where: str) -> None:
    if rc != LH_OK:
        raise LighthouseError(rc, where)


def lh_validate(P: Params) -> int:
    return _lib.lh_validate(ctypes.byref(P.c()))


def lh_S(P: Params) -> int:
    return _lib.lh_S(ctypes.byref(P.c()))


def lh_level_size(P: Params, level: int) -> int:
    return _lib.lh_level_size(ctypes.byref(P.c()), level)


def lh_level_offset(P: Params, level: int) -> int:
    return _lib.lh_level_offset(ctypes.byref(P.c()), level)


def lh_pyramid_rows(P: Params) -> int:
    return _lib.lh_pyramid_rows(ctypes.byref(P.c()))


def lh_score_rows(P: Params) -> int:
    return _lib.lh_score_rows(ctypes.byref(P.c()))


def lh_slot_rows(P: Params) -> int:
    return _lib.lh_slot_rows(ctypes.byref(P.c()))


def lh_ctx_bytes(P: Params) -> int:
    return _lib.lh_ctx_bytes(ctypes.byref(P.c()))


def lh_workspace_bytes(P: Params) -> int:
    return _lib.lh_workspace_bytes(ctypes.byref(P.c()))


def lh_ctx_layout(P: Params) -> LhCtxLayout:
    out = LhCtxLayout()
    _check(_lib.lh_ctx_layout(ctypes.byref(P.c()), ctypes.byref(out)), "lh_ctx_layout")
    return out


# ------------------------------------------------------------------------------------------------------------
# Device entry points (torch tensors in, torch tensors out)
# ------------------------------------------------------------------------------------------------------------

def _ptr(t) -> int | None:
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("tensors must be contiguous CUDA tensors")
    return t.data_ptr()


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _valid(P: Params, where: str) -> None:
    """Raise the library's own status for invalid or unsupported parameters before sizing any buffer."""
    _check(lh_validate(P), where)


def _typed(t, shape, name, dtype=torch.bfloat16):
    if t.dtype != dtype or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")


def _bf16(t, shape, name):
    _typed(t, shape, name, torch.bfloat16)


def new_workspace(P: Params, device) -> torch.Tensor:
    return torch.empty(lh_workspace_bytes(P), dtype=torch.uint8, device=device)


def new_ctx(P: Params, device) -> torch.Tensor:
    return torch.empty(lh_ctx_bytes(P), dtype=torch.uint8, device=device)


def ctx_views(P: Params, ctx: torch.Tensor) -> dict:
    """Typed views of the saved-context buffer written by ``lh_forward``."""
    lay = lh_ctx_layout(P)
    S, rows = lh_S(P), P.B * P.H

    def view(off, n, dtype, shape):
        nbytes = n * torch.tensor([], dtype=dtype).element_size()
        return ctx[off: off + nbytes].view(dtype).view(*shape)

    g = (P.B, P.H, S, P.d)
    return dict(qg=view(lay.qg, rows * S * P.d, torch.float16, g), kg=view(lay.kg, rows * S * P.d, torch.float16, g),
                vg=view(lay.vg, rows * S * P.d, torch.float16, g), og=view(lay.og, rows * S * P.d, torch.float32, g),
                lse=view(lay.lse, rows * S, torch.float32, (P.B, P.H, S)),
                idx_g=view(lay.idx_g, rows * S, torch.int32, (P.B, P.H, S)),
                slot=view(lay.slot, rows * lh_slot_rows(P), torch.int32, (P.B, P.H, lh_slot_rows(P))))


def lh_pool(P: Params, x, pyr=None):
    _valid(P, "lh_pool")
    _bf16(x, (P.B, P.H, P.N, P.d), "x")
    if pyr is None:
        pyr = torch.empty((P.B, P.H, lh_pyramid_rows(P), P.d), dtype=torch.bfloat16, device=x.device)
    _check(_lib.lh_pool(ctypes.byref(P.c()), _ptr(x), _ptr(pyr), _stream(x.device)), "lh_pool")
    return pyr


def lh_score_topk(P: Params, k, scores_in=None, scores_out=None, idx_g=None, slot=None, ws=None):
    _valid(P, "lh_score_topk")
    dev = k.device
    _bf16(k, (P.B, P.H, P.N, P.d), "k")
    if idx_g is None:
        idx_g = torch.empty((P.B, P.H, lh_S(P)), dtype=torch.int32, device=dev)
    if slot is None:
        slot = torch.empty((P.B, P.H, lh_slot_rows(P)), dtype=torch.int32, device=dev)
    if ws is None:
        ws = new_workspace(P, dev)
    for t in (scores_in, scores_out):
        if t is not None and (t.dtype != torch.float32 or tuple(t.shape) != (P.B, P.H, lh_score_rows(P))):
            raise ValueError("scores must be fp32 [B, H, lh_score_rows]")
    rc = _lib.lh_score_topk(ctypes.byref(P.c()), _ptr(k), _ptr(scores_in), _ptr(scores_out), _ptr(idx_g), _ptr(slot),
                            _ptr(ws), ws.numel(), _stream(dev))
    _check(rc, "lh_score_topk")
    return idx_g, slot


def lh_gather(P: Params, q, k, v, q_pyr, k_pyr, v_pyr, idx_g, out=None):
    _valid(P, "lh_gather")
    dev = q.device
    S = lh_S(P)
    if out is None:
        out = tuple(torch.empty((P.B, P.H, S, P.d), dtype=torch.float16, device=dev) for _ in range(3))
    qg, kg, vg = out
    rc = _lib.lh_gather(ctypes.byref(P.c()), _ptr(q), _ptr(k), _ptr(v), _ptr(q_pyr), _ptr(k_pyr), _ptr(v_pyr),
                        _ptr(idx_g), _ptr(qg), _ptr(kg), _ptr(vg), _stream(dev))
    _check(rc, "lh_gather")
    return qg, kg, vg


def lh_attend(P: Params, qg, kg, vg, og=None, lse=None):
    _valid(P, "lh_attend")
    dev = qg.device
    S = lh_S(P)
    for t, n in ((qg, "qg"), (kg, "kg"), (vg, "vg")):
        _typed(t, (P.B, P.H, S, P.d), n, torch.float16)
    if og is None:
        og = torch.empty(qg.shape, dtype=torch.float32, device=dev)
    if lse is None:
        lse = torch.empty((P.B, P.H, S), dtype=torch.float32, device=dev)
    _check(_lib.lh_attend(ctypes.byref(P.c()), _ptr(qg), _ptr(kg), _ptr(vg), _ptr(og), _ptr(lse), _stream(dev)),
           "lh_attend")
    return og, lse


def lh_scatter(P: Params, og, slot, o=None):
    _valid(P, "lh_scatter")
    dev = og.device
    if o is None:
        o = torch.empty((P.B, P.H, P.N, P.d), dtype=torch.bfloat16, device=dev)
    _check(_lib.lh_scatter(ctypes.byref(P.c()), _ptr(og), _ptr(slot), _ptr(o), _stream(dev)), "lh_scatter")
    return o


def lh_forward(P: Params, q, k, v, o=None, ctx=None, ws=None):
    _valid(P, "lh_forward")
    dev = q.device
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _bf16(t, (P.B, P.H, P.N, P.d), n)
    if o is None:
        o = torch.empty_like(q)
    if ctx is None:
        ctx = new_ctx(P, dev)
    if ws is None:
        ws = new_workspace(P, dev)
    rc = _lib.lh_forward(ctypes.byref(P.c()), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(ctx), _ptr(ws), ws.numel(),
                         _stream(dev))
    _check(rc, "lh_forward")
    return o, ctx


def lh_backward(P: Params, dout, ctx, dq=None, dk=None, dv=None, ws=None):
    _valid(P, "lh_backward")
    dev = dout.device
    _bf16(dout, (P.B, P.H, P.N, P.d), "dout")
    dq = torch.empty_like(dout) if dq is None else dq
    dk = torch.empty_like(dout) if dk is None else dk
    dv = torch.empty_like(dout) if dv is None else dv
    if ws is None:
        ws = new_workspace(P, dev)
    rc = _lib.lh_backward(ctypes.byref(P.c()), _ptr(dout), _ptr(ctx), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws),
                          ws.numel(), _stream(dev))
    _check(rc, "lh_backward")
    return dq, dk, dv


# ------------------------------------------------------------------------------------------------------------
# Host-resident step (host tensors in, host tensors out; the copies are pipelined inside the library)
# ------------------------------------------------------------------------------------------------------------

_copy_streams: dict = {}


def default_heads_per_chunk(P: Params) -> int:
    """The largest divisor of H that still gives at least sixteen chunks per batch row (one head when H < 16): the
    first chunk's host-to-device copy and the last chunk's device-to-host copy are not overlapped, so small chunks
    pay less for them."""
    best = 1
    for hc in range(1, P.H + 1):
        if P.H % hc == 0 and P.H // hc >= 16:
            best = hc
    return best


def lh_step_host_bytes(P: Params, heads_per_chunk: int) -> int:
    return _lib.lh_step_host_bytes(ctypes.byref(P.c()), int(heads_per_chunk))


def _host_bf16(t, shape, name):
    _typed(t, shape, name, torch.bfloat16)
    if t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous host (CPU) tensor")
    return t.data_ptr()


def lh_step_host(P: Params, q, k, v, dout, o=None, dq=None, dk=None, dv=None, heads_per_chunk=None, dev_buf=None,
                 device=None):
    """lh_forward + lh_backward on HOST bf16 tensors [B,H,N,d] (page-locked for overlap), returning host (o, dq, dk,
    dv).  Runs on `device` (default: the current CUDA device): the compute on its current stream, the copies on two
    streams of this module; returns once everything is enqueued (synchronise the current stream before reading the
    outputs, and keep the input tensors alive until then: the library copies from them asynchronously)."""
    _valid(P, "lh_step_host")
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    hc = default_heads_per_chunk(P) if heads_per_chunk is None else int(heads_per_chunk)
    shape = (P.B, P.H, P.N, P.d)
    ins = [_host_bf16(t, shape, n) for t, n in ((q, "q"), (k, "k"), (v, "v"), (dout, "dout"))]
    outs = []
    for t, n in ((o, "o"), (dq, "dq"), (dk, "dk"), (dv, "dv")):
        outs.append(torch.empty(shape, dtype=torch.bfloat16, pin_memory=True) if t is None else t)
    out_ptrs = [_host_bf16(t, shape, n) for t, n in zip(outs, ("o", "dq", "dk", "dv"))]
    need = lh_step_host_bytes(P, hc)
    if need == 0:
        raise LighthouseError(LH_ERR_INVALID_ARG, "lh_step_host_bytes")
    if dev_buf is None:
        dev_buf = torch.empty(need, dtype=torch.uint8, device=dev)
    if dev_buf.device != dev:
        raise ValueError("dev_buf must live on the step's device")
    key = dev.index
    if key not in _copy_streams:
        _copy_streams[key] = (torch.cuda.Stream(dev), torch.cuda.Stream(dev))
    h2d, d2h = _copy_streams[key]
    with torch.cuda.device(dev):
        rc = _lib.lh_step_host(ctypes.byref(P.c()), *ins, *out_ptrs, hc, _ptr(dev_buf), dev_buf.numel(),
                               torch.cuda.current_stream(dev).cuda_stream, h2d.cuda_stream, d2h.cuda_stream)
    _check(rc, "lh_step_host")
    return tuple(outs)


def lh_scatter_bwd(P: Params, dout, idx_g, dog=None):
    _valid(P, "lh_scatter_bwd")
    dev = dout.device
    if dog is None:
        dog = torch.empty((P.B, P.H, lh_S(P), P.d), dtype=torch.float32, device=dev)
    _check(_lib.lh_scatter_bwd(ctypes.byref(P.c()), _ptr(dout), _ptr(idx_g), _ptr(dog), _stream(dev)),
           "lh_scatter_bwd")
    return dog


def lh_attend_bwd(P: Params, qg, kg, vg, og, lse, dog, ws=None):
    _valid(P, "lh_attend_bwd")
    dev = qg.device
    S = lh_S(P)
    for t, n in ((qg, "qg"), (kg, "kg"), (vg, "vg")):
        _typed(t, (P.B, P.H, S, P.d), n, torch.float16)
    for t, n in ((og, "og"), (dog, "dog")):
        _typed(t, (P.B, P.H, S, P.d), n, torch.float32)
    dqg = torch.empty(qg.shape, dtype=torch.float32, device=dev)
    dkg = torch.empty(qg.shape, dtype=torch.float32, device=dev)
    dvg = torch.empty(qg.shape, dtype=torch.float32, device=dev)
    if ws is None:
        ws = new_workspace(P, dev)
    rc = _lib.lh_attend_bwd(ctypes.byref(P.c()), _ptr(qg), _ptr(kg), _ptr(vg), _ptr(og), _ptr(lse), _ptr(dog),
                            _ptr(dqg), _ptr(dkg), _ptr(dvg), _ptr(ws), ws.numel(), _stream(dev))
    _check(rc, "lh_attend_bwd")
    return dqg, dkg, dvg


def lh_get_status(device=None) -> int:
    dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
    return _lib.lh_get_status(_stream(dev))


def lh_set_wait_limit_ns(ns: int, device=None) -> None:
    """Bound on every device-side wait of later launches on ``device`` (0 restores the default of 2 s)."""
    dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.device(dev):
        _check(_lib.lh_set_wait_limit_ns(int(ns)), "lh_set_wait_limit_ns")


def lh_profile_enable(on: bool = True) -> None:
    _check(_lib.lh_profile_enable(1 if on else 0), "lh_profile_enable")


def lh_profile_read() -> dict:
    """``{kernel name: (launches, summed device ms)}`` since the last read; clears the record."""
    buf = (LhKernelTime * 64)()
    n = _lib.lh_profile_read(buf, 64)
    if n < 0:
        raise LighthouseError(-n, "lh_profile_read")
    return {buf[i].name.decode(): (int(buf[i].launches), float(buf[i].ms)) for i in range(n)}


LH_STATIC_SCRATCH_BYTES = 16 << 20


def lh_score_topk_static(P: Params, k, scores_in=None, scores_out=None, idx_g=None, slot=None):
    """``lh_score_topk`` without a caller workspace: the library's fixed device scratch array is used instead
    (for callers that cannot allocate device memory where they select).  Output buffers are created here only
    for convenience when not given; the library call itself allocates nothing."""
    _valid(P, "lh_score_topk_static")
    dev = k.device
    _bf16(k, (P.B, P.H, P.N, P.d), "k")
    if idx_g is None:
        idx_g = torch.empty((P.B, P.H, lh_S(P)), dtype=torch.int32, device=dev)
    if slot is None:
        slot = torch.empty((P.B, P.H, lh_slot_rows(P)), dtype=torch.int32, device=dev)
    rc = _lib.lh_score_topk_static(ctypes.byref(P.c()), _ptr(k), _ptr(scores_in), _ptr(scores_out), _ptr(idx_g),
                                   _ptr(slot), _stream(dev))
    _check(rc, "lh_score_topk_static")
    return idx_g, slot


# ------------------------------------------------------------------------------------------------------------
# Dense-stage attention (capped scores, distance biases, document and prefix masks; lengths over a cache)
# ------------------------------------------------------------------------------------------------------------

_ATTN_DTYPES = {torch.bfloat16: LH_BF16, torch.float16: LH_FP16}


@dataclass(frozen=True)
class AttnParams:
    """Sizes and score function of ``lh_attn_forward`` / ``lh_attn_backward`` (see ``lh_attn_params`` in
    ``include/lh.h``).  ``scale`` None is d**-0.5."""

    B: int
    Hq: int
    Hkv: int
    Sq: int
    Skv: int
    d: int
    dtype: torch.dtype = torch.bfloat16
    causal: bool = True
    scale: float | None = None
    softcap: float = 0.0
    buckets: int = 0
    max_distance: int = 0
    bidirectional: bool = False

    def __post_init__(self):
        if self.dtype not in _ATTN_DTYPES:
            raise ValueError(f"dtype: expected torch.bfloat16 or torch.float16, got {self.dtype}")
        for n in ("B", "Hq", "Hkv", "Sq", "Skv", "d", "buckets", "max_distance"):
            if not -2 ** 31 <= getattr(self, n) < 2 ** 31:  # (ctypes would drop the upper bits)
                raise ValueError(f"{n}: expected a 32-bit number, got {getattr(self, n)}")
        c = self.c()
        object.__setattr__(self, "_c", c)  # read by every call, built once
        object.__setattr__(self, "_ref", ctypes.addressof(c))
        object.__setattr__(self, "_status", _lib.lh_attn_validate(self._ref))
        object.__setattr__(self, "_qs", (self.B, self.Hq, self.Sq, self.d))
        object.__setattr__(self, "_ks", (self.B, self.Hkv, self.Skv, self.d))

    def c(self) -> LhAttnParams:
        scale = (self.d ** -0.5 if self.d > 0 else 1.0) if self.scale is None else self.scale
        return LhAttnParams(self.B, self.Hq, self.Hkv, self.Sq, self.Skv, self.d, _ATTN_DTYPES[self.dtype],
                            1 if self.causal else 0, scale, self.softcap, self.buckets, self.max_distance,
                            1 if self.bidirectional else 0)

    def __reduce__(self):
        """Copies and pickles are made anew from the fields: ``_ref`` is the address of this object's own struct."""
        return type(self), tuple(getattr(self, f.name) for f in fields(self))


def lh_attn_validate(P: AttnParams) -> int:
    return P._status


def lh_attn_workspace_bytes(P: AttnParams, backward: bool = False) -> int:
    return _lib.lh_attn_workspace_bytes(P._ref, 1 if backward else 0)


def new_attn_workspace(P: AttnParams, device, backward: bool = False) -> torch.Tensor:
    """Scratch for calls with ``P``; one at a time may use it (calls on one stream may share it)."""
    _check(P._status, "lh_attn_workspace_bytes")
    return torch.empty(lh_attn_workspace_bytes(P, backward), dtype=torch.uint8, device=device)


def lh_attn_bucket_starts(P: AttnParams) -> list:
    """First distance of each bucket of one direction."""
    buf = (ctypes.c_int32 * LH_MAX_BUCKETS)()
    n = _lib.lh_attn_bucket_starts(P._ref, buf)
    if n < 0:
        raise LighthouseError(LH_ERR_INVALID_ARG, "lh_attn_bucket_starts")
    return list(buf[:n])


_pack_rows = struct.Struct("4q").pack  # an lh_tensor
_pack_mods = struct.Struct("5Q").pack  # an lh_attn_mods


def _rows(t, shape, dtype, device, name) -> bytes:
    """Descriptor of a [B, H, S, d] tensor with any layout the library takes: unit feature stride, the others multiples
    of 8 elements."""
    if t.dtype is not dtype or t.shape != shape or t.device != device:
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)} on {device}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    sb, sh, ss, sd = t.stride()
    if sd != 1 or (sb | sh | ss) & 7 or sb <= 0 or sh <= 0 or ss <= 0:
        B, H, S, d = shape  # (a dimension of one may have any stride)
        if (sd != 1 and d > 1) or any(n > 1 and (x <= 0 or x & 7) for n, x in ((B, sb), (H, sh), (S, ss))):
            raise ValueError(f"{name}: features must be contiguous and the other strides positive multiples of 8, got "
                             f"{t.stride()}")
    return _pack_rows(t.data_ptr(), sb, sh, ss)


def _vec(t, shape, dtype, device, name) -> int:
    if t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} {tuple(shape)} on {device}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _attn_mods(P: AttnParams, dev, slopes, table, docs, prefix, kv_len) -> bytes:
    return _pack_mods(0 if slopes is None else _vec(slopes, (P.Hq,), torch.float32, dev, "slopes"),
                      0 if table is None else _vec(table, (P.Hq, P.buckets), P.dtype, dev, "table"),
                      0 if docs is None else _vec(docs, (P.B, P.Skv), torch.int32, dev, "docs"),
                      0 if prefix is None else _vec(prefix, (P.B,), torch.int32, dev, "prefix"),
                      0 if kv_len is None else _vec(kv_len, (P.B,), torch.int32, dev, "kv_len"))


def _attn_ws(P: AttnParams, ws, dev, backward, where):
    if dev.type != "cuda":
        raise ValueError(f"{where}: expected CUDA tensors")
    if ws is None:
        return new_attn_workspace(P, dev, backward)
    if ws.device != dev or ws.dtype is not torch.uint8 or not ws.is_contiguous():
        raise ValueError(f"ws: expected a contiguous uint8 tensor on {dev}")
    return ws


# the current stream's handle without a Stream object around it (these calls are as short as a few microseconds)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _on_device(dev, fn, *args) -> int:
    """The call with the tensors' device current, on its current stream."""
    index = dev.index
    if index == torch.cuda.current_device():
        return fn(*args, _raw_stream(index))
    with torch.cuda.device(dev):
        return fn(*args, _raw_stream(index))


def lh_attn_forward(P: AttnParams, q, k, v, slopes=None, table=None, docs=None, prefix=None, kv_len=None, o=None,
                    lse=None, low=None, ws=None):
    """Dense attention ``(o, lse)`` of ``q`` [B, Hq, Sq, d] over ``k``, ``v`` [B, Hkv, Skv, d]; the rows are the last
    ``Sq`` of each entry's ``kv_len`` positions.  ``slopes`` fp32 [Hq]; ``table`` [Hq, buckets] (dtype of q); ``docs``
    int32 [B, Skv]; ``prefix``, ``kv_len`` int32 [B].  ``low`` (like ``o``): receives what o's rounding dropped; handed to
    ``lh_attn_backward`` it makes the gradients about twice as exact."""
    if P._status:
        _check(P._status, "lh_attn_forward")
    dev = q.device
    ws = _attn_ws(P, ws, dev, False, "lh_attn_forward")
    qs, ks = P._qs, P._ks
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty_strided(qs[:3], (P.Hq * P.Sq, P.Sq, 1), dtype=torch.float32, device=dev)
    dt = P.dtype
    rc = _on_device(dev, _lib.lh_attn_forward, P._ref, _attn_mods(P, dev, slopes, table, docs, prefix, kv_len),
                    _rows(q, qs, dt, dev, "q"), _rows(k, ks, dt, dev, "k"), _rows(v, ks, dt, dev, "v"),
                    _rows(o, qs, dt, dev, "o"), None if low is None else _rows(low, qs, dt, dev, "low"),
                    _vec(lse, qs[:3], torch.float32, dev, "lse"), ws.data_ptr(), ws.numel())
    if rc:
        _check(rc, "lh_attn_forward")
    return o, lse


def lh_attn_backward(P: AttnParams, q, k, v, o, lse, dout, slopes=None, table=None, docs=None, prefix=None, kv_len=None,
                     low=None, dq=None, dk=None, dv=None, dtable=None, ws=None):
    """Gradients ``(dq, dk, dv, dtable)`` of ``lh_attn_forward`` (``dtable`` None without a table); ``o``, ``lse`` and
    ``low`` are its results, the other arguments those it got.  ``ws``: from ``new_attn_workspace(..., backward=True)``."""
    if P._status:
        _check(P._status, "lh_attn_backward")
    if P.buckets and table is None:
        _check(LH_ERR_INVALID_ARG, "lh_attn_backward")
    dev = q.device
    ws = _attn_ws(P, ws, dev, True, "lh_attn_backward")
    qs, ks = P._qs, P._ks
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if P.buckets and dtable is None:
        dtable = torch.empty_like(table)
    dt = P.dtype
    rc = _on_device(dev, _lib.lh_attn_backward, P._ref, _attn_mods(P, dev, slopes, table, docs, prefix, kv_len),
                    _rows(q, qs, dt, dev, "q"), _rows(k, ks, dt, dev, "k"), _rows(v, ks, dt, dev, "v"),
                    _rows(o, qs, dt, dev, "o"), None if low is None else _rows(low, qs, dt, dev, "low"),
                    _vec(lse, qs[:3], torch.float32, dev, "lse"), _rows(dout, qs, dt, dev, "dout"),
                    _rows(dq, qs, dt, dev, "dq"), _rows(dk, ks, dt, dev, "dk"), _rows(dv, ks, dt, dev, "dv"),
                    _vec(dtable, (P.Hq, P.buckets), dt, dev, "dtable") if P.buckets else 0, ws.data_ptr(), ws.numel())
    _check(rc, "lh_attn_backward")
    return dq, dk, dv, dtable
