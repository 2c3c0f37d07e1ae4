"""libmok: one GPU's share of the Mixture-of-Kittens forward MoE layer on MI355X.

A thin ctypes binding over ``libmok.so`` (built from ``csrc/`` with hipcc
for gfx950).  Every function here has the name of the C entry point it
marshals and does nothing but convert arguments: torch tensors become device
pointers, ``stream=None`` becomes torch's current HIP stream, a non-zero
status becomes a :class:`MokError`.  All arithmetic runs in the HIP kernels.

There is no fallback: importing this package without a built ``libmok.so``
raises ``ImportError``.
"""
from __future__ import annotations

import ctypes as C
import os
import re
from typing import List, Optional, Sequence

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmok.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "mok.h")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run `python token_dispatch_grouped_top_amd/build.py`")
# torch ships its own HIP runtime under the same soname; importing torch first
# makes libmok bind to that one, so torch's streams and allocations are valid
# for the library's launches (loading libmok first would pull in a second copy).
import torch  # noqa: E402,F401

_lib = C.CDLL(LIB_PATH)

MOK_OK, MOK_ERR_INVALID_ARG, MOK_ERR_UNSUPPORTED, MOK_ERR_WORKSPACE = 0, 1, 2, 3
MOK_ERR_HIP, MOK_ERR_DEVICE, MOK_ERR_CAPACITY = 4, 5, 6
MOK_ACT_BF16, MOK_ACT_MXFP8_E4M3 = 0, 1
MOK_MODE_STREAM, MOK_MODE_PERSISTENT = 0, 1
MOK_W_BF16, MOK_W_MXFP8_E4M3 = 0, 1
MOK_TYPE_F32, MOK_TYPE_BF16 = 0, 1
MOK_SCORE_SOFTMAX, MOK_SCORE_SIGMOID = 0, 1
MOK_GROUP_MAX, MOK_GROUP_TOP2 = 0, 1
MOK_STATE_F32, MOK_STATE_MXFP8 = 0, 1
MOK_BLOCK8_COPY, MOK_BLOCK8_SWIGLU, MOK_BLOCK8_SWIGLU_BWD = 0, 1, 2
MOK_BLOCK8_LINES, MOK_BLOCK8_BLOCKS = 0, 1


class MokError(RuntimeError):
    def __init__(self, status: int, call: str):
        self.status = status
        super().__init__(f"{call}: {mok_status_str(status)} ({status})")


class mok_layer_desc(C.Structure):
    _fields_ = [(n, C.c_int32) for n in (
        "hidden", "inter", "n_experts", "top_k", "expert_base", "n_local", "act_format",
        "minibatch", "ring_slots", "max_rows", "n_move_cus", "mode", "wait_timeout_us",
        "weights_packed", "no_split_k", "weight_format")]


class mok_tokens(C.Structure):
    _fields_ = [("part_ptr", C.c_void_p), ("n_partitions", C.c_int32), ("part_rows", C.c_int32)]


class mok_router_desc(C.Structure):
    _fields_ = [(n, C.c_int32) for n in (
        "n_experts", "top_k", "score", "n_groups", "top_groups", "group_rule", "renorm")] + [
        ("scale", C.c_float)]


class mok_adamw_tensor(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("p", "p_bf16", "grad", "m", "v", "m_scale", "v_scale")] + [
        ("n", C.c_int64), ("grad_type", C.c_int32), ("state_format", C.c_int32),
        ("lr_scale", C.c_float), ("weight_decay", C.c_float)]


class mok_adamw_hyper(C.Structure):
    _fields_ = [(n, C.c_double) for n in ("lr", "beta1", "beta2", "eps", "grad_scale")] + [
        ("step", C.c_int32), ("seed", C.c_uint32)]


class mok_adamw_plan(C.Structure):
    _fields_ = [("n_units", C.c_int64 * 2), ("n_tensors", C.c_int32 * 2), ("list", C.c_int32),
                ("reserved", C.c_int32)]


class mok_block8_source(C.Structure):
    _fields_ = [("op", C.c_int32), ("type", C.c_int32), ("x", C.c_void_p), ("ld", C.c_int64),
                ("d", C.c_void_p), ("ldd", C.c_int64), ("ring_rows", C.c_int32),
                ("reserved", C.c_int32)]


class mok_newton_schulz(C.Structure):
    _fields_ = [(n, C.c_float) for n in ("a", "b", "c")] + [("steps", C.c_int32)]


class mok_muon_hyper(C.Structure):
    _fields_ = [(n, C.c_double) for n in ("lr", "momentum", "weight_decay", "grad_scale", "scale")] + [
        ("nesterov", C.c_int32), ("reserved", C.c_int32), ("ns", mok_newton_schulz)]


_P, _I32, _I64, _SZ = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t
_DESC, _TOK = C.POINTER(mok_layer_desc), C.POINTER(mok_tokens)
_RTR = C.POINTER(mok_router_desc)
_SIGS = {
    "mok_route_topk": (C.c_int, [_P, _I32, _I32, _I32, _P, _P, _P]),
    "mok_route_scored": (C.c_int, [_RTR, _P, _I32, _I64, _P, _I32, _P, _P, _P, _P]),
    "mok_route_scored_backward": (C.c_int, [_RTR, _P, _I32, _I64, _I32, _P, _P, _P, _I64, _P]),
    "mok_route_bias_update": (C.c_int, [_P, _I32, _I32, C.c_float, _P, _I32, _P]),
    "mok_block8_slots": (_I64, [_I32, _I32]),
    "mok_block8_quantise": (C.c_int, [C.POINTER(mok_block8_source), _I32, _I32, _P, _I32, _P, _P, _P,
                                      _P, _I32, _P]),
    "mok_block8_quantise_weights": (C.c_int, [_P, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P]),
    "mok_block8_gemm": (C.c_int, [_P, _P, _I32, _I32, _P, _I32, _P, _P, _I32, _P, _I32, _P]),
    "mok_block8_wgrad": (C.c_int, [_P, _P, _I32, _P, _P, _I32, _I32, _P, _I32, _P, _I32, _I32, _P]),
    "mok_muon_workspace_size": (_SZ, [_I32, _I32, _I32]),
    "mok_orthogonalise": (C.c_int, [_P, _I32, _I32, _I32, _I32, C.POINTER(mok_newton_schulz), _P, _P,
                                    _SZ, _P]),
    "mok_muon_step": (C.c_int, [_P, _P, _P, _I32, _P, _I32, _I32, _I32, C.POINTER(mok_muon_hyper), _P,
                                _P, _SZ, _P]),
    "mok_adamw_table_size": (_SZ, [_I32]),
    "mok_adamw_build_table": (C.c_int, [C.POINTER(mok_adamw_tensor), _I32, _P, _SZ,
                                        C.POINTER(mok_adamw_plan), _P]),
    "mok_adamw_step": (C.c_int, [_P, C.POINTER(mok_adamw_plan), C.POINTER(mok_adamw_hyper), _P, _P]),
    "mok_moe_forward_scored": (C.c_int, [_DESC, _RTR, _P, _I32, _I64, _P, _I32, _P, _P, _P, _TOK,
                                         _P, _P, _TOK, _P, _SZ, _P]),
    "mok_route_gemm_workspace_size": (_SZ, [_I32, _I32, _I32]),
    "mok_route_topk_gemm": (C.c_int, [_P, _P, _I32, _I32, _I32, _I32, _P, _SZ, _P, _P, _P]),
    "mok_schedule_workspace_size": (_SZ, [_I64, _I32, _I32]),
    "mok_build_schedule": (C.c_int, [_P, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P, _SZ, _P]),
    "mok_schedule_noalloc_max_bytes": (_SZ, []),
    "mok_build_schedule_noalloc": (C.c_int, [_P, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P]),
    "mok_choose_minibatch": (_I32, [_I32, _I32, _I32, _I32, _I64]),
    "mok_build_windows": (C.c_int, [_P, _I32, _I32, _I32, _P, _P]),
    "mok_build_schedule_windows": (C.c_int, [_P, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _I32,
                                             _I32, _P, _P, _SZ, _P]),
    "mok_dispatch_gather": (C.c_int, [_TOK, _I32, _I32, _P, _P, _I32, _I32, _I32, _P, _P, _I32,
                                      _I32, _P, _P]),
    "mok_expert_ffn": (C.c_int, [_DESC, _P, _P, _I32, _P, _I32, _I32, _P, _P, _P, _P, _I32, _P,
                                 _I32, _P, _SZ, _P]),
    "mok_gemm_workspace_size": (_SZ, []),
    "mok_expert_gate_up": (C.c_int, [_DESC, _P, _P, _I32, _P, _I32, _I32, _P, _P, _P, _I32, _P,
                                     _SZ, _P]),
    "mok_packed_weights_size": (C.c_int, [_DESC, C.POINTER(_SZ), C.POINTER(_SZ)]),
    "mok_pack_weights": (C.c_int, [_DESC, _P, _P, _P, _P, _P]),
    "mok_expert_down": (C.c_int, [_DESC, _P, _P, _I32, _P, _I32, _I32, _P, _P, _I32, _P, _SZ,
                                  _P]),
    "mok_combine": (C.c_int, [_P, _I32, _P, _P, _I32, _I32, _I32, _TOK, _P, _P]),
    "mok_combine_slots": (C.c_int, [_P, _I32, _P, _P, _I32, _I32, _P, _P, _I32, _I32, _TOK, _P,
                                    _P]),
    "mok_forward_workspace_size": (_SZ, [_DESC, _I32, _I32]),
    "mok_moe_forward": (C.c_int, [_DESC, _P, _I32, _TOK, _P, _P, _TOK, _P, _SZ, _P]),
    "mok_moe_forward_routed": (C.c_int, [_DESC, _P, _P, _I32, _TOK, _P, _P, _TOK, _P, _SZ, _P]),
    "mok_forward_router_workspace_size": (_SZ, [_DESC, _I32]),
    "mok_moe_forward_router": (C.c_int, [_DESC, _P, _I32, _TOK, _P, _P, _TOK, _P, _SZ, _P]),
    "mok_moe_forward_batches": (C.c_int, [_DESC, _I32, _P, _P, _I32, _TOK, _P, _P, _TOK, _P,
                                          _SZ, _P]),
    "mok_tune_forward": (C.c_int, [_DESC, _P, _I32, _P, _I32, _I32, _I32, _P, _P, _I32, _TOK,
                                   _P, _P, _TOK, _P, _SZ, _DESC, C.POINTER(C.c_float), _P]),
    "mok_packed_weights_bwd_size": (C.c_int, [_DESC, C.POINTER(_SZ), C.POINTER(_SZ)]),
    "mok_pack_weights_bwd": (C.c_int, [_DESC, _P, _P, _P, _P, _P]),
    "mok_combine_backward": (C.c_int, [_TOK, _P, _I32, _P, _P, _I32, _I32, _P, _I32, _I32, _P,
                                       _I32, _P, _P, _P]),
    "mok_expert_ffn_backward": (C.c_int, [_DESC, _P, _I32, _P, _P, _I32, _I32, _P, _P, _P, _P,
                                          _P, _P, _I32, _P]),
    "mok_expert_gate_up_save_h": (C.c_int, [_DESC, _P, _I32, _P, _I32, _I32, _P, _P, _I32, _P,
                                            _P, _SZ, _P]),
    "mok_expert_ffn_backward_saved": (C.c_int, [_DESC, _P, _P, _I32, _I32, _P, _P, _P, _P, _P,
                                                _I32, _P]),
    "mok_wgrad_workspace_size": (_SZ, [_DESC, _I32]),
    "mok_expert_wgrad": (C.c_int, [_DESC, _P, _I32, _P, _I32, _P, _P, _I32, _P, _P, _P, _P, _SZ,
                                   _P]),
    "mok_dispatch_backward": (C.c_int, [_P, _I32, _P, _P, _I32, _I32, _P, _I32, _I32, _TOK, _P,
                                        _P]),
    "mok_expert_down_merge": (C.c_int, [_DESC, _P, _P, _I32, _P, _I32, _I32, _P, _P, _I32, _P,
                                        _P, _P, _TOK, _P, _P, _SZ, _P]),
    "mok_combine_slots_multi": (C.c_int, [_P, _I32, _P, _P, _I32, _I32, _P, _P, _I32, _I32, _TOK,
                                          _P, _P]),
    "mok_combine_backward_mx": (C.c_int, [_TOK, _P, _I32, _P, _P, _I32, _I32, _P, _I32, _I32,
                                          _P, _P, _I32, _P, _P, _P]),
    "mok_expert_gate_up_save_h_mx": (C.c_int, [_DESC, _P, _P, _I32, _P, _I32, _I32, _P, _P, _P,
                                               _I32, _P, _P, _SZ, _P]),
    "mok_expert_ffn_backward_mx": (C.c_int, [_DESC, _P, _P, _I32, _P, _P, _P, _I32, _I32, _P, _P,
                                             _P, _P, _I32, _P, _P, _P, _I32, _P]),
    "mok_expert_wgrad_mx": (C.c_int, [_DESC, _P, _P, _I32, _P, _P, _I32, _P, _P, _P, _P, _I32,
                                      _P, _P, _P, _P, _SZ, _P]),
    "mok_device_status": (C.c_int, [_P, C.POINTER(C.c_int32), _P]),
    "mok_forward_minibatch": (_I32, [_DESC, _I32]),
    "mok_status_str": (C.c_char_p, [C.c_int]),
    "mok_last_hip_error": (C.c_char_p, []),
}
for _name, (_res, _args) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.restype, _f.argtypes = _res, _args


def header_functions() -> List[str]:
    """Names of the functions include/mok.h declares."""
    text = open(HEADER).read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[a-z_0-9]+\s*\*?\s*(mok_[a-z_0-9]+)\s*\(",
                                 text, flags=re.M)))


def _ptr(x) -> int:
    if x is None:
        return 0
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(s) -> int:
    if s is None:
        # the handle alone: building torch's Stream object takes 2.7 us, more than a small launch
        if torch.cuda.is_initialized():
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(status: int, call: str) -> None:
    if status != MOK_OK:
        if status == MOK_ERR_HIP:
            call = f"{call} [{_lib.mok_last_hip_error().decode()}]"
        raise MokError(status, call)


class Tokens:
    """Token partitions on the device (a ``mok_tokens`` plus what keeps it alive).

    ``parts`` are bf16-bit tensors (torch.int16/uint16/bfloat16) of shape
    [part_rows, H] on the GPU; the pointer array is itself a device tensor.
    """

    def __init__(self, parts: Sequence, part_rows: Optional[int] = None):
        import torch
        self.parts = list(parts)
        rows = part_rows if part_rows is not None else self.parts[0].shape[0]
        dev = self.parts[0].device
        self.ptrs = torch.tensor([p.data_ptr() for p in self.parts], dtype=torch.int64, device=dev)
        self.c = mok_tokens(self.ptrs.data_ptr(), len(self.parts), rows)

    @classmethod
    def from_tensor(cls, x):
        return cls([x], x.shape[0])


# ------------------------------------------------------------------ calls
def mok_status_str(status: int) -> str:
    return _lib.mok_status_str(status).decode()


def mok_route_topk(logits, T: int, E: int, k: int, topk_idx, topk_gate, stream=None) -> None:
    _check(_lib.mok_route_topk(_ptr(logits), T, E, k, _ptr(topk_idx), _ptr(topk_gate),
                               _stream(stream)), "mok_route_topk")


_TYPES = {torch.float32: MOK_TYPE_F32, torch.bfloat16: MOK_TYPE_BF16}


def _device() -> int:
    """The current GPU, -1 before torch has touched one."""
    return torch._C._cuda_getDevice() if torch.cuda.is_initialized() else -1


def _stream_of(stream, device: int) -> int:
    """_stream with the current GPU at hand."""
    return torch._C._cuda_getCurrentRawStream(device) if stream is None and device >= 0 else _stream(stream)


def _stream_object(stream):
    """torch's object of a call's stream argument."""
    if stream is None:
        return torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return stream
    handle = _stream(stream)                   # ExternalStream(0) would be a new stream
    return torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()


# The checks of a call are a part of its latency: what is right passes on one line, the error is
# worked out behind it.
def _buffer(x, name: str, dtypes, n: int, device: int) -> int:
    """Address of a buffer of at least n elements: None, a raw address (not checked), or a dense
    tensor of one of dtypes on the GPU `device`."""
    if x is None:
        return 0
    if type(x) is int:
        return x
    if x.dtype in dtypes and x.is_contiguous() and x.numel() >= n and x.get_device() == device >= 0:
        return x.data_ptr()
    if x.dtype not in dtypes:
        raise ValueError(f"{name}: {x.dtype} where {' or '.join(map(str, dtypes))} is wanted")
    if not x.is_contiguous() or x.numel() < n:
        raise ValueError(f"{name}: {tuple(x.shape)} with strides {x.stride()} where {n} dense elements "
                         "are wanted")
    raise ValueError(f"{name}: on {x.device}, which is not the current GPU")


def _rows(x, name: str, T: int, E: int, device: int):
    """(address, mok_type, row stride) of fp32 or bf16 rows, the rows themselves dense."""
    if x is None:
        return 0, MOK_TYPE_F32, E
    kind = _TYPES.get(x.dtype)
    if kind is None:
        raise ValueError(f"{name}: {x.dtype} where torch.float32 or torch.bfloat16 is wanted")
    if x.dim() == 2:
        (rows, width), (ld, step) = x.shape, x.stride()
        if rows >= T and width == E and (step == 1 or E == 1) and x.get_device() == device >= 0:
            return x.data_ptr(), kind, ld if T > 1 else max(ld, E)
        if rows >= T and width == E and (step == 1 or E == 1):
            raise ValueError(f"{name}: on {x.device}, which is not the current GPU")
    raise ValueError(f"{name}: {tuple(x.shape)} with strides {x.stride()} where [{T}][{E}] rows of "
                     "dense values are wanted")


_F32, _I32S, _U8, _BF16 = (torch.float32,), (torch.int32,), (torch.uint8,), (torch.bfloat16,)


def mok_route_scored(router: mok_router_desc, logits, T: int, topk_idx, topk_gate, bias=None,
                     load=None, stream=None) -> None:
    E, n, device = router.n_experts, T * router.top_k, _device()
    at, kind, ld = _rows(logits, "logits", T, E, device)
    _check(_lib.mok_route_scored(C.byref(router), at, kind, ld,
                                 _buffer(bias, "bias", _F32, E, device), T,
                                 _buffer(topk_idx, "topk_idx", _I32S, n, device),
                                 _buffer(topk_gate, "topk_gate", _F32, n, device),
                                 _buffer(load, "load", _I32S, E, device), _stream_of(stream, device)),
           "mok_route_scored")


def mok_route_scored_backward(router: mok_router_desc, logits, T: int, topk_idx, dgate, dlogits,
                              stream=None) -> None:
    E, n, device = router.n_experts, T * router.top_k, _device()
    at, kind, ld = _rows(logits, "logits", T, E, device)
    to, kind_to, ldd = _rows(dlogits, "dlogits", T, E, device)
    if kind_to != kind:
        raise ValueError(f"dlogits: {dlogits.dtype} where the logits are {logits.dtype}")
    _check(_lib.mok_route_scored_backward(C.byref(router), at, kind, ld, T,
                                          _buffer(topk_idx, "topk_idx", _I32S, n, device),
                                          _buffer(dgate, "dgate", _F32, n, device), to, ldd,
                                          _stream_of(stream, device)), "mok_route_scored_backward")


def mok_route_bias_update(load, n_layers: int, E: int, rate: float, bias, clear_load: int = 0,
                          stream=None) -> None:
    n, device = n_layers * E, _device()
    _check(_lib.mok_route_bias_update(_buffer(load, "load", _I32S, n, device), n_layers, E, rate,
                                      _buffer(bias, "bias", _F32, n, device), clear_load,
                                      _stream_of(stream, device)), "mok_route_bias_update")


_CODES = (torch.uint8, torch.float8_e4m3fn)


def mok_block8_slots(rows: int, n_local: int = 1) -> int:
    return int(_lib.mok_block8_slots(rows, n_local))


def _blocks(n: int) -> int:
    return (n + 127) // 128


def _typed(x, name: str, n: int, device: int):
    """(address, mok_type) of a dense fp32 or bf16 buffer of at least n elements (a raw address: fp32)."""
    if x is None or type(x) is int:
        return x or 0, MOK_TYPE_F32
    return _buffer(x, name, tuple(_TYPES), n, device), _TYPES[x.dtype]


def mok_block8_quantise(x, rows: int, W: int, codes=None, scales=None, source: int = MOK_BLOCK8_COPY,
                        d=None, codes_t=None, scales_t=None, t_scales: int = MOK_BLOCK8_LINES,
                        offsets=None, n_local: int = 1, ring_rows: int = 0, stream=None) -> None:
    """x (and d): rows of fp32 or bf16, the rows themselves dense; or, with ring_rows, a dense bf16 buffer of
    column-blocked rows.  codes: uint8 or float8_e4m3fn."""
    device, at_d, ldd = _device(), 0, 0
    if ring_rows:
        if not isinstance(x, int) and x is not None and x.dtype is torch.int16:
            x = x.view(torch.bfloat16)
        at, kind, ld = _buffer(x, "x", _BF16, ring_rows * W, device), MOK_TYPE_BF16, 0
    else:
        at, kind, ld = _rows(x, "x", rows, 2 * W if source == MOK_BLOCK8_SWIGLU else W, device)
        if d is not None:
            at_d, kind_d, ldd = _rows(d, "d", rows, W // 2, device)
            if kind_d != kind:
                raise ValueError(f"d: {d.dtype} where x is {x.dtype}")
    S = 0 if codes_t is None and scales_t is None else mok_block8_slots(rows, n_local)
    n_scales = S // 128 * W if t_scales == MOK_BLOCK8_LINES else S // 128 * _blocks(W)
    _check(_lib.mok_block8_quantise(mok_block8_source(source, kind, at, ld, at_d, ldd, ring_rows), rows, W,
                                    _buffer(offsets, "offsets", _I32S, n_local + 1, device), n_local,
                                    _buffer(codes, "codes", _CODES, rows * W, device),
                                    _buffer(scales, "scales", _F32, rows * _blocks(W), device),
                                    _buffer(codes_t, "codes_t", _CODES, W * S, device),
                                    _buffer(scales_t, "scales_t", _F32, n_scales, device), t_scales,
                                    _stream_of(stream, device)), "mok_block8_quantise")


def mok_block8_quantise_weights(w, n: int, N: int, K: int, codes, scales, codes_t=None, scales_t=None,
                                stream=None) -> None:
    device, blocks = _device(), n * _blocks(N) * _blocks(K)
    at, kind = _typed(w, "w", n * N * K, device)
    _check(_lib.mok_block8_quantise_weights(at, kind, n, N, K,
                                            _buffer(codes, "codes", _CODES, n * N * K, device),
                                            _buffer(scales, "scales", _F32, blocks, device),
                                            _buffer(codes_t, "codes_t", _CODES, n * N * K, device),
                                            _buffer(scales_t, "scales_t", _F32, blocks, device),
                                            _stream_of(stream, device)), "mok_block8_quantise_weights")


def mok_block8_gemm(a, a_scales, rows: int, K: int, w, w_scales, N: int, out, offsets=None,
                    n_local: int = 1, stream=None) -> None:
    device = _device()
    to, kind = _typed(out, "out", rows * N, device)
    _check(_lib.mok_block8_gemm(_buffer(a, "a", _CODES, rows * K, device),
                                _buffer(a_scales, "a_scales", _F32, rows * _blocks(K), device), rows, K,
                                _buffer(offsets, "offsets", _I32S, n_local + 1, device), n_local,
                                _buffer(w, "w", _CODES, n_local * N * K, device),
                                _buffer(w_scales, "w_scales", _F32, n_local * _blocks(N) * _blocks(K), device),
                                N, to, kind, _stream_of(stream, device)), "mok_block8_gemm")


def mok_block8_wgrad(dy_t, dy_scales, M: int, x_t, x_scales, N: int, rows: int, dw, offsets=None,
                     n_local: int = 1, accumulate: int = 0, stream=None) -> None:
    device, S = _device(), mok_block8_slots(rows, n_local)
    to, kind = _typed(dw, "dw", n_local * M * N, device)
    _check(_lib.mok_block8_wgrad(_buffer(dy_t, "dy_t", _CODES, M * S, device),
                                 _buffer(dy_scales, "dy_scales", _F32, M * (S // 128), device), M,
                                 _buffer(x_t, "x_t", _CODES, N * S, device),
                                 _buffer(x_scales, "x_scales", _F32, _blocks(N) * (S // 128), device), N, rows,
                                 _buffer(offsets, "offsets", _I32S, n_local + 1, device), n_local, to, kind,
                                 accumulate, _stream_of(stream, device)), "mok_block8_wgrad")


def mok_muon_workspace_size(n: int, rows: int, cols: int) -> int:
    return int(_lib.mok_muon_workspace_size(n, rows, cols))


NEWTON_SCHULZ = (3.4445, -4.7750, 2.0315)


def _workspace(ws, ws_bytes: Optional[int], device: int):
    """(address, bytes) of a dense buffer on the GPU (a raw address: of ws_bytes)."""
    if ws is None or type(ws) is int:
        return ws or 0, ws_bytes or 0
    size = ws.numel() * ws.element_size()
    return _buffer(ws, "ws", (ws.dtype,), 0, device), size if ws_bytes is None else min(ws_bytes, size)


def mok_orthogonalise(x, n: int, rows: int, cols: int, out, ws, steps: int = 5,
                      coefficients: Sequence[float] = NEWTON_SCHULZ, ws_bytes: Optional[int] = None,
                      stream=None) -> None:
    device, cells = _device(), n * rows * cols
    at, kind = _typed(x, "x", cells, device)
    scratch, size = _workspace(ws, ws_bytes, device)
    _check(_lib.mok_orthogonalise(at, kind, n, rows, cols, C.byref(mok_newton_schulz(*coefficients, steps)),
                                  _buffer(out, "out", _BF16, cells, device), scratch, size,
                                  _stream_of(stream, device)), "mok_orthogonalise")


def mok_muon_step(p, grad, m, n: int, rows: int, cols: int, ws, lr: float, momentum: float, scale: float,
                  weight_decay: float = 0.0, grad_scale: float = 1.0, nesterov: int = 1, steps: int = 5,
                  coefficients: Sequence[float] = NEWTON_SCHULZ, p_bf16=None, scalars=None,
                  ws_bytes: Optional[int] = None, stream=None) -> None:
    """scalars: as for mok_adamw_step."""
    device, cells = _device(), n * rows * cols
    at, kind = _typed(grad, "grad", cells, device)
    scratch, size = _workspace(ws, ws_bytes, device)
    h = mok_muon_hyper(lr, momentum, weight_decay, grad_scale, scale, nesterov, 0,
                       mok_newton_schulz(*coefficients, steps))
    _check(_lib.mok_muon_step(_buffer(p, "p", _F32, cells, device), _buffer(p_bf16, "p_bf16", _BF16, cells, device),
                              at, kind, _buffer(m, "m", _F32, cells, device), n, rows, cols, C.byref(h),
                              _scalars(scalars), scratch, size, _stream_of(stream, device)), "mok_muon_step")


class AdamwTensors:
    """Tensors of an AdamW step: the device table of ``mok_adamw_build_table``, its plan, and what
    keeps the tensors alive.

    One dict per tensor: ``p`` (fp32), ``grad`` (fp32 or bf16), ``m`` and ``v`` (fp32, or uint8
    codes beside ``m_scale`` and ``v_scale``, uint8), and optionally ``p_bf16``, ``lr_scale`` (1)
    and ``weight_decay`` (0).  Dense tensors of the same number of elements on one GPU.  Built
    once for a program's buffers, on the stream given, which is waited for: the list can then be
    used on any stream.  Built during a capture, on a captured stream, it serves the steps of that
    graph, which writes the table anew on each replay.  A program that lets torch allocate new
    gradients for a step builds a new list for them: 35 us for one tensor, 3 us for each more.

    A list may be dropped while a step of it runs, on any stream (a stream given as a raw handle
    lives as long as the list).  The tensors themselves are those of the current stream, as for
    torch's operations.  A captured graph holds addresses: keep its lists as long as the graph.
    """

    def __init__(self, tensors: Sequence[dict], stream=None):
        self.tensors = [dict(t) for t in tensors]
        self.c = (mok_adamw_tensor * len(self.tensors))()
        device = _device()
        for c, t in zip(self.c, self.tensors):
            n = t["p"].numel()
            coded = t["m"].dtype == torch.uint8
            state, blocks = _U8 if coded else _F32, (n + 31) // 32
            for name, kinds, size in (("p", _F32, n), ("grad", tuple(_TYPES), n), ("m", state, n),
                                      ("v", state, n), ("p_bf16", _BF16, n), ("m_scale", _U8, blocks),
                                      ("v_scale", _U8, blocks)):
                x = t.get(name)
                if x is None and (name == "p_bf16" or (name.endswith("scale") and not coded)):
                    continue
                if x is None:
                    raise ValueError(f"{name}: missing")
                address = _buffer(x, name, kinds, size, device)
                if x.numel() != size:
                    raise ValueError(f"{name}: {x.numel()} elements where {size} are wanted")
                setattr(c, name, address)
            c.n, c.grad_type = n, _TYPES[t["grad"].dtype]
            c.state_format = MOK_STATE_MXFP8 if coded else MOK_STATE_F32
            c.lr_scale, c.weight_decay = t.get("lr_scale", 1.0), t.get("weight_decay", 0.0)
        self.plan, self.table, self.address = mok_adamw_plan(), None, 0
        self.device, self.streams = device, set()
        if self.tensors:
            size = mok_adamw_table_size(len(self.c))
            on, captured = _stream_object(stream), torch.cuda.is_current_stream_capturing()
            if on.device.index != device:
                raise ValueError(f"stream: of {on.device}, which is not the current GPU")
            # memory of the stream that writes it: a block of another stream's may still have work pending there
            with torch.cuda.stream(on):
                if captured and not torch.cuda.is_current_stream_capturing():
                    raise ValueError("stream: not captured, while the current stream is")
                self.table = torch.empty(size, dtype=torch.uint8, device=self.tensors[0]["p"].device)
                self.address = self.table.data_ptr()
                mok_adamw_build_table(self.c, self.table, self.plan, on.cuda_stream)
                if not torch.cuda.is_current_stream_capturing():
                    on.synchronize()
            here = torch.cuda.current_stream()
            self.table.record_stream(here)
            self.streams.add(here.cuda_stream)

    def record_stream(self, stream) -> None:
        """torch's ``Tensor.record_stream`` for the table and the list's tensors: their memory is not
        given out again before the work that ``stream`` has when they are dropped is done."""
        if self.table is None:                    # an empty list
            return
        on = _stream_object(stream)
        for x in (self.table, *(x for t in self.tensors for x in t.values())):
            if hasattr(x, "record_stream"):
                x.record_stream(on)
        self.streams.add(on.cuda_stream)


def mok_adamw_table_size(n_tensors: int) -> int:
    return int(_lib.mok_adamw_table_size(n_tensors))


def mok_adamw_build_table(tensors, table, plan: mok_adamw_plan, stream=None) -> None:
    """tensors: a ctypes array of mok_adamw_tensor; table: dense bytes on the GPU; plan: filled in."""
    _check(_lib.mok_adamw_build_table(tensors, len(tensors), _ptr(table), _ws_bytes(table, None),
                                      C.byref(plan), _stream(stream)), "mok_adamw_build_table")


def _scalars(x) -> int:
    """Address of a mok_adamw_scalars: None, a raw address, or 16 dense bytes on the GPU."""
    if x is not None and not isinstance(x, int):
        size = x.element_size()
        if x.numel() * size != 16:
            raise ValueError("scalars: 16 dense bytes are wanted")
        x = _buffer(x, "scalars", (x.dtype,), 16 // size, _device())
    return x or 0


def mok_adamw_step(tensors: AdamwTensors, lr: float, beta1: float, beta2: float, eps: float,
                   step: int, grad_scale: float = 1.0, seed: int = 0, scalars=None,
                   stream=None) -> None:
    """scalars: None, or 16 bytes on the GPU as a ``mok_adamw_scalars`` (lr and grad_scale fp32,
    step and skip int32)."""
    scalars = _scalars(scalars)
    h = mok_adamw_hyper(lr, beta1, beta2, eps, grad_scale, step, seed)
    device = _device()
    if tensors.device != device and tensors.address:
        raise ValueError(f"tensors: a list on cuda:{tensors.device}, which is not the current GPU")
    on = _stream_of(stream, device)
    if on not in tensors.streams:                 # once for each stream but the one that the list was built under
        tensors.record_stream(stream)
    _check(_lib.mok_adamw_step(tensors.address, C.byref(tensors.plan), C.byref(h), scalars, on),
           "mok_adamw_step")


def mok_route_gemm_workspace_size(T: int, E: int, H: int) -> int:
    return int(_lib.mok_route_gemm_workspace_size(T, E, H))


def mok_route_topk_gemm(x, w_router, T: int, H: int, E: int, k: int, ws, topk_idx, topk_gate,
                        ws_bytes: Optional[int] = None, stream=None) -> None:
    _check(_lib.mok_route_topk_gemm(_ptr(x), _ptr(w_router), T, H, E, k, _ptr(ws),
                                    _ws_bytes(ws, ws_bytes), _ptr(topk_idx), _ptr(topk_gate),
                                    _stream(stream)), "mok_route_topk_gemm")


def mok_schedule_workspace_size(T: int, k: int, n_local: int) -> int:
    return int(_lib.mok_schedule_workspace_size(T, k, n_local))


def mok_build_schedule(topk_idx, T: int, k: int, expert_base: int, n_local: int, counts, offsets,
                       slot_of_assign, assign_of_slot, ws, ws_bytes: Optional[int] = None,
                       stream=None) -> None:
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size()
    _check(_lib.mok_build_schedule(_ptr(topk_idx), T, k, expert_base, n_local, _ptr(counts),
                                   _ptr(offsets), _ptr(slot_of_assign), _ptr(assign_of_slot),
                                   _ptr(ws), ws_bytes, _stream(stream)), "mok_build_schedule")


def mok_schedule_noalloc_max_bytes() -> int:
    return int(_lib.mok_schedule_noalloc_max_bytes())


def mok_build_schedule_noalloc(topk_idx, T: int, k: int, expert_base: int, n_local: int, counts,
                               offsets, slot_of_assign, assign_of_slot, stream=None) -> None:
    _check(_lib.mok_build_schedule_noalloc(_ptr(topk_idx), T, k, expert_base, n_local,
                                           _ptr(counts), _ptr(offsets), _ptr(slot_of_assign),
                                           _ptr(assign_of_slot), _stream(stream)),
           "mok_build_schedule_noalloc")


def mok_choose_minibatch(n_cus: int, tile_m: int, tile_n: int, n_out: int, rows: int = 0) -> int:
    return int(_lib.mok_choose_minibatch(n_cus, tile_m, tile_n, n_out, rows))


def mok_build_schedule_windows(topk_idx, T: int, k: int, expert_base: int, n_local: int, counts,
                               offsets, slot_of_assign, assign_of_slot, M: int, nwin: int,
                               win_seg, ws, ws_bytes: Optional[int] = None, stream=None) -> None:
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size()
    _check(_lib.mok_build_schedule_windows(_ptr(topk_idx), T, k, expert_base, n_local,
                                           _ptr(counts), _ptr(offsets), _ptr(slot_of_assign),
                                           _ptr(assign_of_slot), M, nwin, _ptr(win_seg), _ptr(ws),
                                           ws_bytes, _stream(stream)), "mok_build_schedule_windows")


def mok_build_windows(offsets, n_local: int, M: int, nwin: int, win_seg, stream=None) -> None:
    _check(_lib.mok_build_windows(_ptr(offsets), n_local, M, nwin, _ptr(win_seg),
                                  _stream(stream)), "mok_build_windows")


def mok_dispatch_gather(src: Tokens, H: int, k: int, assign_of_slot, offsets, n_local: int,
                        slot_begin: int, slot_end: int, ring, ring_scales, ring_slots: int,
                        act_format: int, dev_status=None, stream=None) -> None:
    _check(_lib.mok_dispatch_gather(C.byref(src.c), H, k, _ptr(assign_of_slot), _ptr(offsets),
                                    n_local, slot_begin, slot_end, _ptr(ring), _ptr(ring_scales),
                                    ring_slots, act_format, _ptr(dev_status), _stream(stream)),
           "mok_dispatch_gather")


def _ws_bytes(ws, ws_bytes):
    if ws is None:
        return 0
    return ws.numel() * ws.element_size() if ws_bytes is None else ws_bytes


def mok_gemm_workspace_size() -> int:
    return int(_lib.mok_gemm_workspace_size())


def mok_expert_ffn(desc: mok_layer_desc, ring, ring_scales, ring_slots: int, offsets,
                   slot_begin: int, slot_end: int, w_gate_up, w_down, act, act_scales,
                   act_rows: int, y, y_rows: int, ws=None, ws_bytes: Optional[int] = None,
                   stream=None) -> None:
    _check(_lib.mok_expert_ffn(C.byref(desc), _ptr(ring), _ptr(ring_scales), ring_slots,
                               _ptr(offsets), slot_begin, slot_end, _ptr(w_gate_up), _ptr(w_down),
                               _ptr(act), _ptr(act_scales), act_rows, _ptr(y), y_rows, _ptr(ws),
                               _ws_bytes(ws, ws_bytes), _stream(stream)), "mok_expert_ffn")


def mok_packed_weights_size(desc: mok_layer_desc):
    """(gate_up_bytes, down_bytes) of the packed weights for desc."""
    gu, dn = _SZ(0), _SZ(0)
    _check(_lib.mok_packed_weights_size(C.byref(desc), C.byref(gu), C.byref(dn)),
           "mok_packed_weights_size")
    return gu.value, dn.value


def mok_pack_weights(desc: mok_layer_desc, w_gate_up, w_down, packed_gate_up, packed_down,
                     stream=None) -> None:
    _check(_lib.mok_pack_weights(C.byref(desc), _ptr(w_gate_up), _ptr(w_down),
                                 _ptr(packed_gate_up), _ptr(packed_down), _stream(stream)),
           "mok_pack_weights")


def mok_expert_gate_up(desc: mok_layer_desc, ring, ring_scales, ring_slots: int, offsets,
                       slot_begin: int, slot_end: int, w_gate_up, act, act_scales, act_rows: int,
                       ws=None, ws_bytes: Optional[int] = None, stream=None) -> None:
    _check(_lib.mok_expert_gate_up(C.byref(desc), _ptr(ring), _ptr(ring_scales), ring_slots,
                                   _ptr(offsets), slot_begin, slot_end, _ptr(w_gate_up),
                                   _ptr(act), _ptr(act_scales), act_rows, _ptr(ws),
                                   _ws_bytes(ws, ws_bytes), _stream(stream)),
           "mok_expert_gate_up")


def mok_expert_down(desc: mok_layer_desc, act, act_scales, act_rows: int, offsets,
                    slot_begin: int, slot_end: int, w_down, y, y_rows: int, ws=None,
                    ws_bytes: Optional[int] = None, stream=None) -> None:
    _check(_lib.mok_expert_down(C.byref(desc), _ptr(act), _ptr(act_scales), act_rows,
                                _ptr(offsets), slot_begin, slot_end, _ptr(w_down), _ptr(y),
                                y_rows, _ptr(ws), _ws_bytes(ws, ws_bytes), _stream(stream)),
           "mok_expert_down")


def mok_combine(y, y_rows: int, slot_of_assign, topk_gate, T: int, k: int, H: int, out: Tokens,
                dev_status=None, stream=None) -> None:
    _check(_lib.mok_combine(_ptr(y), y_rows, _ptr(slot_of_assign), _ptr(topk_gate), T, k, H,
                            C.byref(out.c), _ptr(dev_status), _stream(stream)), "mok_combine")


def mok_combine_slots(y, y_rows: int, assign_of_slot, offsets, n_local: int, n_slots: int,
                      slot_of_assign, topk_gate, k: int, H: int, out: Tokens, dev_status=None,
                      stream=None) -> None:
    _check(_lib.mok_combine_slots(_ptr(y), y_rows, _ptr(assign_of_slot), _ptr(offsets), n_local,
                                  n_slots, _ptr(slot_of_assign), _ptr(topk_gate), k, H,
                                  C.byref(out.c), _ptr(dev_status), _stream(stream)),
           "mok_combine_slots")


def mok_forward_workspace_size(desc: mok_layer_desc, T: int, n_macro: int = 1) -> int:
    return int(_lib.mok_forward_workspace_size(C.byref(desc), T, n_macro))


def mok_forward_minibatch(desc: mok_layer_desc, T: int) -> int:
    return int(_lib.mok_forward_minibatch(C.byref(desc), T))


def mok_moe_forward(desc: mok_layer_desc, logits, T: int, x: Tokens, w_gate_up, w_down,
                    out: Tokens, ws, ws_bytes: Optional[int] = None, stream=None) -> None:
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size()
    _check(_lib.mok_moe_forward(C.byref(desc), _ptr(logits), T, C.byref(x.c), _ptr(w_gate_up),
                                _ptr(w_down), C.byref(out.c), _ptr(ws), ws_bytes,
                                _stream(stream)), "mok_moe_forward")


def mok_forward_router_workspace_size(desc: mok_layer_desc, T: int) -> int:
    return int(_lib.mok_forward_router_workspace_size(C.byref(desc), T))


def mok_moe_forward_scored(desc: mok_layer_desc, router: mok_router_desc, logits, T: int, x: Tokens,
                           w_gate_up, w_down, out: Tokens, ws, bias=None, topk_idx=None,
                           topk_gate=None, load=None, ws_bytes: Optional[int] = None,
                           stream=None) -> None:
    E, n, device = router.n_experts, T * router.top_k, _device()
    at, kind, ld = _rows(logits, "logits", T, E, device)
    _check(_lib.mok_moe_forward_scored(C.byref(desc), C.byref(router), at, kind, ld,
                                       _buffer(bias, "bias", _F32, E, device), T,
                                       _buffer(topk_idx, "topk_idx", _I32S, n, device),
                                       _buffer(topk_gate, "topk_gate", _F32, n, device),
                                       _buffer(load, "load", _I32S, E, device), C.byref(x.c),
                                       _ptr(w_gate_up), _ptr(w_down), C.byref(out.c), _ptr(ws),
                                       _ws_bytes(ws, ws_bytes), _stream_of(stream, device)),
           "mok_moe_forward_scored")


def mok_moe_forward_router(desc: mok_layer_desc, w_router, T: int, x: Tokens, w_gate_up, w_down,
                           out: Tokens, ws, ws_bytes: Optional[int] = None, stream=None) -> None:
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size()
    _check(_lib.mok_moe_forward_router(C.byref(desc), _ptr(w_router), T, C.byref(x.c),
                                       _ptr(w_gate_up), _ptr(w_down), C.byref(out.c), _ptr(ws),
                                       ws_bytes, _stream(stream)), "mok_moe_forward_router")


def mok_moe_forward_routed(desc: mok_layer_desc, topk_idx, topk_gate, T: int, x: Tokens,
                           w_gate_up, w_down, out: Tokens, ws, ws_bytes: Optional[int] = None,
                           stream=None) -> None:
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size()
    _check(_lib.mok_moe_forward_routed(C.byref(desc), _ptr(topk_idx), _ptr(topk_gate), T,
                                       C.byref(x.c), _ptr(w_gate_up), _ptr(w_down),
                                       C.byref(out.c), _ptr(ws), ws_bytes, _stream(stream)),
           "mok_moe_forward_routed")


def mok_moe_forward_batches(desc: mok_layer_desc, n_macro: int, topk_idx: Sequence,
                            topk_gate: Sequence, T: int, x: Tokens, w_gate_up, w_down,
                            out: Sequence[Tokens], ws, ws_bytes: Optional[int] = None,
                            stream=None) -> None:
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size()
    idx_arr = (C.c_void_p * n_macro)(*[_ptr(t) for t in topk_idx])
    gate_arr = (C.c_void_p * n_macro)(*[_ptr(t) for t in topk_gate])
    out_arr = (mok_tokens * n_macro)(*[o.c for o in out])
    _check(_lib.mok_moe_forward_batches(C.byref(desc), n_macro, C.cast(idx_arr, C.c_void_p),
                                        C.cast(gate_arr, C.c_void_p), T, C.byref(x.c),
                                        _ptr(w_gate_up), _ptr(w_down), out_arr, _ptr(ws),
                                        ws_bytes, _stream(stream)), "mok_moe_forward_batches")


def mok_tune_forward(desc: mok_layer_desc, minibatches: Sequence[int], n_moves: Sequence[int],
                     reps: int, topk_idx: Sequence, topk_gate: Sequence, T: int, x: Tokens,
                     w_gate_up, w_down, out: Sequence[Tokens], ws, ws_bytes: Optional[int] = None,
                     stream=None):
    """Returns (best descriptor, its mean ms per call)."""
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size()
    n_macro = len(topk_idx)
    mb = (C.c_int32 * len(minibatches))(*minibatches)
    mv = (C.c_int32 * max(len(n_moves), 1))(*(list(n_moves) or [0]))
    idx_arr = (C.c_void_p * n_macro)(*[_ptr(t) for t in topk_idx])
    gate_arr = (C.c_void_p * n_macro)(*[_ptr(t) for t in topk_gate])
    out_arr = (mok_tokens * n_macro)(*[o.c for o in out])
    best = mok_layer_desc()
    ms = C.c_float(0.0)
    _check(_lib.mok_tune_forward(C.byref(desc), mb, len(minibatches), mv, len(n_moves), reps,
                                 n_macro, C.cast(idx_arr, C.c_void_p), C.cast(gate_arr, C.c_void_p),
                                 T, C.byref(x.c), _ptr(w_gate_up), _ptr(w_down), out_arr, _ptr(ws),
                                 ws_bytes, C.byref(best), C.byref(ms), _stream(stream)),
           "mok_tune_forward")
    return best, float(ms.value)


def mok_packed_weights_bwd_size(desc: mok_layer_desc):
    a, b = _SZ(0), _SZ(0)
    _check(_lib.mok_packed_weights_bwd_size(C.byref(desc), C.byref(a), C.byref(b)),
           "mok_packed_weights_bwd_size")
    return int(a.value), int(b.value)


def mok_pack_weights_bwd(desc: mok_layer_desc, w_gate_up, w_down, packed_gate_up_t, packed_down_t,
                         stream=None) -> None:
    _check(_lib.mok_pack_weights_bwd(C.byref(desc), _ptr(w_gate_up), _ptr(w_down),
                                     _ptr(packed_gate_up_t), _ptr(packed_down_t), _stream(stream)),
           "mok_pack_weights_bwd")


def mok_combine_backward(dout: Tokens, y, y_rows: int, assign_of_slot, offsets, n_local: int,
                         n_slots: int, topk_gate, k: int, H: int, dy, dy_rows: int, dgate,
                         dev_status=None, stream=None) -> None:
    _check(_lib.mok_combine_backward(C.byref(dout.c), _ptr(y), y_rows, _ptr(assign_of_slot),
                                     _ptr(offsets), n_local, n_slots, _ptr(topk_gate), k, H,
                                     _ptr(dy), dy_rows, _ptr(dgate), _ptr(dev_status),
                                     _stream(stream)), "mok_combine_backward")


def mok_expert_ffn_backward(desc: mok_layer_desc, ring, ring_slots: int, dy, offsets,
                            slot_begin: int, slot_end: int, w_gate_up, packed_gate_up_t,
                            packed_down_t, h, dh, dx_slots, rows: int, stream=None) -> None:
    _check(_lib.mok_expert_ffn_backward(C.byref(desc), _ptr(ring), ring_slots, _ptr(dy),
                                        _ptr(offsets), slot_begin, slot_end, _ptr(w_gate_up),
                                        _ptr(packed_gate_up_t), _ptr(packed_down_t), _ptr(h),
                                        _ptr(dh), _ptr(dx_slots), rows, _stream(stream)),
           "mok_expert_ffn_backward")


def mok_expert_gate_up_save_h(desc: mok_layer_desc, ring, ring_slots: int, offsets,
                              slot_begin: int, slot_end: int, w_gate_up, act, act_rows: int, h,
                              ws=None, ws_bytes: Optional[int] = None, stream=None) -> None:
    _check(_lib.mok_expert_gate_up_save_h(C.byref(desc), _ptr(ring), ring_slots, _ptr(offsets),
                                          slot_begin, slot_end, _ptr(w_gate_up), _ptr(act),
                                          act_rows, _ptr(h), _ptr(ws), _ws_bytes(ws, ws_bytes),
                                          _stream(stream)),
           "mok_expert_gate_up_save_h")


def mok_expert_ffn_backward_saved(desc: mok_layer_desc, dy, offsets, slot_begin: int,
                                  slot_end: int, packed_gate_up_t, packed_down_t, h, dh, dx_slots,
                                  rows: int, stream=None) -> None:
    _check(_lib.mok_expert_ffn_backward_saved(C.byref(desc), _ptr(dy), _ptr(offsets), slot_begin,
                                              slot_end, _ptr(packed_gate_up_t),
                                              _ptr(packed_down_t), _ptr(h), _ptr(dh),
                                              _ptr(dx_slots), rows, _stream(stream)),
           "mok_expert_ffn_backward_saved")


def mok_wgrad_workspace_size(desc: mok_layer_desc, rows: int) -> int:
    return int(_lib.mok_wgrad_workspace_size(C.byref(desc), rows))


def mok_expert_wgrad(desc: mok_layer_desc, ring, ring_slots: int, act, act_rows: int, dy, dh,
                     rows: int, offsets, dw_gate_up, dw_down, ws, ws_bytes: Optional[int] = None,
                     stream=None) -> None:
    _check(_lib.mok_expert_wgrad(C.byref(desc), _ptr(ring), ring_slots, _ptr(act), act_rows,
                                 _ptr(dy), _ptr(dh), rows, _ptr(offsets), _ptr(dw_gate_up),
                                 _ptr(dw_down), _ptr(ws), _ws_bytes(ws, ws_bytes), _stream(stream)),
           "mok_expert_wgrad")


def mok_dispatch_backward(dx_slots, rows: int, assign_of_slot, offsets, n_local: int, n_slots: int,
                          slot_of_assign, k: int, H: int, dx: Tokens, dev_status=None,
                          stream=None) -> None:
    _check(_lib.mok_dispatch_backward(_ptr(dx_slots), rows, _ptr(assign_of_slot), _ptr(offsets),
                                      n_local, n_slots, _ptr(slot_of_assign), k, H, C.byref(dx.c),
                                      _ptr(dev_status), _stream(stream)), "mok_dispatch_backward")


def mok_expert_down_merge(desc: mok_layer_desc, act, act_scales, act_rows: int, offsets,
                          slot_begin: int, slot_end: int, w_down, y, y_rows: int, assign_of_slot,
                          slot_of_assign, topk_gate, out: Tokens, merge_plan, ws=None,
                          ws_bytes: Optional[int] = None, stream=None) -> None:
    _check(_lib.mok_expert_down_merge(C.byref(desc), _ptr(act), _ptr(act_scales), act_rows,
                                      _ptr(offsets), slot_begin, slot_end, _ptr(w_down), _ptr(y),
                                      y_rows, _ptr(assign_of_slot), _ptr(slot_of_assign),
                                      _ptr(topk_gate), C.byref(out.c), _ptr(merge_plan), _ptr(ws),
                                      _ws_bytes(ws, ws_bytes), _stream(stream)),
           "mok_expert_down_merge")


def mok_combine_slots_multi(y, y_rows: int, assign_of_slot, offsets, n_local: int, n_slots: int,
                            slot_of_assign, topk_gate, k: int, H: int, out: Tokens,
                            dev_status=None, stream=None) -> None:
    _check(_lib.mok_combine_slots_multi(_ptr(y), y_rows, _ptr(assign_of_slot), _ptr(offsets),
                                        n_local, n_slots, _ptr(slot_of_assign), _ptr(topk_gate), k,
                                        H, C.byref(out.c), _ptr(dev_status), _stream(stream)),
           "mok_combine_slots_multi")


def mok_combine_backward_mx(dout: Tokens, y, y_rows: int, assign_of_slot, offsets, n_local: int,
                            n_slots: int, topk_gate, k: int, H: int, dy, dy_scales, dy_rows: int,
                            dgate, dev_status=None, stream=None) -> None:
    _check(_lib.mok_combine_backward_mx(C.byref(dout.c), _ptr(y), y_rows, _ptr(assign_of_slot),
                                        _ptr(offsets), n_local, n_slots, _ptr(topk_gate), k, H,
                                        _ptr(dy), _ptr(dy_scales), dy_rows, _ptr(dgate),
                                        _ptr(dev_status), _stream(stream)),
           "mok_combine_backward_mx")


def mok_expert_gate_up_save_h_mx(desc: mok_layer_desc, ring, ring_scales, ring_slots: int,
                                 offsets, slot_begin: int, slot_end: int, w_gate_up, act,
                                 act_scales, act_rows: int, h, ws=None,
                                 ws_bytes: Optional[int] = None, stream=None) -> None:
    _check(_lib.mok_expert_gate_up_save_h_mx(C.byref(desc), _ptr(ring), _ptr(ring_scales),
                                             ring_slots, _ptr(offsets), slot_begin, slot_end,
                                             _ptr(w_gate_up), _ptr(act), _ptr(act_scales),
                                             act_rows, _ptr(h), _ptr(ws), _ws_bytes(ws, ws_bytes),
                                             _stream(stream)),
           "mok_expert_gate_up_save_h_mx")


def mok_expert_ffn_backward_mx(desc: mok_layer_desc, ring, ring_scales, ring_slots: int, dy,
                               dy_scales, offsets, slot_begin: int, slot_end: int, w_gate_up,
                               packed_gate_up_t, packed_down_t, h, h_kept: bool, dh, dh_scales,
                               dx_slots, rows: int, stream=None) -> None:
    _check(_lib.mok_expert_ffn_backward_mx(C.byref(desc), _ptr(ring), _ptr(ring_scales),
                                           ring_slots, _ptr(dy), _ptr(dy_scales), _ptr(offsets),
                                           slot_begin, slot_end, _ptr(w_gate_up),
                                           _ptr(packed_gate_up_t), _ptr(packed_down_t), _ptr(h),
                                           1 if h_kept else 0, _ptr(dh), _ptr(dh_scales),
                                           _ptr(dx_slots), rows, _stream(stream)),
           "mok_expert_ffn_backward_mx")


def mok_expert_wgrad_mx(desc: mok_layer_desc, ring, ring_scales, ring_slots: int, act,
                        act_scales, act_rows: int, dy, dy_scales, dh, dh_scales, rows: int,
                        offsets, dw_gate_up, dw_down, ws, ws_bytes: Optional[int] = None,
                        stream=None) -> None:
    _check(_lib.mok_expert_wgrad_mx(C.byref(desc), _ptr(ring), _ptr(ring_scales), ring_slots,
                                    _ptr(act), _ptr(act_scales), act_rows, _ptr(dy),
                                    _ptr(dy_scales), _ptr(dh), _ptr(dh_scales), rows,
                                    _ptr(offsets), _ptr(dw_gate_up), _ptr(dw_down), _ptr(ws),
                                    _ws_bytes(ws, ws_bytes), _stream(stream)),
           "mok_expert_wgrad_mx")


def mok_device_status(ws, stream=None) -> int:
    v = C.c_int32(-1)
    _check(_lib.mok_device_status(_ptr(ws), C.byref(v), _stream(stream)), "mok_device_status")
    return int(v.value)
