"""ctypes binding of librawint4_moe.so (include/rawint4_moe.h).

Argument marshalling only: torch tensors are passed as raw device pointers,
every computation happens in the library's CUDA kernels. There is no CPU
fallback: importing this module fails loudly when the library is missing.
"""

from __future__ import annotations

import ctypes
import importlib.util
import os
import warnings
from dataclasses import dataclass
from typing import Dict, Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "librawint4_moe.so")

OK = 0
INVALID_ARGUMENT = 1
FROZEN_BASE = 2
NO_SAVED_FORWARD = 3
CUDA_ERROR = 4
BAD_EXPERT_ID = 5
DEVICE_TIMEOUT = 6
FP16_OVERFLOW = 7
UNSUPPORTED = 8
STATIC_SCRATCH_TOO_SMALL = 9

DEV_BAD_EXPERT_ID = 1 << 0
DEV_NO_SAVED_FORWARD = 1 << 1
DEV_TIMEOUT = 1 << 2
DEV_FP16_OVERFLOW = 1 << 3

EXPORTED_SYMBOLS = (
    "rawint4_moe_lora_workspace_size",
    "rawint4_moe_lora_fwd",
    "rawint4_moe_lora_bwd",
    "rawint4_moe_lora_status",
    "rawint4_moe_lora_strerror",
    "rawint4_decode",
    "rawint4_moe_permute_workspace_size",
    "rawint4_moe_permute",
    "rawint4_moe_profile_begin",
    "rawint4_moe_profile_end",
    "rawint4_moe_permute_static",
    "rawint4_moe_permute_static_max_bytes",
    "rawint4_moe_set_wait_limit_ns",
    "rawint4_moe_lora_saved_preacts",
    "rawint4_moe_router_topk",
    "rawint4_moe_router_bwd",
    "rawint4_mxfp4_decode",
    "rawint4_moe_dispatch_rows",
    "rawint4_moe_combine_slots",
    "rawint4_moe_gather_slots",
    "rawint4_moe_router_select",
    "rawint4_moe_router_select_bwd",
    "rawint4_ckpt8_save",
    "rawint4_ckpt8_load",
    "rawint4_norm_fwd",
    "rawint4_norm_bwd_workspace_size",
    "rawint4_norm_bwd",
)


class Cfg(ctypes.Structure):
    _fields_ = [("experts", ctypes.c_int32), ("top_k", ctypes.c_int32), ("hidden", ctypes.c_int32),
                ("inter", ctypes.c_int32), ("rank", ctypes.c_int32), ("alpha", ctypes.c_float),
                ("swiglu_limit", ctypes.c_float), ("max_tokens", ctypes.c_int32), ("weight_format", ctypes.c_int32)]


class Base(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("gate_q", "up_q", "down_q", "gate_s", "up_s", "down_s")]


class Lora(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("gate_a", "gate_b", "up_a", "up_b", "down_a", "down_b")]


class LoraGrads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("gate_a", "gate_b", "up_a", "up_b", "down_a", "down_b")]


class SelectCfg(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("experts", "top_k", "groups", "groups_kept", "group_top", "score",
                                              "renormalise", "type")] + [("scale", ctypes.c_float)]


class Ckpt8Ptrs(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("format", ctypes.c_int32)]


class NormCfg(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("width", ctypes.c_int32), ("kind", ctypes.c_int32), ("type", ctypes.c_int32),
                ("weight_type", ctypes.c_int32), ("eps", ctypes.c_float)]


class RawInt4Error(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {strerror(code)} (code {code})")


class FrozenBaseError(RawInt4Error, ValueError):
    pass


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m int4_quantised_moe_b200.build` "
            "(the layer has no CPU fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    vp, sz, i32, i64, f32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    P = ctypes.POINTER
    lib.rawint4_moe_lora_workspace_size.argtypes = [P(Cfg), P(sz)]
    lib.rawint4_moe_lora_fwd.argtypes = [P(Cfg), P(Base), P(Lora), i32, vp, vp, vp, vp, ctypes.c_int, vp, sz, vp]
    lib.rawint4_moe_lora_bwd.argtypes = [P(Cfg), P(Base), P(Lora), vp, vp, vp, P(LoraGrads), vp, vp, vp,
                                         ctypes.c_int, f32, vp, sz, vp]
    lib.rawint4_moe_lora_status.argtypes = [vp, vp, P(ctypes.c_uint32)]
    lib.rawint4_moe_lora_strerror.argtypes = [ctypes.c_int]
    lib.rawint4_moe_lora_strerror.restype = ctypes.c_char_p
    lib.rawint4_decode.argtypes = [vp, vp, i64, i64, vp, vp, vp]
    lib.rawint4_moe_permute_workspace_size.argtypes = [i32, i32, i32, P(sz)]
    lib.rawint4_moe_permute.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp, sz, vp]
    lib.rawint4_moe_permute_static.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp]
    lib.rawint4_moe_permute_static_max_bytes.argtypes = []
    lib.rawint4_moe_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
    lib.rawint4_moe_lora_saved_preacts.argtypes = [P(Cfg), vp, sz, vp, vp, vp, P(i32), vp]
    lib.rawint4_moe_router_topk.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp]
    lib.rawint4_moe_router_bwd.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp, vp, vp]
    lib.rawint4_mxfp4_decode.argtypes = [vp, vp, i64, i64, vp, vp, vp]
    lib.rawint4_moe_dispatch_rows.argtypes = [vp, vp, i32, i32, i32, vp, vp]
    lib.rawint4_moe_combine_slots.argtypes = [vp, vp, i32, i32, i32, vp, vp]
    lib.rawint4_moe_gather_slots.argtypes = [vp, vp, i32, vp, vp]
    lib.rawint4_moe_router_select.argtypes = [P(SelectCfg), vp, i64, i32, vp, vp, vp, vp, vp]
    lib.rawint4_moe_router_select_bwd.argtypes = [P(SelectCfg), vp, i64, i32, vp, vp, vp, vp]
    lib.rawint4_ckpt8_save.argtypes = [i32, i32, vp, i64, i64, i32, vp, vp, vp]
    lib.rawint4_ckpt8_load.argtypes = [i32, vp, vp, i64, i32, i32, vp, vp]
    lib.rawint4_norm_fwd.argtypes = [P(NormCfg), vp, i64, P(Ckpt8Ptrs), vp, vp, vp, vp, vp, i32, vp, vp, vp]
    lib.rawint4_norm_bwd_workspace_size.argtypes = [P(NormCfg), P(sz)]
    lib.rawint4_norm_bwd.argtypes = [P(NormCfg), vp, i64, P(Ckpt8Ptrs), vp, i64, vp, vp, vp, vp, vp, vp, ctypes.c_int,
                                     vp, sz, vp]
    for name in EXPORTED_SYMBOLS:
        if name != "rawint4_moe_lora_strerror":
            getattr(lib, name).restype = ctypes.c_int  # raises AttributeError if the library lacks it
    lib.rawint4_moe_permute_static_max_bytes.restype = ctypes.c_size_t
    return lib


_lib = _load()

class _NoFastcall:
    """In the extension's place where there is none: every call is left to the code below."""

    router_select = router_select_bwd = ckpt8_save = ckpt8_load = norm_fwd = norm_bwd = staticmethod(lambda *args: None)


def _load_fastcall():
    """The extension csrc/fastcall.cpp for this Python and torch; without it nothing is lost but the time
    that ctypes takes on the host."""
    from . import build
    path = build.fastcall_path()
    try:
        if not os.path.exists(path):
            raise ImportError(f"{path} is missing")
        spec = importlib.util.spec_from_file_location(f"{__package__}._fastcall", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        return module
    except ImportError as e:
        warnings.warn(f"the quick way into the operators around the layer does not load ({e}); their calls go through "
                      "ctypes, some 10 us longer each. `python -m int4_quantised_moe_b200.build` builds it",
                      RuntimeWarning, stacklevel=3)
        return _NoFastcall


_fast = _load_fastcall()


def library() -> ctypes.CDLL:
    return _lib


def strerror(code: int) -> str:
    return _lib.rawint4_moe_lora_strerror(int(code)).decode()


def _check(code: int, what: str):
    if code == FROZEN_BASE:
        raise FrozenBaseError(code, what)
    if code != OK:
        raise RawInt4Error(code, what)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to the layer must be contiguous")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


FORMAT_RAWINT4 = 0
FORMAT_MXFP4 = 1
FORMATS = {"rawint4": FORMAT_RAWINT4, "mxfp4": FORMAT_MXFP4}


def make_cfg(experts, top_k, hidden, inter, rank, alpha, swiglu_limit, max_tokens, weight_format="rawint4") -> Cfg:
    return Cfg(int(experts), int(top_k), int(hidden), int(inter), int(rank), float(alpha), float(swiglu_limit),
               int(max_tokens), FORMATS[weight_format])


def rawint4_moe_lora_workspace_size(cfg: Cfg) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.rawint4_moe_lora_workspace_size(ctypes.byref(cfg), ctypes.byref(n)), "rawint4_moe_lora_workspace_size")
    return int(n.value)


def make_base(gate_q, gate_s, up_q, up_s, down_q, down_s) -> Base:
    return Base(_ptr(gate_q), _ptr(up_q), _ptr(down_q), _ptr(gate_s), _ptr(up_s), _ptr(down_s))


def make_lora(lora: Dict[str, torch.Tensor]) -> Lora:
    return Lora(*[_ptr(lora[n]) for n in ("gate_lora_a", "gate_lora_b", "up_lora_a", "up_lora_b",
                                          "down_lora_a", "down_lora_b")])


def make_grads(grads: Dict[str, torch.Tensor]) -> LoraGrads:
    return LoraGrads(*[_ptr(grads[n]) for n in ("gate_lora_a", "gate_lora_b", "up_lora_a", "up_lora_b",
                                                "down_lora_a", "down_lora_b")])


def rawint4_moe_lora_fwd(cfg: Cfg, base: Base, lora: Optional[Lora], qlen: int, expert_ids, route_weights, x, out,
                         save_for_backward: bool, workspace: torch.Tensor, stream=None) -> None:
    """lora=None: frozen-base inference forward (save_for_backward must be False)."""
    lora_ref = ctypes.byref(lora) if lora is not None else None
    rc = _lib.rawint4_moe_lora_fwd(ctypes.byref(cfg), ctypes.byref(base), lora_ref, int(qlen),
                                   _ptr(expert_ids), _ptr(route_weights), _ptr(x), _ptr(out),
                                   1 if save_for_backward else 0, _ptr(workspace), workspace.numel(),
                                   _stream(stream))
    _check(rc, "rawint4_moe_lora_fwd")


def rawint4_moe_lora_bwd(cfg: Cfg, base: Base, lora: Lora, grad_out, grad_in, grad_route, grads: LoraGrads,
                         accumulate: bool, grad_scale: float, workspace: torch.Tensor, stream=None,
                         base_grad_gate=None, base_grad_up=None, base_grad_down=None) -> None:
    rc = _lib.rawint4_moe_lora_bwd(ctypes.byref(cfg), ctypes.byref(base), ctypes.byref(lora), _ptr(grad_out),
                                   _ptr(grad_in), _ptr(grad_route), ctypes.byref(grads), _ptr(base_grad_gate),
                                   _ptr(base_grad_up), _ptr(base_grad_down), 1 if accumulate else 0,
                                   float(grad_scale), _ptr(workspace), workspace.numel(), _stream(stream))
    _check(rc, "rawint4_moe_lora_bwd")


def rawint4_moe_lora_status(workspace: torch.Tensor, stream=None) -> int:
    v = ctypes.c_uint32(0)
    _check(_lib.rawint4_moe_lora_status(_ptr(workspace), _stream(stream), ctypes.byref(v)), "rawint4_moe_lora_status")
    return int(v.value)


def rawint4_decode(q: torch.Tensor, s: torch.Tensor, out_f32=None, out_f16=None, stream=None) -> None:
    n, k2 = q.shape[-2], q.shape[-1]
    rows = q.numel() // k2
    _check(_lib.rawint4_decode(_ptr(q), _ptr(s), rows, 2 * k2, _ptr(out_f32), _ptr(out_f16), _stream(stream)),
           "rawint4_decode")


def rawint4_mxfp4_decode(q: torch.Tensor, s: torch.Tensor, out_f32=None, out_f16=None, stream=None) -> None:
    """MXFP4 check decode: q uint8 [N, K/2], s uint8 [N, K/32] -> fp32 and/or fp16 [N, K]."""
    k2 = q.shape[-1]
    rows = q.numel() // k2
    _check(_lib.rawint4_mxfp4_decode(_ptr(q), _ptr(s), rows, 2 * k2, _ptr(out_f32), _ptr(out_f16), _stream(stream)),
           "rawint4_mxfp4_decode")


def rawint4_moe_permute(expert_ids: torch.Tensor, experts: int, offsets, perm, inv, stream=None) -> None:
    q, k = expert_ids.shape
    n = ctypes.c_size_t(0)
    _check(_lib.rawint4_moe_permute_workspace_size(q, k, experts, ctypes.byref(n)), "permute_workspace_size")
    ws = torch.empty(max(int(n.value), 256), dtype=torch.uint8, device=expert_ids.device)
    _check(_lib.rawint4_moe_permute(_ptr(expert_ids), q, k, experts, _ptr(offsets), _ptr(perm), _ptr(inv),
                                    _ptr(ws), ws.numel(), _stream(stream)), "rawint4_moe_permute")


def rawint4_moe_permute_static(expert_ids: torch.Tensor, experts: int, offsets, perm, inv, stream=None) -> None:
    """rawint4_moe_permute without caller scratch: for callers that cannot
    allocate device memory; uses the library's fixed 1 MiB device array."""
    q, k = expert_ids.shape
    _check(_lib.rawint4_moe_permute_static(_ptr(expert_ids), q, k, experts, _ptr(offsets), _ptr(perm), _ptr(inv),
                                           _stream(stream)), "rawint4_moe_permute_static")


def rawint4_moe_permute_static_max_bytes() -> int:
    return int(_lib.rawint4_moe_permute_static_max_bytes())


def rawint4_moe_dispatch_rows(src: torch.Tensor, perm: torch.Tensor, n: int, top_k: int, dst: torch.Tensor,
                              stream=None) -> None:
    """dst[p] = src[perm[p] // top_k] for p < n (bf16 rows)."""
    _require(src, torch.bfloat16, src.device, "src")
    _require(dst, torch.bfloat16, src.device, "dst")
    _require(perm, torch.int32, src.device, "perm")
    if dst.shape[0] < n or dst.shape[1] != src.shape[1] or perm.numel() < n:
        raise ValueError("dispatch_rows: dst must hold n rows of src's width and perm n entries")
    _check(_lib.rawint4_moe_dispatch_rows(_ptr(src), _ptr(perm), int(n), int(top_k), src.shape[1], _ptr(dst),
                                          _stream(stream)), "rawint4_moe_dispatch_rows")


def rawint4_moe_combine_slots(src: torch.Tensor, inv: torch.Tensor, qlen: int, top_k: int, out: torch.Tensor,
                              stream=None) -> None:
    """out[t] = bf16(sum over s of src[inv[t * top_k + s]]) in slot order (fp32 sums)."""
    _require(out, torch.bfloat16, out.device, "out")
    _require(inv, torch.int32, out.device, "inv")
    if src.numel():
        _require(src, torch.bfloat16, out.device, "src")
        if src.shape[1] != out.shape[1]:
            raise ValueError("combine_slots: src and out widths differ")
    if out.shape[0] < qlen or inv.numel() < qlen * top_k:
        raise ValueError("combine_slots: out needs qlen rows and inv qlen * top_k entries")
    _check(_lib.rawint4_moe_combine_slots(_ptr(src) if src.numel() else None, _ptr(inv), int(qlen), int(top_k),
                                          out.shape[1], _ptr(out), _stream(stream)), "rawint4_moe_combine_slots")


def rawint4_moe_gather_slots(src: torch.Tensor, inv: torch.Tensor, out: torch.Tensor, stream=None) -> None:
    """out[f] = src[inv[f]] where inv[f] >= 0, else 0 (fp32)."""
    _require(out, torch.float32, out.device, "out")
    _require(inv, torch.int32, out.device, "inv")
    if src.numel():
        _require(src, torch.float32, out.device, "src")
    if inv.numel() < out.numel():
        raise ValueError("gather_slots: inv needs one entry per output")
    _check(_lib.rawint4_moe_gather_slots(_ptr(src) if src.numel() else None, _ptr(inv), out.numel(), _ptr(out),
                                         _stream(stream)), "rawint4_moe_gather_slots")


# ---------------------------------------------------------------------------
# Convenience holder used by tests and the bench: keeps the layer's tensors
# and one workspace together and calls the two entry points.
# ---------------------------------------------------------------------------

def _require(t, dtype: torch.dtype, device: torch.device, name: str) -> None:
    """Like _expect, without a fixed shape."""
    _expect(t, name, dtype, tuple(t.shape) if isinstance(t, torch.Tensor) else (), device)


def _expect(t, name: str, dtype: torch.dtype, shape: tuple, device: Optional[torch.device] = None) -> None:
    """Host-side argument check: the C ABI sees raw pointers only, so a wrong
    dtype, shape, device or layout is caught here with a readable message."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected dtype {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor, got one on {t.device}")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: expected a tensor on {device}, got one on {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: tensors passed to the layer must be contiguous")


LORA_TENSOR_NAMES = ("gate_lora_a", "gate_lora_b", "up_lora_a", "up_lora_b", "down_lora_a", "down_lora_b")


def lora_tensor_shapes(experts: int, hidden: int, inter: int, rank: int) -> Dict[str, tuple]:
    """Shapes of the six LoRA tensors (and of their gradient buffers)."""
    E, H, I, r = experts, hidden, inter, rank
    return {"gate_lora_a": (E, r, H), "gate_lora_b": (E, I, r), "up_lora_a": (E, r, H), "up_lora_b": (E, I, r),
            "down_lora_a": (E, r, I), "down_lora_b": (E, H, r)}

@dataclass
class Layer:
    cfg: Cfg
    base: Base
    lora: Lora
    workspace: torch.Tensor
    keep: tuple  # tensors whose pointers live in base/lora
    passes: int = 0  # forwards and backwards so far: each replaces or consumes the saved context

    @classmethod
    def create(cls, experts, top_k, hidden, inter, rank, alpha, swiglu_limit, max_tokens, gate_q, gate_s, up_q, up_s,
               down_q, down_s, lora: Dict[str, torch.Tensor], device=None, weight_format="rawint4"):
        """weight_format "rawint4" (bf16 scales) or "mxfp4" (E2M1 codes, UE8M0 scale bytes, uint8)."""
        cfg = make_cfg(experts, top_k, hidden, inter, rank, alpha, swiglu_limit, max_tokens, weight_format)
        nbytes = rawint4_moe_lora_workspace_size(cfg)  # validates the configuration
        dev = device if device is not None else gate_q.device
        E, H, I = int(experts), int(hidden), int(inter)
        sdt = torch.uint8 if weight_format == "mxfp4" else torch.bfloat16
        for name, t, dt, shape in (("gate_q", gate_q, torch.uint8, (E, I, H // 2)),
                                   ("up_q", up_q, torch.uint8, (E, I, H // 2)),
                                   ("down_q", down_q, torch.uint8, (E, H, I // 2)),
                                   ("gate_s", gate_s, sdt, (E, I, H // 32)),
                                   ("up_s", up_s, sdt, (E, I, H // 32)),
                                   ("down_s", down_s, sdt, (E, H, I // 32))):
            _expect(t, name, dt, shape, gate_q.device)
        for name, shape in lora_tensor_shapes(E, H, I, int(rank)).items():
            if name not in lora:
                raise KeyError(f"lora: missing {name}")
            _expect(lora[name], name, torch.bfloat16, shape, gate_q.device)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        ws[:256].zero_()
        base = make_base(gate_q, gate_s, up_q, up_s, down_q, down_s)
        lo = make_lora(lora)
        return cls(cfg, base, lo, ws, (gate_q, gate_s, up_q, up_s, down_q, down_s, dict(lora)))

    def forward(self, expert_ids, route_weights, x, out=None, save_for_backward=True, stream=None, use_lora=True):
        """use_lora=False: frozen-base inference forward (no LoRA terms, nothing saved)."""
        q, k, H = x.shape[0] if x.dim() == 2 else -1, self.cfg.top_k, self.cfg.hidden
        dev = self.workspace.device
        _expect(x, "x", torch.bfloat16, (q, H), dev)
        _expect(expert_ids, "expert_ids", torch.int64, (q, k), dev)
        _expect(route_weights, "route_weights", torch.float32, (q, k), dev)
        if out is None:
            out = torch.empty_like(x)
        _expect(out, "out", torch.bfloat16, (q, H), dev)
        rawint4_moe_lora_fwd(self.cfg, self.base, self.lora if use_lora else None, q, expert_ids, route_weights, x,
                             out, save_for_backward, self.workspace, stream)
        self.passes += 1  # a refused call leaves the context as it was
        return out

    def backward(self, grad_out, grads: Dict[str, torch.Tensor], accumulate=False, grad_scale=1.0, grad_in=None,
                 grad_route=None, stream=None, **base_grads):
        dev = self.workspace.device
        q, k, H = grad_out.shape[0] if grad_out.dim() == 2 else -1, self.cfg.top_k, self.cfg.hidden
        _expect(grad_out, "grad_out", torch.bfloat16, (q, H), dev)
        if grad_in is None:
            grad_in = torch.empty_like(grad_out)
        _expect(grad_in, "grad_in", torch.bfloat16, (q, H), dev)
        if grad_route is not None:
            _expect(grad_route, "grad_route", torch.float32, (q, k), dev)
        c = self.cfg
        for name, shape in lora_tensor_shapes(c.experts, c.hidden, c.inter, c.rank).items():
            if name not in grads:
                raise KeyError(f"grads: missing {name}")
            _expect(grads[name], f"grads[{name}]", torch.bfloat16, shape, dev)
        rawint4_moe_lora_bwd(self.cfg, self.base, self.lora, grad_out, grad_in, grad_route, make_grads(grads),
                             accumulate, grad_scale, self.workspace, stream, **base_grads)
        self.passes += 1
        return grad_in

    def status(self, stream=None) -> int:
        return rawint4_moe_lora_status(self.workspace, stream)

    def saved_preacts(self, stream=None):
        """(perm int32 [R], G fp32 [R, I], U fp32 [R, I]) of the pending saved
        forward, R = routed rows (test export; see include/rawint4_moe.h)."""
        c = self.cfg
        rows = int(c.max_tokens) * int(c.top_k)
        dev = self.workspace.device
        perm = torch.empty(rows, dtype=torch.int32, device=dev)
        g = torch.empty((rows, int(c.inter)), dtype=torch.float32, device=dev)
        u = torch.empty_like(g)
        routed = ctypes.c_int32(0)
        rc = _lib.rawint4_moe_lora_saved_preacts(ctypes.byref(self.cfg), _ptr(self.workspace), self.workspace.numel(),
                                                 _ptr(perm), _ptr(g), _ptr(u), ctypes.byref(routed), _stream(stream))
        _check(rc, "rawint4_moe_lora_saved_preacts")
        n = int(routed.value)
        return perm[:n], g[:n], u[:n]


# ---------------------------------------------------------------------------
# Timing hook (measurement only)
# ---------------------------------------------------------------------------

def router_topk(scores: torch.Tensor, top_k: int, escale: Optional[torch.Tensor] = None, stream=None):
    """Expert ids int64 [Q, k] and route weights fp32 [Q, k] from router scores fp32 [Q, E]
    (softmax, top-k, renormalised, times the per-expert scale)."""
    q, E = scores.shape
    _expect(scores, "scores", torch.float32, (q, E))
    if escale is not None:
        _expect(escale, "escale", torch.float32, (E,), scores.device)
    ids = torch.empty((q, int(top_k)), dtype=torch.int64, device=scores.device)
    w = torch.empty((q, int(top_k)), dtype=torch.float32, device=scores.device)
    _check(_lib.rawint4_moe_router_topk(_ptr(scores), q, E, int(top_k), _ptr(escale), _ptr(ids), _ptr(w),
                                        _stream(stream)), "rawint4_moe_router_topk")
    return ids, w


def router_bwd(scores: torch.Tensor, ids: torch.Tensor, grad_route: torch.Tensor, escale: Optional[torch.Tensor] = None,
               want_escale_grad: bool = False, stream=None):
    """dL/dscores fp32 [Q, E] (and dL/descale fp32 [E]) from the layer's grad_route."""
    q, E = scores.shape
    k = ids.shape[1] if ids.dim() == 2 else -1
    _expect(scores, "scores", torch.float32, (q, E))
    _expect(ids, "ids", torch.int64, (q, k), scores.device)
    _expect(grad_route, "grad_route", torch.float32, (q, k), scores.device)
    if escale is not None:
        _expect(escale, "escale", torch.float32, (E,), scores.device)
    dz = torch.empty_like(scores)
    dc = torch.empty(E, dtype=torch.float32, device=scores.device) if want_escale_grad else None
    _check(_lib.rawint4_moe_router_bwd(_ptr(scores), q, E, k, _ptr(ids), _ptr(grad_route), _ptr(escale), _ptr(dz),
                                       _ptr(dc), _stream(stream)), "rawint4_moe_router_bwd")
    return (dz, dc) if want_escale_grad else dz


# ---------------------------------------------------------------------------
# Around the layer: expert selection, 8-bit activation checkpoints, norm
# ---------------------------------------------------------------------------
# Every call runs on the device of its tensors, on `stream` or that device's
# current stream. Results and scratch are allocated on the stream that the call
# runs on; tensors passed to a call on another stream are recorded there, so
# they may be dropped at once. Using a result on a third stream is ordered by
# the caller, as with any torch operation.
#
# The ordinary call (right arguments, current device and stream) is made by the
# extension of csrc/fastcall.cpp; it answers None to every other one, which is
# then checked and made here. Without the extension all calls are made here.

TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
SCORES = {"softmax": 0, "sigmoid": 1}
CKPT_FORMATS = {"e4m3": 0, "int8": 1}
NORM_KINDS = {"layer": 0, "rms": 1}
CKPT_GROUP = 32  # columns under one scale of a checkpoint
_INT32_MAX = (1 << 31) - 1  # sizes travel as int32; the library has lower limits of its own


def _elsewhere(device: torch.device, stream, *tensors):
    """The context in which a call has to be made again, or None when it can run right here: on the
    current device and its current stream."""
    if stream is None:
        return None if device.index == torch._C._cuda_getDevice() else torch.cuda.device(device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on {device}")
    if device.index == torch._C._cuda_getDevice() and stream.cuda_stream == _here(device):
        return None
    for t in tensors:
        if isinstance(t, Ckpt8):
            t.codes.record_stream(stream)
            t.scales.record_stream(stream)
        elif t is not None:
            t.record_stream(stream)
    return torch.cuda.stream(stream)


def _here(device: torch.device) -> int:
    """Handle of the device's current stream."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _choice(table: dict, value, name: str) -> int:
    code = table.get(value)
    if code is None:
        raise ValueError(f"{name}: expected one of {sorted(map(str, table))}, got {value!r}")
    return code


def _rows(t, name: str, width: Optional[int] = None, device: Optional[torch.device] = None, dtype=None) -> int:
    """Checks a [rows, width] CUDA tensor of fp32, bf16 or fp16 whose rows are dense (any row pitch of
    at least the width); returns the pitch."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype not in TYPES or (dtype is not None and t.dtype != dtype):
        raise TypeError(f"{name}: expected dtype {dtype or 'float32, bfloat16 or float16'}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 2 or (width is not None and shape[1] != width):
        raise ValueError(f"{name}: expected shape [rows, {'width' if width is None else width}], got {tuple(shape)}")
    if max(shape) > _INT32_MAX:
        raise ValueError(f"{name}: shape {tuple(shape)} has a size above {_INT32_MAX}")
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor, got one on {t.device}")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: expected a tensor on {device}, got one on {t.device}")
    pitch, inner = t.stride()
    if shape[0] <= 1:
        pitch = shape[1]  # torch leaves the pitch of a single row open
    if (inner != 1 and shape[1] > 1) or pitch < shape[1]:
        raise ValueError(f"{name}: expected dense rows (strides (pitch >= width, 1)), got strides {t.stride()}")
    return pitch


def make_select_cfg(experts: int, top_k: int, score: str = "sigmoid", groups: int = 1, groups_kept: Optional[int] = None,
                    group_top: int = 1, renormalise: bool = True, scale: float = 1.0) -> SelectCfg:
    """Configuration of router_select: `score` "sigmoid" or "softmax"; `groups` equal runs of experts of
    which the groups_kept (default: all) of largest score, the sum of their group_top best keys, stay in."""
    return SelectCfg(int(experts), int(top_k), int(groups), int(groups if groups_kept is None else groups_kept),
                     int(group_top), _choice(SCORES, score, "score"), 1 if renormalise else 0, 0, float(scale))


def _typed(cfg: SelectCfg, dtype: torch.dtype) -> SelectCfg:
    return SelectCfg(cfg.experts, cfg.top_k, cfg.groups, cfg.groups_kept, cfg.group_top, cfg.score, cfg.renormalise,
                     TYPES[dtype], cfg.scale)


def router_select(scores: torch.Tensor, cfg: SelectCfg, bias: Optional[torch.Tensor] = None,
                  counts: Optional[torch.Tensor] = None, stream=None):
    """Expert ids int64 [Q, k] and route weights fp32 [Q, k] from router scores [Q, E] (fp32, bf16 or
    fp16): sigmoid or softmax, a balance bias fp32 [E] that ranks only, groups, top-k, optionally
    renormalised, times cfg.scale. `counts` int32 [E] (optional, overwritten) receives the slots routed
    to each expert."""
    if stream is None:
        r = _fast.router_select(scores, cfg, bias, counts)
        if r is not None:
            return r if type(r) is tuple else _check(r, "rawint4_moe_router_select")
    E = cfg.experts
    pitch = _rows(scores, "scores", E)
    dev = scores.device
    if bias is not None:
        _expect(bias, "bias", torch.float32, (E,), dev)
    if counts is not None:
        _expect(counts, "counts", torch.int32, (E,), dev)
    ctx = _elsewhere(dev, stream, scores, bias, counts)
    if ctx is not None:
        with ctx:
            return router_select(scores, cfg, bias, counts)
    q = scores.shape[0]
    ids = scores.new_empty((q, cfg.top_k), dtype=torch.int64)
    w = scores.new_empty((q, cfg.top_k), dtype=torch.float32)
    _check(_lib.rawint4_moe_router_select(_typed(cfg, scores.dtype), scores.data_ptr(), pitch, q,
                                          None if bias is None else bias.data_ptr(), ids.data_ptr(), w.data_ptr(),
                                          None if counts is None else counts.data_ptr(), _here(dev)),
           "rawint4_moe_router_select")
    return ids, w


def router_select_bwd(scores: torch.Tensor, cfg: SelectCfg, ids: torch.Tensor, grad_route: torch.Tensor,
                      stream=None) -> torch.Tensor:
    """dL/dscores [Q, E] in the scores' type from the layer's grad_route fp32 [Q, k]."""
    if stream is None:
        r = _fast.router_select_bwd(scores, cfg, ids, grad_route)
        if r is not None:
            return _check(r, "rawint4_moe_router_select_bwd") if type(r) is int else r
    pitch = _rows(scores, "scores", cfg.experts)
    dev = scores.device
    q = scores.shape[0]
    _expect(ids, "ids", torch.int64, (q, cfg.top_k), dev)
    _expect(grad_route, "grad_route", torch.float32, (q, cfg.top_k), dev)
    ctx = _elsewhere(dev, stream, scores, ids, grad_route)
    if ctx is not None:
        with ctx:
            return router_select_bwd(scores, cfg, ids, grad_route)
    grad = scores.new_empty((q, cfg.experts))
    _check(_lib.rawint4_moe_router_select_bwd(_typed(cfg, scores.dtype), scores.data_ptr(), pitch, q, ids.data_ptr(),
                                              grad_route.data_ptr(), grad.data_ptr(), _here(dev)),
           "rawint4_moe_router_select_bwd")
    return grad


@dataclass
class Ckpt8:
    """Rows kept in 8 bits: codes uint8 [rows, width], one scale byte per 32 columns uint8
    [rows, ceil(width / 32)], format "e4m3" or "int8"."""

    codes: torch.Tensor
    scales: torch.Tensor
    format: str

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel()

    def check(self, name: str, device: Optional[torch.device] = None) -> int:
        """Raises unless the tensors fit together; returns the format's number."""
        fmt = _choice(CKPT_FORMATS, self.format, f"{name}.format")
        codes = self.codes
        if not isinstance(codes, torch.Tensor) or codes.dim() != 2:
            raise ValueError(f"{name}.codes: expected a uint8 tensor [rows, width]")
        rows, width = codes.shape
        if max(rows, width) > _INT32_MAX:
            raise ValueError(f"{name}.codes: shape {tuple(codes.shape)} has a size above {_INT32_MAX}")
        _expect(codes, f"{name}.codes", torch.uint8, (rows, width), device)
        _expect(self.scales, f"{name}.scales", torch.uint8, (rows, -(-width // CKPT_GROUP)), codes.device)
        return fmt


def _empty_ckpt8(x: torch.Tensor, fmt: str) -> Ckpt8:
    rows, width = x.shape
    return Ckpt8(x.new_empty((rows, width), dtype=torch.uint8),
                 x.new_empty((rows, -(-width // CKPT_GROUP)), dtype=torch.uint8), fmt)


def ckpt8_save(x: torch.Tensor, format: str = "e4m3", stream=None) -> Ckpt8:
    """x [rows, width] (fp32, bf16 or fp16) in 8 bits; see include/rawint4_moe.h for the format."""
    fmt = _choice(CKPT_FORMATS, format, "format")
    if stream is None:
        r = _fast.ckpt8_save(x, fmt)
        if r is not None:
            return Ckpt8(r[0], r[1], format) if type(r) is tuple else _check(r, "rawint4_ckpt8_save")
    pitch = _rows(x, "x")
    ctx = _elsewhere(x.device, stream, x)
    if ctx is not None:
        with ctx:
            return ckpt8_save(x, format)
    rows, width = x.shape
    out = _empty_ckpt8(x, format)
    _check(_lib.rawint4_ckpt8_save(fmt, TYPES[x.dtype], x.data_ptr(), pitch, rows, width, out.codes.data_ptr(),
                                   out.scales.data_ptr(), _here(x.device)), "rawint4_ckpt8_save")
    return out


def ckpt8_load(ckpt: Ckpt8, dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """The rows of a checkpoint, [rows, width] in `dtype`."""
    if stream is None and ckpt.format in CKPT_FORMATS:
        r = _fast.ckpt8_load(ckpt.codes, ckpt.scales, CKPT_FORMATS[ckpt.format], dtype)
        if r is not None:
            return _check(r, "rawint4_ckpt8_load") if type(r) is int else r
    fmt = ckpt.check("ckpt")
    typ = _choice(TYPES, dtype, "dtype")
    codes = ckpt.codes
    ctx = _elsewhere(codes.device, stream, ckpt)
    if ctx is not None:
        with ctx:
            return ckpt8_load(ckpt, dtype)
    rows, width = codes.shape
    out = codes.new_empty((rows, width), dtype=dtype)
    _check(_lib.rawint4_ckpt8_load(fmt, codes.data_ptr(), ckpt.scales.data_ptr(), rows, width, typ, out.data_ptr(),
                                   _here(codes.device)), "rawint4_ckpt8_load")
    return out


def _fast_input(x) -> tuple:
    """(x, codes, scales, format) for the extension."""
    if isinstance(x, Ckpt8):
        return None, x.codes, x.scales, CKPT_FORMATS.get(x.format, -1)
    return x, None, None, 0


def _norm_input(x, name: str):
    """(rows, width, device, pointer, pitch, checkpoint pointers) of a norm's input."""
    if isinstance(x, Ckpt8):
        fmt = x.check(name)
        rows, width = x.codes.shape
        return rows, width, x.codes.device, None, 0, Ckpt8Ptrs(x.codes.data_ptr(), x.scales.data_ptr(), fmt)
    pitch = _rows(x, name)
    return x.shape[0], x.shape[1], x.device, x.data_ptr(), pitch, None


def _vector(t, name: str, width: int, device: torch.device) -> None:
    if not isinstance(t, torch.Tensor) or t.dtype not in TYPES:
        raise TypeError(f"{name}: expected a float32, bfloat16 or float16 tensor")
    _expect(t, name, t.dtype, (width,), device)


def norm_fwd(x, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None, kind: str = "rms",
             eps: float = 1e-6, dtype: Optional[torch.dtype] = None, save: Optional[str] = None, stream=None):
    """Layer or RMS norm of the rows of x, a tensor [rows, width] or a Ckpt8 (then `dtype` is the
    result's type, bf16 by default). Returns (y, mean, rstd, ckpt): mean is None for kind "rms", ckpt is
    x in 8 bits when `save` names a format, else None."""
    if stream is None and kind in NORM_KINDS and (save is None or save in CKPT_FORMATS):
        r = _fast.norm_fwd(*_fast_input(x), weight, bias, NORM_KINDS[kind], eps, dtype,
                           -1 if save is None else CKPT_FORMATS[save])
        if r is not None:
            if type(r) is int:
                _check(r, "rawint4_norm_fwd")
            return r[0], r[1], r[2], None if save is None else Ckpt8(r[3], r[4], save)
    rows, width, dev, ptr, pitch, ck = _norm_input(x, "x")
    k = _choice(NORM_KINDS, kind, "kind")
    if ck is None:
        if dtype is not None and dtype != x.dtype:
            raise TypeError(f"dtype: a tensor's norm has its type {x.dtype}, got {dtype}")
        dtype = x.dtype
    elif save is not None:
        raise ValueError("save: the input is a checkpoint already")
    elif dtype is None:
        dtype = torch.bfloat16
    typ = _choice(TYPES, dtype, "dtype")
    fmt = 0 if save is None else _choice(CKPT_FORMATS, save, "save")
    wdtype = dtype
    if weight is not None:
        _vector(weight, "weight", width, dev)
        wdtype = weight.dtype
    if bias is not None:
        if weight is None:
            wdtype = bias.dtype
        _vector(bias, "bias", width, dev)
        _expect(bias, "bias", wdtype, (width,), dev)
    ctx = _elsewhere(dev, stream, x, weight, bias)
    if ctx is not None:
        with ctx:
            return norm_fwd(x, weight, bias, kind, eps, dtype, save)
    like = x if ck is None else x.codes
    y = like.new_empty((rows, width), dtype=dtype)
    rstd = like.new_empty(rows, dtype=torch.float32)
    mean = like.new_empty(rows, dtype=torch.float32) if kind == "layer" else None
    out = None if save is None else _empty_ckpt8(x, save)
    _check(_lib.rawint4_norm_fwd(NormCfg(rows, width, k, typ, TYPES[wdtype], eps), ptr, pitch, ck, _ptr(weight),
                                 _ptr(bias), y.data_ptr(), _ptr(mean), rstd.data_ptr(), fmt,
                                 None if out is None else out.codes.data_ptr(),
                                 None if out is None else out.scales.data_ptr(), _here(dev)), "rawint4_norm_fwd")
    return y, mean, rstd, out


def norm_bwd(grad_y: torch.Tensor, x, rstd: torch.Tensor, weight: Optional[torch.Tensor] = None,
             mean: Optional[torch.Tensor] = None, kind: str = "rms", bias_grad: bool = False,
             grad_weight: Optional[torch.Tensor] = None, grad_bias: Optional[torch.Tensor] = None,
             accumulate: bool = False, stream=None):
    """Backward of norm_fwd from its input x (a tensor, or the Ckpt8 kept in its place) and statistics.
    Returns (grad_x, grad_weight, grad_bias) in the types of grad_y and of the weight; grad_weight is None
    without a weight, grad_bias unless it is asked for. Buffers may be given; accumulate=True adds to them."""
    if stream is None and kind in NORM_KINDS:
        r = _fast.norm_bwd(*_fast_input(x), grad_y, rstd, weight, mean, NORM_KINDS[kind], bias_grad, grad_weight,
                           grad_bias, accumulate)
        if r is not None:
            return r if type(r) is tuple else _check(r, "rawint4_norm_bwd")
    rows, width, dev, ptr, pitch, ck = _norm_input(x, "x")
    k = _choice(NORM_KINDS, kind, "kind")
    gpitch = _rows(grad_y, "grad_y", width, dev, None if ck is not None else x.dtype)
    if grad_y.shape[0] != rows:
        raise ValueError(f"grad_y: expected {rows} rows, got {grad_y.shape[0]}")
    _expect(rstd, "rstd", torch.float32, (rows,), dev)
    if kind == "layer":
        _expect(mean, "mean", torch.float32, (rows,), dev)
    elif mean is not None:
        raise ValueError("mean: the RMS norm has none")
    dtype = grad_y.dtype
    wdtype = dtype
    if weight is not None:
        _vector(weight, "weight", width, dev)
        wdtype = weight.dtype
    elif grad_weight is not None:
        raise ValueError("grad_weight: the norm has no weight")
    elif grad_bias is not None:
        _vector(grad_bias, "grad_bias", width, dev)
        wdtype = grad_bias.dtype
    if accumulate and ((weight is not None and grad_weight is None) or (bias_grad and grad_bias is None)):
        raise ValueError("accumulate: needs the buffers to add to")
    if grad_weight is not None:
        _expect(grad_weight, "grad_weight", wdtype, (width,), dev)
    if grad_bias is not None:
        _expect(grad_bias, "grad_bias", wdtype, (width,), dev)
    ctx = _elsewhere(dev, stream, grad_y, x, rstd, weight, mean, grad_weight, grad_bias)
    if ctx is not None:
        with ctx:
            return norm_bwd(grad_y, x, rstd, weight, mean, kind, bias_grad, grad_weight, grad_bias, accumulate)
    grad_x = grad_y.new_empty((rows, width))
    if weight is not None and grad_weight is None:
        grad_weight = grad_y.new_empty(width, dtype=wdtype)
    if bias_grad and grad_bias is None:
        grad_bias = grad_y.new_empty(width, dtype=wdtype)
    cfg = NormCfg(rows, width, k, TYPES[dtype], TYPES[wdtype], 1.0)  # eps is in rstd already
    ws, nbytes = None, 0
    if grad_weight is not None or grad_bias is not None:
        n = ctypes.c_size_t(0)
        _check(_lib.rawint4_norm_bwd_workspace_size(cfg, n), "rawint4_norm_bwd_workspace_size")
        nbytes = n.value
        ws = grad_y.new_empty(nbytes, dtype=torch.uint8)
    _check(_lib.rawint4_norm_bwd(cfg, ptr, pitch, ck, grad_y.data_ptr(), gpitch, _ptr(weight), _ptr(mean),
                                 rstd.data_ptr(), grad_x.data_ptr(), _ptr(grad_weight), _ptr(grad_bias),
                                 1 if accumulate else 0, _ptr(ws), nbytes, _here(dev)), "rawint4_norm_bwd")
    return grad_x, grad_weight, grad_bias


def set_wait_limit_ns(ns: int) -> None:
    """Bound on every pipeline wait of the GEMM kernels launched from now on
    (0 restores the default of 4 s); see include/rawint4_moe.h."""
    _check(_lib.rawint4_moe_set_wait_limit_ns(int(ns)), "rawint4_moe_set_wait_limit_ns")


def profile_begin(max_launches: int = 4096) -> None:
    _lib.rawint4_moe_profile_begin.argtypes = [ctypes.c_int]
    _lib.rawint4_moe_profile_begin.restype = ctypes.c_int
    _check(_lib.rawint4_moe_profile_begin(int(max_launches)), "rawint4_moe_profile_begin")


def profile_end(max_out: int = 4096):
    """Per launch in issue order: (kernel name, milliseconds)."""
    _lib.rawint4_moe_profile_end.argtypes = [ctypes.c_int, ctypes.POINTER(ctypes.c_int),
                                             ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(ctypes.c_float)]
    _lib.rawint4_moe_profile_end.restype = ctypes.c_int
    n = ctypes.c_int(0)
    names = (ctypes.c_char_p * max_out)()
    ms = (ctypes.c_float * max_out)()
    _check(_lib.rawint4_moe_profile_end(max_out, ctypes.byref(n), names, ms), "rawint4_moe_profile_end")
    return [(names[i].decode(), float(ms[i])) for i in range(min(n.value, max_out))]
