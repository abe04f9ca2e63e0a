"""Python binding of libmoe_gb300.so (ctypes).

Argument marshalling only: torch supplies device memory and the stream, every
step of the layer runs in the library's CUDA kernels.  There is no fallback:
when the library is missing or the device is not a CUDA GPU the calls raise.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import re
import sys
from typing import Optional, Tuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_gb300.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "moe.h")

(MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_CUDA, MOE_ERR_DEVICE_TIMEOUT,
 MOE_ERR_DEVICE_RANGE, MOE_ERR_DEVICE_INDEX, MOE_ERR_DEVICE_POOL) = range(9)
SCORE_SOFTMAX, SCORE_SIGMOID, SCORE_SQRTSOFTPLUS = 0, 1, 2
# the workspace's start gate (include/moe.h) and the info word of its timeout
WS_HOLD_OFFSET = 8
INFO_HOLD = 15
# the status block at a workspace's start, and the info words of an index
# outside its table (include/moe.h)
STATUS_BYTES = 256
INFO_POSITION, INFO_SLOT, INFO_PAGE, INFO_LENGTH, INFO_STARTS = 17, 18, 19, 20, 21
INFO_KV_RANGE, INFO_FORK, INFO_KEEP, INFO_POOL = 30, 31, 32, 33
DTYPE_BF16, DTYPE_F16 = 0, 1
# routed-expert formats of the block-scaled path
FMT_FP4, FMT_FP8 = 1, 2


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


class Recipe(ctypes.Structure):
    """Mirror of ``moe_recipe`` in include/moe.h."""

    _fields_ = [
        ("num_experts", ctypes.c_int32),
        ("top_k", ctypes.c_int32),
        ("score_fn", ctypes.c_int32),
        ("n_group", ctypes.c_int32),
        ("topk_group", ctypes.c_int32),
        ("group_topn", ctypes.c_int32),
        ("norm_topk_prob", ctypes.c_int32),
        ("norm_eps", ctypes.c_float),
        ("route_scale", ctypes.c_float),
        ("swiglu_limit", ctypes.c_float),
    ]

    @classmethod
    def make(cls, num_experts, top_k, score_fn=SCORE_SOFTMAX, n_group=1, topk_group=1, group_topn=2,
             norm_topk_prob=True, norm_eps=1e-20, route_scale=1.0, swiglu_limit=0.0) -> "Recipe":
        return cls(num_experts, top_k, score_fn, n_group, topk_group if n_group > 1 else 1, group_topn,
                   1 if norm_topk_prob else 0, norm_eps, route_scale, swiglu_limit)

    @classmethod
    def from_config(cls, cfg) -> "Recipe":
        """From a ``synthetic.LayerConfig``."""
        return cls.make(cfg.E, cfg.K, cfg.score_fn, cfg.n_group, cfg.topk_group, cfg.group_topn,
                        cfg.norm_topk_prob, cfg.norm_eps, cfg.route_scale, cfg.swiglu_limit)


_lib_handle: Optional[ctypes.CDLL] = None

_P = ctypes.c_void_p
_I = ctypes.c_int
_SZ = ctypes.c_size_t
_L = ctypes.c_longlong
_F = ctypes.c_float
_SIGS = {
    "moe_status_string": (ctypes.c_char_p, [_I]),
    "moe_route_workspace_bytes": (_SZ, [_I, _I]),
    "moe_route": (_I, [_P, _I, _I, _P, _P, _P, ctypes.POINTER(Recipe), _P, _P, _P, _P, _SZ, _P]),
    "moe_route_noalloc": (_I, [_P, _I, _I, _P, _P, _P, ctypes.POINTER(Recipe), _P, _P, _P, _P]),
    "moe_route_from_logits": (_I, [_P, _I, _P, ctypes.POINTER(Recipe), _P, _P, _P]),
    "moe_permute": (_I, [_P, _I, _I, _I, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_ffn_workspace_bytes": (_SZ, [_I, _I, _I, _I, ctypes.POINTER(Recipe)]),
    "moe_workspace_init": (_I, [_P, _SZ, _P]),
    "moe_ffn_forward": (_I, [_P, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _I, _P, ctypes.POINTER(Recipe),
                             _P, _SZ, _P, _P, _P, _P, _P]),
    "moe_get_device_status": (_I, [_P, _P, ctypes.POINTER(ctypes.c_int32)]),
    "moe_set_profile_events": (None, [_P, _I]),
    "moe_set_l2_prefetch": (_I, [_P, _P, _I]),
    "moe_set_schedule": (_I, [_I]),
    "moe_set_launch_overlap": (_I, [_I]),
    "moe_ffn_schedule": (_I, [_I, _I, _I, _I, ctypes.POINTER(Recipe), _I]),
    "moe_fp4_scales_bytes": (_SZ, [_I, _I, _I]),
    "moe_fp4_prepare_scales": (_I, [_P, _P, _I, _I, _I, _P, _SZ, _P]),
    "moe_ffn_forward_fp4": (_I, [_P, _I, _I, _I, _P, _P, _P, _P, _P, _P, _SZ, _P, _P, _I, _P,
                                 ctypes.POINTER(Recipe), _P, _SZ, _P, _P, _P, _P, _P]),
    "moe_mx_scales_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "moe_mx_prepare_scales": (_I, [_I, _P, _P, _I, _I, _I, _P, _P, _I, _P, _SZ, _P]),
    "moe_ffn_forward_mx": (_I, [_P, _I, _I, _I, _P, _P, _P, _I, _P, _P, _P, _P, _I, _P, _P, _SZ,
                                ctypes.POINTER(Recipe), _P, _SZ, _P, _P, _P, _P, _P]),
    "moe_qk_norm_rope": (_I, [_P, _L, _P, _L, _P, _L, _I, _I, _I, _I, _I, _P, _P, _F, _P, _I, _I, _I, _P, _P, _L,
                              _P, _P, _P, _L, _P, _SZ, _P]),
    "moe_prefix_attention_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "moe_prefix_attention": (_I, [_P, _L, _I, _I, _P, _I, _I, _I, _I, _P, _P, _I, _I, _P, _I, _P, _P, _I, _P, _I, _F,
                                  _P, _P, _P, _SZ, _P]),
    "moe_linear_workspace_bytes": (_SZ, [_I, _I, _I]),
    "moe_linear": (_I, [_P, _L, _I, _I, _P, _I, _I, _P, _I, _P, _L, _P, _L, _P, _SZ, _P]),
    "moe_q4_weight_bytes": (_SZ, [_I, _I, _I, _I]),
    "moe_q4_prepare": (_I, [_P, _P, _P, _I, _I, _I, _P, _SZ, _P]),
    "moe_linear_q4_workspace_bytes": (_SZ, [_I, _I, _I]),
    "moe_linear_q4": (_I, [_P, _L, _I, _I, _P, _SZ, _I, _I, _I, _I, _P, _I, _P, _L, _P, _L, _P, _SZ, _P]),
    "moe_kv4_write": (_I, [_P, _L, _P, _L, _I, _I, _I, _I, _P, _P, _I, _I, _P, _SZ, _P]),
    "moe_kv4_read": (_I, [_P, _I, _I, _I, _I, _P, _I, _P, _P, _I, _P, _SZ, _P]),
    "moe_prefix_attention_kv4_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "moe_prefix_attention_kv4": (_I, [_P, _L, _I, _I, _P, _I, _I, _I, _I, _P, _I, _I, _P, _I, _P, _P, _I, _P, _I, _F, _P,
                                      _P, _P, _SZ, _P]),
    "moe_pages_workspace_bytes": (_SZ, [_I, _I]),
    "moe_pages_resize": (_I, [_P, _I, _P, _I, _I, _I, _P, _P, _P, _I, _P, _SZ, _P]),
    "moe_pages_fork": (_I, [_P, _I, _P, _I, _I, _I, _P, _P, _P, _I, _P, _I, _P, _SZ, _P]),
    "moe_pages_compact": (_I, [_P, _I, _I, _I, _I, _P, _P, _I, _P, _I, _P, _P, _SZ, _P]),
}

SCHEDULE_AUTO, SCHEDULE_STREAM_K, SCHEDULE_SLICE = 0, 1, 2
SCHEDULE_NAMES = {SCHEDULE_STREAM_K: "stream_k", SCHEDULE_SLICE: "slice"}


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib_handle
    if _lib_handle is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with moe_ffn_speculative_gb300.build.build()")
        h = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(h, name)
            fn.restype = res
            fn.argtypes = args
        _lib_handle = h
    return _lib_handle


def header_functions():
    """Names of the functions include/moe.h declares."""
    with open(HEADER_PATH) as f:
        text = f.read()
    return re.findall(r"MOE_API\s+[\w\s\*]+?\b(moe_\w+)\s*\(", text)


def status_string(status: int) -> str:
    return lib().moe_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != MOE_OK:
        raise MoeError(status, where)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        # the current stream's handle, without the Stream object around it
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream


def _need_cuda(*ts):
    for t in ts:
        if t is not None:
            if not t.is_cuda:
                raise ValueError("tensor is not on a CUDA device")
            if not t.is_contiguous():
                raise ValueError("tensor is not contiguous")


def _u16(t: torch.Tensor) -> torch.Tensor:
    if t.dtype != torch.bfloat16:
        raise TypeError("expected a bfloat16 tensor")
    return t


# --------------------------------------------------------------------------- workspaces

class Workspace:
    """A zero-filled device workspace owned by torch's allocator."""

    def __init__(self, nbytes: int, device=None):
        self.nbytes = int(nbytes)
        self.buf = torch.zeros(max(self.nbytes, 256), dtype=torch.uint8,
                               device=device or torch.device("cuda", torch.cuda.current_device()))

    def ptr(self) -> int:
        return self.buf.data_ptr()

    def reset(self, stream=None) -> None:
        """Zero-fill again (moe_workspace_init), as after a device-side error."""
        _check(lib().moe_workspace_init(self.ptr(), self.nbytes, _stream(stream)), "moe_workspace_init")

    def set_start_gate(self, closed: bool, stream=None) -> None:
        """Close (non-zero) or open (zero) the workspace's start gate."""
        v = torch.tensor([1 if closed else 0], dtype=torch.int32, device=self.buf.device)
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            self.buf[WS_HOLD_OFFSET:WS_HOLD_OFFSET + 4].copy_(v.view(torch.uint8))

    def device_status(self, stream=None) -> Tuple[int, int]:
        info = ctypes.c_int32(0)
        st = lib().moe_get_device_status(self.ptr(), _stream(stream), ctypes.byref(info))
        return st, info.value


def ffn_workspace_bytes(T: int, H: int, I: int, Is: int, recipe: Recipe) -> int:
    n = lib().moe_ffn_workspace_bytes(T, H, I, Is, ctypes.byref(recipe))
    if n == 0:
        raise MoeError(MOE_ERR_INVALID_ARG, "moe_ffn_workspace_bytes")
    return n


def ffn_workspace_bytes_upto(max_tokens: int, H: int, I: int, Is: int, recipe: Recipe) -> int:
    """Bytes of a workspace that serves every token count 1..max_tokens: the
    size for exactly T is not monotone in T (above 128 tokens the token tile
    narrows to about four times an expert's mean load, shrinking its
    partial-accumulator region)."""
    n = 0
    for T in range(1, max_tokens + 1):
        n = max(n, ffn_workspace_bytes(T, H, I, Is, recipe))
    return n


# --------------------------------------------------------------------------- entry points

def moe_route(x, gate, recipe: Recipe, router_bias=None, expert_bias=None, ws: Workspace = None,
              want_logits=True, stream=None):
    """-> (topk_idx int32 [T,K], topk_w fp32 [T,K], logits fp32 [T,E] or None)."""
    _need_cuda(x, gate, router_bias, expert_bias)
    T, H = x.shape
    E, K = recipe.num_experts, recipe.top_k
    dev = x.device
    idx = torch.empty((T, K), dtype=torch.int32, device=dev)
    w = torch.empty((T, K), dtype=torch.float32, device=dev)
    logits = torch.empty((T, E), dtype=torch.float32, device=dev) if want_logits else None
    if ws is None:
        ws = Workspace(lib().moe_route_workspace_bytes(T, E), dev)
    _check(lib().moe_route(_ptr(_u16(x)), T, H, _ptr(_u16(gate)), _ptr(router_bias), _ptr(expert_bias),
                           ctypes.byref(recipe), _ptr(logits), _ptr(idx), _ptr(w), ws.ptr(), ws.nbytes,
                           _stream(stream)), "moe_route")
    return idx, w, logits


def moe_route_noalloc(x, gate, recipe: Recipe, router_bias=None, expert_bias=None, want_logits=True,
                      stream=None):
    """moe_route with the library's fixed scratch array instead of a workspace.
    -> (topk_idx int32 [T,K], topk_w fp32 [T,K], logits fp32 [T,E] or None)."""
    _need_cuda(x, gate, router_bias, expert_bias)
    T, H = x.shape
    E, K = recipe.num_experts, recipe.top_k
    dev = x.device
    idx = torch.empty((T, K), dtype=torch.int32, device=dev)
    w = torch.empty((T, K), dtype=torch.float32, device=dev)
    logits = torch.empty((T, E), dtype=torch.float32, device=dev) if want_logits else None
    _check(lib().moe_route_noalloc(_ptr(_u16(x)), T, H, _ptr(_u16(gate)), _ptr(router_bias), _ptr(expert_bias),
                                   ctypes.byref(recipe), _ptr(logits), _ptr(idx), _ptr(w), _stream(stream)),
           "moe_route_noalloc")
    return idx, w, logits


def moe_route_from_logits(logits, recipe: Recipe, expert_bias=None, stream=None):
    """-> (topk_idx int32 [T,K], topk_w fp32 [T,K])."""
    _need_cuda(logits, expert_bias)
    T = logits.shape[0]
    K = recipe.top_k
    idx = torch.empty((T, K), dtype=torch.int32, device=logits.device)
    w = torch.empty((T, K), dtype=torch.float32, device=logits.device)
    _check(lib().moe_route_from_logits(_ptr(logits), T, _ptr(expert_bias), ctypes.byref(recipe), _ptr(idx),
                                       _ptr(w), _stream(stream)), "moe_route_from_logits")
    return idx, w


def moe_permute(topk_idx, num_experts: int, stream=None):
    """-> (counts [E], offsets [E+1], sorted_pair [T*K], pair_pos [T*K]), int32."""
    _need_cuda(topk_idx)
    T, K = topk_idx.shape
    dev = topk_idx.device
    counts = torch.empty(num_experts, dtype=torch.int32, device=dev)
    offsets = torch.empty(num_experts + 1, dtype=torch.int32, device=dev)
    sp = torch.empty(T * K, dtype=torch.int32, device=dev)
    pp = torch.empty(T * K, dtype=torch.int32, device=dev)
    _check(lib().moe_permute(_ptr(topk_idx), T, K, num_experts, _ptr(counts), _ptr(offsets), _ptr(sp), _ptr(pp),
                             None, 0, _stream(stream)), "moe_permute")
    return counts, offsets, sp, pp


def moe_ffn_forward(x, gate, w_gate_up, w_down, recipe: Recipe, ws: Workspace, router_bias=None,
                    expert_bias=None, sh_gate_up=None, sh_down=None, sh_gate=None, y=None,
                    topk_idx_out=None, topk_w_out=None, counts_out=None, stream=None):
    """The whole layer; returns y [T,H] bf16."""
    _need_cuda(x, gate, w_gate_up, w_down, router_bias, expert_bias, sh_gate_up, sh_down, sh_gate, y,
               topk_idx_out, topk_w_out, counts_out)
    T, H = x.shape
    I = w_down.shape[2]
    Is = 0 if sh_gate_up is None else sh_down.shape[1]
    if y is None:
        y = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
    _check(lib().moe_ffn_forward(
        _ptr(_u16(x)), T, H, I, _ptr(_u16(gate)), _ptr(router_bias), _ptr(expert_bias), _ptr(_u16(w_gate_up)),
        _ptr(_u16(w_down)), _ptr(sh_gate_up), _ptr(sh_down), Is, _ptr(sh_gate), ctypes.byref(recipe), ws.ptr(),
        ws.nbytes, _ptr(y), _ptr(topk_idx_out), _ptr(topk_w_out), _ptr(counts_out), _stream(stream)),
        "moe_ffn_forward")
    return y


def _u8(t: torch.Tensor) -> torch.Tensor:
    if t.dtype != torch.uint8:
        raise TypeError("expected a uint8 tensor")
    return t


def fp4_prepare_scales(w_gate_up_s, w_down_s, stream=None) -> torch.Tensor:
    """The e8m0 scales [E,2I,H/32] and [E,H,I/32] re-laid for
    moe_ffn_forward_fp4 (once per set of weights); returns the uint8 buffer."""
    _need_cuda(w_gate_up_s, w_down_s)
    E, H = w_down_s.shape[0], w_down_s.shape[1]
    I = w_gate_up_s.shape[1] // 2
    n = lib().moe_fp4_scales_bytes(E, H, I)
    if n == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED, "moe_fp4_scales_bytes")
    out = torch.empty(n, dtype=torch.uint8, device=w_down_s.device)
    _check(lib().moe_fp4_prepare_scales(_ptr(_u8(w_gate_up_s)), _ptr(_u8(w_down_s)), E, H, I, _ptr(out), n,
                                        _stream(stream)), "moe_fp4_prepare_scales")
    return out


def moe_ffn_forward_fp4(x, gate, w_gate_up_q, w_down_q, scales, recipe: Recipe, ws: Workspace, router_bias=None,
                        expert_bias=None, sh_gate_up=None, sh_down=None, sh_gate=None, y=None,
                        topk_idx_out=None, topk_w_out=None, counts_out=None, stream=None):
    """The whole layer with FP4 routed experts (codes [E,2I,H/2], [E,H,I/2];
    ``scales`` from fp4_prepare_scales); returns y [T,H] bf16."""
    _need_cuda(x, gate, w_gate_up_q, w_down_q, scales, router_bias, expert_bias, sh_gate_up, sh_down, sh_gate, y,
               topk_idx_out, topk_w_out, counts_out)
    T, H = x.shape
    I = w_down_q.shape[2] * 2
    Is = 0 if sh_gate_up is None else sh_down.shape[1]
    if y is None:
        y = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
    _check(lib().moe_ffn_forward_fp4(
        _ptr(_u16(x)), T, H, I, _ptr(_u16(gate)), _ptr(router_bias), _ptr(expert_bias), _ptr(_u8(w_gate_up_q)),
        _ptr(_u8(w_down_q)), _ptr(_u8(scales)), scales.numel(), _ptr(sh_gate_up), _ptr(sh_down), Is, _ptr(sh_gate),
        ctypes.byref(recipe), ws.ptr(), ws.nbytes, _ptr(y), _ptr(topk_idx_out), _ptr(topk_w_out), _ptr(counts_out),
        _stream(stream)), "moe_ffn_forward_fp4")
    return y


def mx_format(t: dict) -> int:
    """Routed-expert format of a block-scaled layer's tensors: FP4 scales
    [E,2I,H/32] have a row per weight row, FP8 scales [E,2I/32,H/32] one per
    32 rows."""
    return FMT_FP4 if t["w_gate_up_s"].shape[1] == t["w_gate_up_q"].shape[1] else FMT_FP8


def mx_dims(t: dict):
    """(E, H, I, Is) of a block-scaled layer's tensors."""
    q = t["w_gate_up_q"]
    E, I = q.shape[0], q.shape[1] // 2
    H = q.shape[2] * (2 if mx_format(t) == FMT_FP4 else 1)
    Is = 0 if t.get("sh_gate_up_q") is None else t["sh_gate_up_q"].shape[0] // 2
    return E, H, I, Is


def mx_prepare_scales(t: dict, stream=None) -> torch.Tensor:
    """The weight scales of a block-scaled layer (routed w_gate_up_s, w_down_s,
    shared sh_gate_up_s, sh_down_s) re-laid for moe_ffn_forward_mx (once per
    set of weights); returns the uint8 buffer."""
    fmt = mx_format(t)
    E, H, I, Is = mx_dims(t)
    _need_cuda(t["w_gate_up_s"], t["w_down_s"], t.get("sh_gate_up_s"), t.get("sh_down_s"))
    n = lib().moe_mx_scales_bytes(fmt, E, H, I, Is)
    if n == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED, "moe_mx_scales_bytes")
    out = torch.empty(n, dtype=torch.uint8, device=t["w_down_s"].device)
    _check(lib().moe_mx_prepare_scales(fmt, _ptr(_u8(t["w_gate_up_s"])), _ptr(_u8(t["w_down_s"])), E, H, I,
                                       _ptr(t.get("sh_gate_up_s")), _ptr(t.get("sh_down_s")), Is, _ptr(out), n,
                                       _stream(stream)), "moe_mx_prepare_scales")
    return out


def moe_ffn_forward_mx(x, gate, routed_fmt: int, w_gate_up_q, w_down_q, scales, recipe: Recipe, ws: Workspace,
                       I: int, router_bias=None, expert_bias=None, sh_gate_up_q=None, sh_down_q=None, sh_gate=None,
                       y=None, topk_idx_out=None, topk_w_out=None, counts_out=None, stream=None):
    """The whole layer with block-scaled experts (FP4 or FP8 routed, FP8
    shared); returns y [T,H] bf16."""
    _need_cuda(x, gate, w_gate_up_q, w_down_q, scales, router_bias, expert_bias, sh_gate_up_q, sh_down_q, sh_gate, y,
               topk_idx_out, topk_w_out, counts_out)
    T, H = x.shape
    Is = 0 if sh_gate_up_q is None else sh_gate_up_q.shape[0] // 2
    if y is None:
        y = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
    _check(lib().moe_ffn_forward_mx(
        _ptr(_u16(x)), T, H, I, _ptr(_u16(gate)), _ptr(router_bias), _ptr(expert_bias), int(routed_fmt),
        _ptr(_u8(w_gate_up_q)), _ptr(_u8(w_down_q)), _ptr(sh_gate_up_q), _ptr(sh_down_q), Is, _ptr(sh_gate),
        _ptr(_u8(scales)), scales.numel(), ctypes.byref(recipe), ws.ptr(), ws.nbytes, _ptr(y), _ptr(topk_idx_out),
        _ptr(topk_w_out), _ptr(counts_out), _stream(stream)), "moe_ffn_forward_mx")
    return y


# --------------------------------------------------------------------------- the attention side of the layer
#
# A small call's time is the binding's.  These calls go through _binding.so
# (csrc/binding.cpp), which checks every argument and calls the library; it
# answers None where one of them is not as it has to be, and the checks below,
# which then run, say which and why.

_binding_module = None


def _binding():
    """The extension module; raises if it has not been built."""
    global _binding_module
    if _binding_module is None:
        path = os.path.join(_PKG, "_binding.so")
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with moe_ffn_speculative_gb300.build.build()")
        spec = importlib.util.spec_from_file_location("_binding", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _same_versions(module)
        _binding_module = module
    return _binding_module


def _same_versions(module) -> None:
    """Raises unless the extension was compiled for this torch and this Python: it
    reads their objects by their headers' layout."""
    version = re.match(r"\d+\.\d+\.\d+", torch.__version__).group()
    python = sys.hexversion >> 16
    if module.torch_version != version or module.python_version != python:
        raise RuntimeError(f"_binding.so was built for torch {module.torch_version}, Python {module.python_version:#x}; "
                           f"this is torch {version}, Python {python:#x}: build it again with "
                           "moe_ffn_speculative_gb300.build.build()")


_DTYPES = {torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16}


def _dtype16(t: torch.Tensor) -> int:
    """The library's code of a call's one 16-bit type."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a tensor")
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError("expected a bfloat16 or float16 tensor")
    return code


def _refuse(t, dtype, name: str) -> None:
    """Says what keeps `t` from being a contiguous GPU tensor of `dtype`."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected a {dtype} tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: tensor is not on a CUDA device")
    if t.get_device() != torch.cuda.current_device():
        raise ValueError(f"{name}: tensor is not on the current CUDA device")
    raise ValueError(f"{name}: tensor is not contiguous")


def _elsewhere(t: torch.Tensor) -> bool:
    return not t.is_cuda or t.get_device() != torch.cuda.current_device()


def _flat(t: Optional[torch.Tensor], dtype, n: int, name: str) -> Optional[int]:
    """Address of a contiguous tensor of n elements, or None."""
    if t is None:
        return None
    if t.dtype is not dtype or _elsewhere(t) or not t.is_contiguous():
        _refuse(t, dtype, name)
    if t.numel() != n:
        raise ValueError(f"{name}: expected {n} elements")
    return t.data_ptr()


def _heads(t: torch.Tensor, dtype, T: int, h: int, D: int, name: str) -> int:
    """Row stride of a [T, h, D] tensor on the GPU whose rows may lie apart (a
    slice of a fused projection)."""
    if t.dtype is not dtype or _elsewhere(t):
        _refuse(t, dtype, name)
    if t.shape != (T, h, D):
        raise ValueError(f"{name}: expected [{T}, {h}, {D}]")
    s0, s1, s2 = t.stride()
    if (s2 != 1 and D > 1) or (s1 != D and h > 1):
        if t.numel():
            raise ValueError(f"{name}: the heads of a row are not contiguous")
    return s0 if T > 1 else h * D


def _made(shape, like: torch.Tensor, stream) -> torch.Tensor:
    """A buffer of `like`'s type for a call on `stream`: from that stream's memory,
    since a block that the current stream's work still reads is free for the
    current stream only; and kept, once dropped, until the current stream's work
    of then has ended, as the caller reads it there."""
    if stream is None:
        return torch.empty(shape, dtype=like.dtype, device=like.device)
    current = torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=like.dtype, device=like.device)
    t.record_stream(current)
    return t


def rope_table(max_positions: int, rot_dim: int, base: float = 10000.0, scale: float = 1.0,
               device=None) -> torch.Tensor:
    """Cosines and sines of every position for ``qk_norm_rope``: fp32
    [max_positions, rot_dim], the angles position * scale * base^(-2i/rot_dim)
    taken in 64 bits.  Any other table of that layout serves as well."""
    device = device or torch.device("cuda", torch.cuda.current_device())
    inv = float(base) ** (-torch.arange(0, rot_dim, 2, device=device, dtype=torch.float64) / rot_dim)
    angle = torch.arange(max_positions, device=device, dtype=torch.float64)[:, None] * (scale * inv)
    return torch.cat([angle.cos(), angle.sin()], dim=1).float()


def qk_norm_rope(q, k, v, positions, rope, ws: Workspace, q_weight=None, k_weight=None, eps: float = 1e-6,
                 interleaved: bool = False, q_out=None, k_cache=None, v_cache=None, slots=None, stream=None):
    """RMS norms of the query and key heads, the position rotation and the
    cache write in one launch (moe_qk_norm_rope).

    q [T,Hq,D], k, v [T,Hkv,D] (rows may lie apart, e.g. slices of a fused
    projection); positions int32 [T], rope fp32 [max_pos, rot_dim]
    (``rope_table``), both None for no rotation; q_weight, k_weight [D] or None
    for no norm; k_cache, v_cache contiguous [..., Hkv, D]
    ([pages, page_size, Hkv, D] for a cache of pages), slots int32 [T] their
    rows (negative: not cached; None: row t).  q, k and v may be None.
    -> (q_out, k_cache, v_cache); buffers that are not given are made."""
    lead = q if q is not None else k
    if lead.is_cuda and (k is None) == (k_cache is None) and (v is None) == (v_cache is None):
        if q is not None and q_out is None:
            q_out = _made(q.shape, q, stream)
        status = _binding().qk_norm_rope(q, k, v, positions, rope, q_weight, k_weight, eps, interleaved, q_out, k_cache,
                                         v_cache, slots, ws.ptr(), ws.nbytes, _stream(stream))
        if status == 0:
            return q_out, k_cache, v_cache
        if status is not None:
            raise MoeError(status, "moe_qk_norm_rope")
    dt, dtype = _dtype16(lead), lead.dtype
    if lead.dim() != 3:
        raise ValueError("expected [T, heads, D]")
    if k is not None and k.dtype is not dtype:
        _refuse(k, dtype, "k")
    T, h, D = lead.shape
    Hq = Hkv = qs = ks = vs = qos = n_slots = rot = max_pos = 0
    pk = pv = pkc = pvc = None
    if q is not None:
        Hq = h
        qs = _heads(q, dtype, T, h, D, "q")
        if q_out is None:
            q_out = _made((T, h, D), q, stream)
            qos = h * D
        else:
            qos = _heads(q_out, dtype, T, h, D, "q_out")
    if k is not None:
        if k.dim() != 3:
            raise ValueError("k: expected [T, heads, D]")
        Hkv = k.shape[1]
        ks = _heads(k, dtype, T, Hkv, D, "k")
        pk = k.data_ptr()
        if k_cache is None or (v is not None and v_cache is None):
            if slots is not None:
                raise ValueError("slots name rows of a cache: pass k_cache and v_cache")
            if k_cache is None:
                k_cache = _made((T, Hkv, D), k, stream)
            if v is not None and v_cache is None:
                v_cache = _made((T, Hkv, D), k, stream)
        size = k_cache.numel()
        if k_cache.shape[-2:] != (Hkv, D):
            raise ValueError("k_cache: expected [..., Hkv, D]")
        n_slots = size // (Hkv * D)
        pkc = _flat(k_cache, dtype, size, "k_cache")
        if v is not None:
            vs = _heads(v, dtype, T, Hkv, D, "v")
            pv = v.data_ptr()
            if v_cache.shape[-2:] != (Hkv, D):
                raise ValueError("v_cache: expected [..., Hkv, D]")
            pvc = _flat(v_cache, dtype, size, "v_cache")
    if (v is not None and k is None) or (v_cache is not None and v is None):
        raise ValueError("v needs k, v_cache needs v")
    if rope is not None:
        max_pos, rot = rope.shape
        rope = _flat(rope, torch.float32, max_pos * rot, "rope")
    status = lib().moe_qk_norm_rope(
        None if q is None else q.data_ptr(), qs, pk, ks, pv, vs, T, Hq, Hkv, D, dt,
        _flat(q_weight, dtype, D, "q_weight"), _flat(k_weight, dtype, D, "k_weight"), eps, rope, rot, max_pos,
        1 if interleaved else 0, _flat(positions, torch.int32, T, "positions"),
        None if q_out is None else q_out.data_ptr(), qos, pkc, pvc, _flat(slots, torch.int32, T, "slots"), n_slots,
        ws.ptr(), ws.nbytes, _stream(stream))
    if status:
        raise MoeError(status, "moe_qk_norm_rope")
    return q_out, k_cache, v_cache


def prefix_attention_workspace_bytes(T: int, B: int, Hq: int, Hkv: int, D: int) -> int:
    n = lib().moe_prefix_attention_workspace_bytes(T, B, Hq, Hkv, D)
    if n == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED, "moe_prefix_attention_workspace_bytes")
    return n


def prefix_attention(q, k_cache, v_cache, q_start, prefix_pages, prefix_len, page_table, own_len, ws: Workspace,
                     causal: bool = True, scale: Optional[float] = None, out=None, lse=None, stream=None):
    """Attention of a batch of requests over a prefix that all of them share
    and pages of their own (moe_prefix_attention).

    q [T,Hq,D] (rows may lie apart); k_cache, v_cache [pages, page_size, Hkv, D];
    q_start int32 [B+1]; prefix_pages int32 [n] with prefix_len int32 [1], or
    both None; page_table int32 [B, width] with own_len int32 [B], or both
    None; scale 1/sqrt(D) unless given; lse fp32 [T,Hq] is written when given.
    -> out [T,Hq,D]."""
    if not q.is_cuda:
        _refuse(q, q.dtype, "q")
    if out is None:
        out = _made(q.shape, q, stream)
    if scale is None:
        scale = q.shape[-1] ** -0.5
    status = _binding().prefix_attention(q, k_cache, v_cache, q_start, prefix_pages, prefix_len, page_table, own_len,
                                         causal, scale, out, lse, ws.ptr(), ws.nbytes, _stream(stream))
    if status == 0:
        return out
    if status is not None:
        raise MoeError(status, "moe_prefix_attention")
    dt, dtype = _dtype16(q), q.dtype
    if q.dim() != 3 or k_cache.dim() != 4:
        raise ValueError("expected q [T, Hq, D], caches [pages, page_size, Hkv, D]")
    T, Hq, D = q.shape
    qs = _heads(q, dtype, T, Hq, D, "q")
    pages, page, Hkv, dk = k_cache.shape
    size = pages * page * Hkv * dk
    if dk != D:
        raise ValueError("caches: expected heads of q's size")
    if v_cache.shape != k_cache.shape:
        raise ValueError("v_cache: expected the shape of k_cache")
    B = q_start.numel() - 1
    if B < 0 or (prefix_pages is None) != (prefix_len is None) or (page_table is None) != (own_len is None):
        raise ValueError("q_start has B+1 elements; page lists come with their lengths")
    cap = 0 if prefix_pages is None else prefix_pages.numel()
    width = 0
    if page_table is not None:
        rows, width = page_table.shape
        if rows != B:
            raise ValueError("page_table: expected [B, width]")
    if out.shape != q.shape:
        raise ValueError("out: expected the shape of q")
    i32 = torch.int32
    status = lib().moe_prefix_attention(
        q.data_ptr(), qs, T, B, _flat(q_start, i32, B + 1, "q_start"), Hq, Hkv, D, dt,
        _flat(k_cache, dtype, size, "k_cache"), _flat(v_cache, dtype, size, "v_cache"), pages, page,
        _flat(prefix_pages, i32, cap, "prefix_pages"), cap, _flat(prefix_len, i32, 1, "prefix_len"),
        _flat(page_table, i32, B * width, "page_table"), width, _flat(own_len, i32, B, "own_len"), 1 if causal else 0,
        scale, _flat(out, dtype, T * Hq * D, "out"),
        _flat(lse, torch.float32, T * Hq, "lse"), ws.ptr(), ws.nbytes, _stream(stream))
    if status:
        raise MoeError(status, "moe_prefix_attention")
    return out


ACTIVATIONS = {"none": 0, "silu": 1, "gelu": 2, "gelu_tanh": 3, "relu": 4}


def linear_workspace_bytes(M: int, N: int, K: int) -> int:
    n = lib().moe_linear_workspace_bytes(M, N, K)
    if n == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED, "moe_linear_workspace_bytes")
    return n


def _rows(t: torch.Tensor, dtype, m: int, n: int, name: str) -> int:
    """Row stride of an [m, n] matrix on the GPU whose rows may lie apart."""
    if t.dtype is not dtype or _elsewhere(t):
        _refuse(t, dtype, name)
    if t.shape != (m, n):
        raise ValueError(f"{name}: expected [{m}, {n}]")
    s0, s1 = t.stride()
    if s1 != 1 and n > 1:
        raise ValueError(f"{name}: the elements of a row are not contiguous")
    return s0 if m > 1 else n


def linear(x, w, ws: Workspace, bias=None, activation: str = "none", residual=None, y=None, stream=None):
    """act(x w^T + bias) + residual (moe_linear): x [M,K], w [N,K], bias [N],
    residual [M,N]; activation one of ACTIVATIONS; rows of x, residual and y
    may lie apart; residual may be y.  -> y [M,N]."""
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"unknown activation {activation!r}")
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError("expected x [M, K], w [N, K]")
    if not x.is_cuda:
        _refuse(x, x.dtype, "x")
    if y is None:
        y = _made((x.shape[0], w.shape[0]), x, stream)
    status = _binding().linear(x, w, bias, act, residual, y, ws.ptr(), ws.nbytes, _stream(stream))
    if status == 0:
        return y
    if status is not None:
        raise MoeError(status, "moe_linear")
    dt, dtype = _dtype16(x), x.dtype
    M, K = x.shape
    N = w.shape[0]
    xs = _rows(x, dtype, M, K, "x")
    ys = _rows(y, dtype, M, N, "y")
    rs, pr = 0, None
    if residual is not None:
        rs, pr = _rows(residual, dtype, M, N, "residual"), residual.data_ptr()
    status = lib().moe_linear(x.data_ptr(), xs, M, K, _flat(w, dtype, N * K, "w"), N, dt, _flat(bias, dtype, N, "bias"),
                              act, pr, rs, y.data_ptr(), ys, ws.ptr(), ws.nbytes, _stream(stream))
    if status:
        raise MoeError(status, "moe_linear")
    return y


# --------------------------------------------------------------------------- the attention side in 4 bits, pages
#
# As above: the extension module answers None where something is wrong with the
# arguments, and the checks below say what.

def _wrong(where: str) -> ValueError:
    return ValueError(f"{where}: the arguments do not fit together")


def _contiguous(t, dtype, name: str) -> None:
    """Raises unless `t` is a contiguous tensor of `dtype` on the current GPU."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or _elsewhere(t) or not t.is_contiguous():
        _refuse(t, dtype, name)


class Q4Weight:
    """Weights of 4 bits as ``q4_prepare`` lays them out: N outputs, K inputs, groups
    of `group` inputs with scales of `dtype` and zero points or none."""

    def __init__(self, data, N: int, K: int, group: int, dtype, zeros: bool):
        self.data, self.N, self.K, self.group, self.dtype, self.zeros = data, N, K, group, dtype, zeros


def q4_prepare(codes, scales, zeros=None, stream=None) -> Q4Weight:
    """Lays out weights of 4 bits for ``linear_q4`` (moe_q4_prepare), once a set:
    codes uint8 [N, K/2] (the even input in the low nibble), scales [N, K/group] of the
    activations' type, zeros uint8 [N, K/group] or None (8 everywhere); the weight is
    scale * (code - zero)."""
    _contiguous(codes, torch.uint8, "codes")
    _dtype16(scales)
    _contiguous(scales, scales.dtype, "scales")
    if codes.dim() != 2 or scales.dim() != 2 or scales.shape[0] != codes.shape[0] or scales.shape[1] < 1:
        raise ValueError("expected codes [N, K/2], scales [N, K/group]")
    N, K = codes.shape[0], 2 * codes.shape[1]
    if K % scales.shape[1]:
        raise ValueError("scales: expected [N, K/group]")
    group = K // scales.shape[1]
    _flat(zeros, torch.uint8, scales.numel(), "zeros")
    n = lib().moe_q4_weight_bytes(N, K, group, 0 if zeros is None else 1)
    if n == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED, "moe_q4_weight_bytes")
    data = _made(n, codes, stream)
    _check(lib().moe_q4_prepare(_ptr(codes), _ptr(scales), _ptr(zeros), N, K, group, _ptr(data), n, _stream(stream)),
           "moe_q4_prepare")
    return Q4Weight(data, N, K, group, scales.dtype, zeros is not None)


def linear_q4_workspace_bytes(M: int, N: int, K: int) -> int:
    n = lib().moe_linear_q4_workspace_bytes(M, N, K)
    if n == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED, "moe_linear_q4_workspace_bytes")
    return n


def linear_q4(x, w: Q4Weight, ws: Workspace, bias=None, activation: str = "none", residual=None, y=None, stream=None):
    """act(x w^T + bias) + residual with weights of 4 bits (moe_linear_q4): x [M,K], w
    from ``q4_prepare``, the others as in ``linear``.  -> y [M,N]."""
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"unknown activation {activation!r}")
    if not isinstance(w, Q4Weight):
        raise TypeError("w: expected the weights that q4_prepare gives")
    if x.dtype is not w.dtype:
        raise TypeError(f"x: expected the scales' type, {w.dtype}")
    if x.dim() != 2:
        raise ValueError("expected x [M, K]")
    if not x.is_cuda:
        _refuse(x, x.dtype, "x")
    if y is None:
        y = _made((x.shape[0], w.N), x, stream)
    status = _binding().linear_q4(x, w.data, w.N, w.K, w.group, w.zeros, bias, act, residual, y, ws.ptr(), ws.nbytes,
                                  _stream(stream))
    if status == 0:
        return y
    if status is not None:
        raise MoeError(status, "moe_linear_q4")
    M = x.shape[0]
    _rows(x, x.dtype, M, w.K, "x")
    _rows(y, x.dtype, M, w.N, "y")
    if residual is not None:
        _rows(residual, x.dtype, M, w.N, "residual")
    _flat(bias, x.dtype, w.N, "bias")
    _contiguous(w.data, torch.uint8, "w")
    raise _wrong("linear_q4")


def kv4_shape(pages: int, page_size: int, Hkv: int, D: int) -> Tuple[int, int, int]:
    """Shape of a cache in 4 bits (uint8): e2m1 codes of keys and values with an
    e8m0 scale per 32 channels (moe_kv4_write has the layout of a block)."""
    return pages, Hkv, page_size * (D + D // 16)


def _kv4_page(cache, D: int) -> int:
    """Page size of a kv4 cache of heads of D channels."""
    _contiguous(cache, torch.uint8, "cache")
    slot = D + D // 16
    if cache.dim() != 3 or slot == 0 or cache.shape[2] % slot:
        raise ValueError(f"cache: expected [pages, Hkv, page_size * {slot}] (kv4_shape)")
    return cache.shape[2] // slot


def kv4_write(k, v, slots, cache, ws: Workspace, stream=None):
    """Keys and values rounded to 4 bits into their slots of a cache
    (moe_kv4_write).

    k, v [T,Hkv,D] (rows may lie apart); slots int32 [T] (page * page_size +
    offset; negative: padding; None: token t goes to slot t); cache uint8 of
    ``kv4_shape``.  -> cache."""
    status = _binding().kv4_write(k, v, slots, cache, ws.ptr(), ws.nbytes, _stream(stream))
    if status == 0:
        return cache
    if status is not None:
        raise MoeError(status, "moe_kv4_write")
    _dtype16(k)
    if k.dim() != 3:
        raise ValueError("k: expected [T, heads, D]")
    T, Hkv, D = k.shape
    _heads(k, k.dtype, T, Hkv, D, "k")
    _heads(v, k.dtype, T, Hkv, D, "v")
    _kv4_page(cache, D)
    if cache.shape[1] != Hkv:
        raise ValueError("cache: expected the heads of k")
    _flat(slots, torch.int32, T, "slots")
    raise _wrong("kv4_write")


def kv4_read(cache, D: int, ws: Workspace, pages=None, k=None, v=None, dtype=torch.bfloat16, stream=None):
    """Pages of a 4-bit cache expanded to 16 bits (moe_kv4_read): pages int32 [n]
    (None: all).  -> k, v [n, page_size, Hkv, D], of `dtype` where they are not
    given."""
    page = _kv4_page(cache, D)
    n = cache.shape[0] if pages is None else pages.numel()
    like = cache.new_empty(0, dtype=dtype) if k is None or v is None else None
    k = _made((n, page, cache.shape[1], D), like, stream) if k is None else k
    v = _made((n, page, cache.shape[1], D), like, stream) if v is None else v
    status = _binding().kv4_read(cache, D, pages, k, v, ws.ptr(), ws.nbytes, _stream(stream))
    if status == 0:
        return k, v
    if status is not None:
        raise MoeError(status, "moe_kv4_read")
    _dtype16(k)
    for t, name in ((k, "k"), (v, "v")):
        if t.shape != (n, page, cache.shape[1], D):
            raise ValueError(f"{name}: expected [n, page_size, Hkv, D]")
        _contiguous(t, k.dtype, name)
    _flat(pages, torch.int32, n, "pages")
    raise _wrong("kv4_read")


def prefix_attention_kv4_workspace_bytes(T: int, B: int, Hq: int, Hkv: int, D: int) -> int:
    n = lib().moe_prefix_attention_kv4_workspace_bytes(T, B, Hq, Hkv, D)
    if n == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED, "moe_prefix_attention_kv4_workspace_bytes")
    return n


def prefix_attention_kv4(q, cache, q_start, prefix_pages, prefix_len, page_table, own_len, ws: Workspace,
                         causal: bool = True, scale: Optional[float] = None, out=None, lse=None, stream=None):
    """``prefix_attention`` over a cache in 4 bits (moe_prefix_attention_kv4): cache
    uint8 of ``kv4_shape``, the other arguments as there.  -> out [T,Hq,D]."""
    if not q.is_cuda:
        _refuse(q, q.dtype, "q")
    if out is None:
        out = _made(q.shape, q, stream)
    if scale is None:
        scale = q.shape[-1] ** -0.5
    status = _binding().prefix_attention_kv4(q, cache, q_start, prefix_pages, prefix_len, page_table, own_len, causal,
                                             scale, out, lse, ws.ptr(), ws.nbytes, _stream(stream))
    if status == 0:
        return out
    if status is not None:
        raise MoeError(status, "moe_prefix_attention_kv4")
    _dtype16(q)
    if q.dim() != 3:
        raise ValueError("expected q [T, Hq, D]")
    T, Hq, D = q.shape
    _heads(q, q.dtype, T, Hq, D, "q")
    _kv4_page(cache, D)
    B = q_start.numel() - 1
    if B < 0 or (prefix_pages is None) != (prefix_len is None) or (page_table is None) != (own_len is None):
        raise ValueError("q_start has B+1 elements; page lists come with their lengths")
    if page_table is not None and (page_table.dim() != 2 or page_table.shape[0] != B):
        raise ValueError("page_table: expected [B, width]")
    if out.shape != q.shape:
        raise ValueError("out: expected the shape of q")
    i32 = torch.int32
    for t, n, name in ((q_start, B + 1, "q_start"), (prefix_len, 1, "prefix_len"), (own_len, B, "own_len")):
        _flat(t, i32, n, name)
    for t, name in ((prefix_pages, "prefix_pages"), (page_table, "page_table")):
        if t is not None:
            _contiguous(t, i32, name)
    _contiguous(out, q.dtype, "out")
    _flat(lse, torch.float32, T * Hq, "lse")
    raise _wrong("prefix_attention_kv4")


def pages_workspace_bytes(B: int, n_pages: int) -> int:
    n = lib().moe_pages_workspace_bytes(B, n_pages)
    if n == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED, "moe_pages_workspace_bytes")
    return n


def _check_pools(caches, n_pages: int, page_size: int) -> None:
    """Says what keeps the caches from being pools of n_pages pages."""
    if len(caches) > 64:
        raise ValueError("caches: at most 64")
    for i, t in enumerate(caches):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"caches[{i}]: expected a tensor")
        _contiguous(t, t.dtype, f"caches[{i}]")
        if t.dim() < 3 or t.shape[0] != n_pages:
            raise ValueError(f"caches[{i}]: expected {n_pages} pages")
        kv4 = t.dtype is torch.uint8 and t.dim() == 3
        if kv4 and (t.shape[2] % page_size or t.shape[2] // page_size * 16 % 17):
            raise ValueError(f"caches[{i}]: expected [pages, Hkv, page_size * (D + D / 16)]")
        if not kv4 and t.shape[1] != page_size:
            raise ValueError(f"caches[{i}]: expected [pages, page_size, ...]")


def _check_page_state(refs, page_table, own_len, page_size: int, caches) -> None:
    _contiguous(refs, torch.int32, "refs")
    _contiguous(page_table, torch.int32, "page_table")
    if page_table.dim() != 2:
        raise ValueError("page_table: expected [B, width]")
    _flat(own_len, torch.int32, page_table.shape[0], "own_len")
    if page_size < 1:
        raise ValueError("page_size: expected a positive number")
    _check_pools(caches, refs.numel(), page_size)


def pages_resize(refs, page_table, own_len, new_len, page_size: int, ws: Workspace, caches=(), stream=None) -> None:
    """Gives every request the pages of its new length and takes back the others
    (moe_pages_resize); 0 frees a request.

    refs int32 [pages], page_table int32 [B, width] and own_len int32 [B] are the
    state, changed in place; new_len int32 [B]; caches: the tensors whose pages these
    are, [pages, page_size, ...] or of ``kv4_shape``, in which a page that is written
    on while another request shares it is copied."""
    caches = tuple(caches)
    status = _binding().pages_resize(refs, page_table, own_len, new_len, page_size, caches, ws.ptr(), ws.nbytes,
                                     _stream(stream))
    if status == 0:
        return
    if status is not None:
        raise MoeError(status, "moe_pages_resize")
    _check_page_state(refs, page_table, own_len, page_size, caches)
    _contiguous(new_len, torch.int32, "new_len")
    _flat(new_len, torch.int32, page_table.shape[0], "new_len")
    raise _wrong("pages_resize")


def pages_fork(refs, page_table, own_len, src, dst, page_size: int, ws: Workspace, caches=(), stream=None) -> None:
    """Makes request dst[i] a copy of request src[i] (moe_pages_fork): full pages are
    shared, the last one is copied in every cache.  src, dst int32 [n]; the rest as in
    ``pages_resize``."""
    caches = tuple(caches)
    status = _binding().pages_fork(refs, page_table, own_len, src, dst, page_size, caches, ws.ptr(), ws.nbytes,
                                   _stream(stream))
    if status == 0:
        return
    if status is not None:
        raise MoeError(status, "moe_pages_fork")
    _check_page_state(refs, page_table, own_len, page_size, caches)
    _contiguous(src, torch.int32, "src")
    _contiguous(dst, torch.int32, "dst")
    _flat(dst, torch.int32, src.numel(), "dst")
    raise _wrong("pages_fork")


def pages_compact(page_table, base, keep, page_size: int, ws: Workspace, caches=(), new_len=None, stream=None):
    """Moves the kept tokens of every request's block up in every cache
    (moe_pages_compact): token base[b] + keep[b, j] goes to base[b] + j.

    base int32 [B], keep int32 [B, n] (growing offsets, the first negative one ends a
    row); caches as in ``pages_resize``.  -> new_len int32 [B], the length after them."""
    caches = tuple(caches)
    if new_len is None:
        new_len = _made(base.shape, base, stream)
    n_pages = caches[0].shape[0] if caches else (2 ** 31 - 1) // max(1, page_size)
    status = _binding().pages_compact(page_table, base, keep, page_size, n_pages, caches, new_len, ws.ptr(), ws.nbytes,
                                      _stream(stream))
    if status == 0:
        return new_len
    if status is not None:
        raise MoeError(status, "moe_pages_compact")
    _contiguous(page_table, torch.int32, "page_table")
    if page_table.dim() != 2 or keep.dim() != 2 or keep.shape[0] != page_table.shape[0]:
        raise ValueError("expected page_table [B, width], keep [B, n]")
    _contiguous(keep, torch.int32, "keep")
    for t, name in ((base, "base"), (new_len, "new_len")):
        _flat(t, torch.int32, page_table.shape[0], name)
    if page_size < 1:
        raise ValueError("page_size: expected a positive number")
    _check_pools(caches, n_pages, page_size)
    raise _wrong("pages_compact")


def set_schedule(schedule: int) -> None:
    """Expert schedule of later moe_ffn_forward calls on this thread:
    SCHEDULE_AUTO, SCHEDULE_STREAM_K or SCHEDULE_SLICE."""
    _check(lib().moe_set_schedule(int(schedule)), "moe_set_schedule")


def set_launch_overlap(enable: bool) -> None:
    """Whether later fused-schedule launches on this thread overlap the
    previous kernel on their stream (True, the default) or are cooperative
    launches (False); both compute the same bits."""
    _check(lib().moe_set_launch_overlap(1 if enable else 0), "moe_set_launch_overlap")


def ffn_schedule(T: int, H: int, I: int, Is: int, recipe: Recipe, gated: bool = False) -> int:
    """The schedule moe_ffn_forward would run for this shape (SCHEDULE_STREAM_K
    or SCHEDULE_SLICE)."""
    s = lib().moe_ffn_schedule(T, H, I, Is, ctypes.byref(recipe), 1 if gated else 0)
    if s < 0:
        raise MoeError(1, "moe_ffn_schedule")
    return s


def set_l2_prefetch(tensors) -> None:
    """The next forward on this thread prefetches these tensors' bytes into
    L2 in its expert kernel's tail (moe_set_l2_prefetch); None or [] clears."""
    ts = [t for t in (tensors or []) if t is not None]
    _need_cuda(*ts)
    ptrs = (ctypes.c_void_p * max(1, len(ts)))(*[t.data_ptr() for t in ts])
    sizes = (ctypes.c_size_t * max(1, len(ts)))(*[t.numel() * t.element_size() for t in ts])
    _check(lib().moe_set_l2_prefetch(ctypes.cast(ptrs, ctypes.c_void_p), ctypes.cast(sizes, ctypes.c_void_p),
                                     len(ts)), "moe_set_l2_prefetch")


def set_profile_events(events) -> None:
    """events: a list of torch.cuda.Event (pairs around each launch) or None."""
    global _profile_keepalive
    if not events:
        lib().moe_set_profile_events(None, 0)
        _profile_keepalive = None
        return
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    _profile_keepalive = arr
    lib().moe_set_profile_events(ctypes.cast(arr, ctypes.c_void_p), len(events) // 2)


_profile_keepalive = None


def layer_path(tensors: dict, mx: Optional[bool] = None) -> str:
    """Which entry point runs a layer with these weights: "bf16"
    (moe_ffn_forward), "mx" (moe_ffn_forward_mx: FP4 or FP8 routed codes,
    no shared expert or an FP8 one) or "fp4" (moe_ffn_forward_fp4: FP4
    routed codes, no shared expert or a bf16 one).  mx=None picks the
    block-scaled path wherever it takes the layer (H, I and the shared
    expert's width multiples of 128, no bf16 shared expert); True / False
    ask for it or for the converter path.  Raises ValueError for weights
    that no path takes as asked."""
    if tensors.get("w_down_q") is None:
        if mx:
            raise ValueError("the block-scaled path takes coded routed experts (w_gate_up_q, w_down_q)")
        return "bf16"
    bf16_shared = tensors.get("sh_gate_up") is not None
    fp8_shared = tensors.get("sh_gate_up_q") is not None
    if bf16_shared and fp8_shared:
        raise ValueError("both a bf16 and an FP8 shared expert given")
    fmt = mx_format(tensors)
    if mx is None:
        _, H, I, Is = mx_dims(tensors)
        fits = H % 128 == 0 and I % 128 == 0 and Is % 128 == 0
        mx = fmt == FMT_FP8 or fp8_shared or (fits and not bf16_shared)
    if mx and bf16_shared:
        raise ValueError("the block-scaled path takes an FP8 shared expert (sh_gate_up_q), not a bf16 one")
    if not mx and (fmt == FMT_FP8 or fp8_shared):
        raise ValueError("FP8 weights run only on the block-scaled path")
    return "mx" if mx else "fp4"


class MoELayer:
    """Weights of one layer plus its workspace; ``forward(x)`` runs the layer."""

    def __init__(self, tensors: dict, recipe: Recipe, max_tokens: int, mx: Optional[bool] = None):
        """Routed experts as bf16 (w_gate_up, w_down), or as codes
        (w_gate_up_q, w_down_q with scales w_gate_up_s, w_down_s, re-laid once
        here).  The entry point is chosen by layer_path(tensors, mx): coded
        weights take the block-scaled path (moe_ffn_forward_mx) wherever it
        takes the layer, else FP4 codes take moe_ffn_forward_fp4."""
        self.t = tensors
        self.recipe = recipe
        path = layer_path(tensors, mx)
        self.mx = path == "mx"
        self.fp4 = path == "fp4"
        if self.mx:
            self.fmt = mx_format(tensors)
            _, self.H, self.I, self.Is = mx_dims(tensors)
            self.scales = mx_prepare_scales(tensors)
        elif self.fp4:
            self.H = tensors["w_down_q"].shape[1]
            self.I = tensors["w_down_q"].shape[2] * 2
            self.scales = fp4_prepare_scales(tensors["w_gate_up_s"], tensors["w_down_s"])
        else:
            self.H = tensors["w_down"].shape[1]
            self.I = tensors["w_down"].shape[2]
        if not self.mx:
            self.Is = 0 if tensors.get("sh_gate_up") is None else tensors["sh_down"].shape[1]
        self.max_tokens = max_tokens
        # one workspace for every token count up to max_tokens: its counters
        # sit in a fixed header and return to zero after every call
        self.ws = Workspace(ffn_workspace_bytes_upto(max_tokens, self.H, self.I, self.Is, recipe),
                            tensors["gate"].device)

    def routing_independent(self):
        """The tensors of this layer that do not depend on its routing: the
        router gate and biases, the shared expert and its gate."""
        t = self.t
        keys = ["gate", "router_bias", "expert_bias", "sh_gate", "sh_gate_up", "sh_down", "sh_gate_up_q", "sh_down_q"]
        return [t[k] for k in keys if t.get(k) is not None]

    def forward(self, x, y=None, topk_idx_out=None, topk_w_out=None, counts_out=None, stream=None, ahead=None):
        """ahead: the next MoELayer, whose routing-independent weights this
        forward prefetches into L2 in its expert kernel's tail."""
        T = x.shape[0]
        if ahead is not None:
            set_l2_prefetch(ahead.routing_independent())
        if T > self.max_tokens:
            raise ValueError("more tokens than the workspace was sized for")
        t = self.t
        if self.mx:
            return moe_ffn_forward_mx(x, t["gate"], self.fmt, t["w_gate_up_q"], t["w_down_q"], self.scales,
                                      self.recipe, self.ws, self.I, router_bias=t.get("router_bias"),
                                      expert_bias=t.get("expert_bias"), sh_gate_up_q=t.get("sh_gate_up_q"),
                                      sh_down_q=t.get("sh_down_q"), sh_gate=t.get("sh_gate"), y=y,
                                      topk_idx_out=topk_idx_out, topk_w_out=topk_w_out, counts_out=counts_out,
                                      stream=stream)
        if self.fp4:
            return moe_ffn_forward_fp4(x, t["gate"], t["w_gate_up_q"], t["w_down_q"], self.scales, self.recipe,
                                       self.ws, router_bias=t.get("router_bias"), expert_bias=t.get("expert_bias"),
                                       sh_gate_up=t.get("sh_gate_up"), sh_down=t.get("sh_down"),
                                       sh_gate=t.get("sh_gate"), y=y, topk_idx_out=topk_idx_out,
                                       topk_w_out=topk_w_out, counts_out=counts_out, stream=stream)
        return moe_ffn_forward(x, t["gate"], t["w_gate_up"], t["w_down"], self.recipe, self.ws,
                               router_bias=t.get("router_bias"), expert_bias=t.get("expert_bias"),
                               sh_gate_up=t.get("sh_gate_up"), sh_down=t.get("sh_down"), sh_gate=t.get("sh_gate"),
                               y=y, topk_idx_out=topk_idx_out, topk_w_out=topk_w_out, counts_out=counts_out,
                               stream=stream)
