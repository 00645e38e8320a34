"""MI355X (gfx950) fine-grained MoE layer: route -> permute -> grouped SwiGLU -> combine.

Thin ctypes binding over libmoe.so (include/moe.h).  Each function marshals
torch CUDA tensors into device pointers and the current HIP stream and calls
the C entry point of the same name; every step of the layer runs in the
library's HIP kernels.  torch supplies device memory and streams only.  If the
library is missing the calls raise: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe.so")

MOE_F32, MOE_BF16, MOE_E4M3_B128, MOE_NVFP4, MOE_MXFP4 = 0, 1, 2, 3, 4
_DTYPES = {"f32": MOE_F32, "bf16": MOE_BF16, "e4m3": MOE_E4M3_B128, "nvfp4": MOE_NVFP4,
           "mxfp4": MOE_MXFP4}


class MoeConfig(ctypes.Structure):
    _fields_ = [("num_tokens", ctypes.c_int64), ("hidden", ctypes.c_int32),
                ("intermediate", ctypes.c_int32), ("num_experts", ctypes.c_int32),
                ("num_groups", ctypes.c_int32), ("topk_groups", ctypes.c_int32),
                ("topk", ctypes.c_int32), ("num_shared", ctypes.c_int32),
                ("act_dtype", ctypes.c_int32), ("weight_dtype", ctypes.c_int32)]


class MoeWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "w_router", "router_bias", "w_gate", "w_up", "w_down", "s_gate", "s_up", "s_down",
        "sh_gate", "sh_up", "sh_down", "sh_s_gate", "sh_s_up", "sh_s_down",
        "b_gate", "b_up", "b_down", "g_gate", "g_up", "g_down",
        "sh_b_gate", "sh_b_up", "sh_b_down", "sh_g_gate", "sh_g_up", "sh_g_down")]


class DenseConfig(ctypes.Structure):
    _fields_ = [("num_tokens", ctypes.c_int64), ("hidden", ctypes.c_int32),
                ("intermediate", ctypes.c_int32), ("act_dtype", ctypes.c_int32)]


class DenseWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("w_gate", "w_up", "w_down", "s_gate", "s_up",
                                               "s_down")]


ENTRY_POINTS = ("moe_workspace_size", "moe_route", "moe_permute", "moe_expert_ffn",
                "moe_combine", "moe_forward", "moe_forward_timed", "moe_forward_residual",
                "moe_workspace_slot", "moe_forward_noalloc", "moe_pager_state_layout",
                "moe_pager_reset", "moe_paged_workspace_size", "moe_forward_paged",
                "moe_norm_quant_rows", "moe_linear_i8", "moe_glu_i8", "moe_dense_workspace_size",
                "moe_dense_residual_i8", "moe_strerror")
ROW_FORMATS = {"rows": 0, "i8": 1, "e4m3": 2, "mxfp8": 3}   # MOE_ROWS_*
NOALLOC_SCRATCH_BYTES = 16 << 20   # MOE_NOALLOC_SCRATCH_BYTES
WS_LOGITS, WS_ACT_CODES, WS_ACT_SCALES, WS_NORM_ROWS = 0, 1, 2, 3   # MOE_WS_* slots
TIMED_EVENTS = 4   # MOE_TIMED_EVENTS: start/stop of the gate/up kernel, start/stop of the down kernel

_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libmoe.so and declare its signatures.  Raises if it is not built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with __graft_entry__.build() "
                           "(hipcc, gfx950); there is no fallback path")
    lib = ctypes.CDLL(path)
    P, SZ = ctypes.c_void_p, ctypes.c_size_t
    cfgp = ctypes.POINTER(MoeConfig)
    wp = ctypes.POINTER(MoeWeights)
    I32, I64 = ctypes.c_int32, ctypes.c_int64
    dcfgp, dwp = ctypes.POINTER(DenseConfig), ctypes.POINTER(DenseWeights)
    sig = {
        "moe_workspace_size": [cfgp, ctypes.POINTER(SZ)],
        "moe_route": [cfgp, P, P, P, P, P, P, P, SZ, P],
        "moe_permute": [cfgp, P, P, P, P, P, SZ, P],
        "moe_expert_ffn": [cfgp, P, P, P, wp, P, P, SZ, P],
        "moe_combine": [cfgp, P, P, P, P, P, P],
        "moe_forward": [cfgp, P, wp, P, P, P, P, SZ, P],
        "moe_forward_timed": [cfgp, P, wp, P, P, P, P, SZ, P, P],
        "moe_forward_residual": [cfgp, P, P, ctypes.c_float, wp, P, P, P, P, SZ, P],
        "moe_workspace_slot": [cfgp, ctypes.c_int, ctypes.POINTER(SZ), ctypes.POINTER(SZ)],
        "moe_forward_noalloc": [cfgp, P, wp, P, P, P, P],
        "moe_pager_state_layout": [cfgp, ctypes.c_int32, ctypes.POINTER(SZ), ctypes.POINTER(SZ)],
        "moe_pager_reset": [cfgp, ctypes.c_int32, P, P],
        "moe_paged_workspace_size": [cfgp, ctypes.c_int32, ctypes.POINTER(SZ)],
        "moe_forward_paged": [cfgp, P, wp, wp, ctypes.c_int32, P, P, P, P, P, SZ, P],
        "moe_norm_quant_rows": [I64, I32, I32, I32, P, P, P, ctypes.c_float, P, P, P, P],
        "moe_linear_i8": [I64, I32, I32, I32, P, P, P, P, P, P, P],
        "moe_glu_i8": [I64, I32, I32, I32, P, P, P, P, P, P, P, P],
        "moe_dense_workspace_size": [dcfgp, ctypes.POINTER(SZ)],
        "moe_dense_residual_i8": [dcfgp, P, P, ctypes.c_float, dwp, P, P, SZ, P],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    lib.moe_strerror.argtypes = [ctypes.c_int]
    lib.moe_strerror.restype = ctypes.c_char_p
    _lib = lib
    return lib


class MoeError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"moe status {status}: {msg}")
        self.status = status


def _check(rc: int) -> None:
    if rc != 0:
        raise MoeError(rc, load_library().moe_strerror(rc).decode())


def make_config(T: int, H: int, I: int, E: int, G: int, Gk: int, k: int, S: int = 0,
                act: str = "bf16", wt: str = "bf16") -> MoeConfig:
    return MoeConfig(T, H, I, E, G, Gk, k, S, _DTYPES[act], _DTYPES[wt])


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("device tensors only")
    if not t.is_contiguous():
        raise ValueError("contiguous tensors only")
    return t.data_ptr()


def _stream() -> int:
    return torch.cuda.current_stream().cuda_stream


def workspace_size(cfg: MoeConfig) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().moe_workspace_size(ctypes.byref(cfg), ctypes.byref(n)))
    return int(n.value)


def workspace_slot(cfg: MoeConfig, slot: int):
    """(byte offset, bytes) of an inspectable workspace slot (MOE_WS_*)."""
    off, n = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(load_library().moe_workspace_slot(ctypes.byref(cfg), slot, ctypes.byref(off),
                                             ctypes.byref(n)))
    return int(off.value), int(n.value)


def alloc_workspace(cfg: MoeConfig, device="cuda") -> torch.Tensor:
    """Caller-owned scratch (torch allocation is 256-byte aligned)."""
    return torch.empty(max(workspace_size(cfg), 256), dtype=torch.uint8, device=device)


def weights_struct(w: dict) -> MoeWeights:
    """Build the weight struct from a dict of CUDA tensors (keys as in moe.h)."""
    return MoeWeights(*[_ptr(w.get(n)) for n, _ in MoeWeights._fields_])


def route(cfg, x, w_router, bias, ws, logits: Optional[torch.Tensor] = None):
    T, k = cfg.num_tokens, cfg.topk
    ids = torch.empty((T, k), dtype=torch.int32, device=x.device)
    wts = torch.empty((T, k), dtype=torch.float32, device=x.device)
    _check(load_library().moe_route(ctypes.byref(cfg), _ptr(x), _ptr(w_router), _ptr(bias),
                                    _ptr(ids), _ptr(wts), _ptr(logits), _ptr(ws), ws.numel(),
                                    _stream()))
    return ids, wts


def permute(cfg, ids, ws):
    T, k, E, S = cfg.num_tokens, cfg.topk, cfg.num_experts, cfg.num_shared
    offsets = torch.empty(E + S + 1, dtype=torch.int32, device=ids.device)
    row_token = torch.empty(T * (k + S), dtype=torch.int32, device=ids.device)
    inv = torch.empty((T, k), dtype=torch.int32, device=ids.device)
    _check(load_library().moe_permute(ctypes.byref(cfg), _ptr(ids), _ptr(offsets), _ptr(row_token),
                                      _ptr(inv), _ptr(ws), ws.numel(), _stream()))
    return offsets, row_token, inv


def expert_ffn(cfg, x, offsets, row_token, weights: dict, ws):
    R = cfg.num_tokens * (cfg.topk + cfg.num_shared)
    y_perm = torch.empty((R, cfg.hidden), dtype=torch.float32, device=x.device)
    wst = weights_struct(weights)
    _check(load_library().moe_expert_ffn(ctypes.byref(cfg), _ptr(x), _ptr(offsets),
                                         _ptr(row_token), ctypes.byref(wst), _ptr(y_perm),
                                         _ptr(ws), ws.numel(), _stream()))
    return y_perm


def combine(cfg, y_perm, offsets, inv, wts, out_dtype):
    y = torch.empty((cfg.num_tokens, cfg.hidden), dtype=out_dtype, device=y_perm.device)
    _check(load_library().moe_combine(ctypes.byref(cfg), _ptr(y_perm), _ptr(offsets), _ptr(inv),
                                      _ptr(wts), _ptr(y), _stream()))
    return y


def forward(cfg, x, weights: dict, ws, y: Optional[torch.Tensor] = None,
            ids: Optional[torch.Tensor] = None, wts: Optional[torch.Tensor] = None,
            wst: Optional[MoeWeights] = None):
    """The whole layer.  Returns y (and writes ids / wts when given)."""
    if y is None:
        y = torch.empty((cfg.num_tokens, cfg.hidden), dtype=x.dtype, device=x.device)
    if wst is None:
        wst = weights_struct(weights)
    _check(load_library().moe_forward(ctypes.byref(cfg), _ptr(x), ctypes.byref(wst), _ptr(y),
                                      _ptr(ids), _ptr(wts), _ptr(ws), ws.numel(), _stream()))
    return y


def forward_noalloc(cfg, x, weights: dict, y: Optional[torch.Tensor] = None,
                    ids: Optional[torch.Tensor] = None, wts: Optional[torch.Tensor] = None,
                    wst: Optional[MoeWeights] = None):
    """The whole layer on the library's own fixed scratch (no workspace argument, no
    allocation inside the call).  Returns y (and writes ids / wts when given)."""
    if y is None:
        y = torch.empty((cfg.num_tokens, cfg.hidden), dtype=x.dtype, device=x.device)
    if wst is None:
        wst = weights_struct(weights)
    _check(load_library().moe_forward_noalloc(ctypes.byref(cfg), _ptr(x), ctypes.byref(wst),
                                              _ptr(y), _ptr(ids), _ptr(wts), _stream()))
    return y


PAGER_COUNTERS = ("calls", "refs", "lookups", "hits", "misses", "bytes_copied")


def pager_state_layout(cfg, num_slots: int):
    """(offsets of counters, key_slot, slot_key, stamp; total bytes) of a pager state."""
    offs = (ctypes.c_size_t * 4)()
    n = ctypes.c_size_t(0)
    _check(load_library().moe_pager_state_layout(ctypes.byref(cfg), num_slots, offs,
                                                 ctypes.byref(n)))
    return tuple(int(v) for v in offs), int(n.value)


def alloc_pager_state(cfg, num_slots: int, device="cuda") -> torch.Tensor:
    """A pager state, initialised (empty arena, zero counters) on the current stream."""
    _, n = pager_state_layout(cfg, num_slots)
    state = torch.empty(n, dtype=torch.uint8, device=device)
    _check(load_library().moe_pager_reset(ctypes.byref(cfg), num_slots, _ptr(state), _stream()))
    return state


def pager_tables(cfg, num_slots: int, state: torch.Tensor) -> dict:
    """Counters and residency tables of a pager state, copied to the host."""
    (oc, ok, osl, ost), _ = pager_state_layout(cfg, num_slots)
    raw = state.cpu()
    E = cfg.num_experts
    c = raw[oc:oc + 64].view(torch.int64).tolist()
    out = dict(zip(PAGER_COUNTERS, c))
    out["key_slot"] = raw[ok:ok + 4 * E].view(torch.int32).numpy().copy()
    out["slot_key"] = raw[osl:osl + 4 * num_slots].view(torch.int32).numpy().copy()
    out["stamp"] = raw[ost:ost + 8 * num_slots].view(torch.int64).numpy().copy()
    return out


def paged_workspace(cfg, num_slots: int, device="cuda") -> torch.Tensor:
    n = ctypes.c_size_t(0)
    _check(load_library().moe_paged_workspace_size(ctypes.byref(cfg), num_slots, ctypes.byref(n)))
    return torch.empty(max(int(n.value), 256), dtype=torch.uint8, device=device)


def forward_paged(cfg, x, host_experts: MoeWeights, resident: MoeWeights, num_slots: int,
                  state, ws, y: Optional[torch.Tensor] = None, ids: Optional[torch.Tensor] = None,
                  wts: Optional[torch.Tensor] = None):
    """The layer with its routed experts paged from pinned host memory into an arena of
    `num_slots` slots (device-side decisions).  `host_experts` holds host pointers
    (pinned tensors: use weights_struct_host), `resident` device pointers."""
    if y is None:
        y = torch.empty((cfg.num_tokens, cfg.hidden), dtype=x.dtype, device=x.device)
    _check(load_library().moe_forward_paged(ctypes.byref(cfg), _ptr(x), ctypes.byref(host_experts),
                                            ctypes.byref(resident), num_slots, _ptr(state),
                                            _ptr(y), _ptr(ids), _ptr(wts), _ptr(ws), ws.numel(),
                                            _stream()))
    return y


def weights_struct_host(w: dict) -> MoeWeights:
    """Weight struct of pinned host tensors (the paged layer's expert store)."""
    def hp(t):
        if t is None:
            return None
        if not (t.is_pinned() and t.is_contiguous()):
            raise ValueError("the expert store must be contiguous pinned host tensors")
        return t.data_ptr()
    return MoeWeights(*[hp(w.get(n)) for n, _ in MoeWeights._fields_])


def forward_residual(cfg, x, norm_weight, weights: dict, ws, x_out: Optional[torch.Tensor] = None,
                     eps: float = 1e-6, ids: Optional[torch.Tensor] = None,
                     wts: Optional[torch.Tensor] = None, wst: Optional[MoeWeights] = None):
    """The decoder step around the layer: x_out = x + MoE(RMSNorm(x) * norm_weight).
    x_out may be x itself.  Returns x_out (and writes ids / wts when given)."""
    if x_out is None:
        x_out = torch.empty_like(x)
    if wst is None:
        wst = weights_struct(weights)
    _check(load_library().moe_forward_residual(ctypes.byref(cfg), _ptr(x), _ptr(norm_weight),
                                               ctypes.c_float(eps), ctypes.byref(wst),
                                               _ptr(x_out), _ptr(ids), _ptr(wts), _ptr(ws),
                                               ws.numel(), _stream()))
    return x_out


def forward_timed(cfg, x, wst: MoeWeights, ws, y, events_array) -> None:
    """moe_forward with start/stop events attached to the gate/up and down kernel
    dispatches.  `events_array` is a ctypes array of MOE_TIMED_EVENTS hipEvent_t
    handles (timing events: torch.cuda.Event(enable_timing=True).cuda_event, or events
    created with hipEventDisableSystemFence, as bench.py does)."""
    _check(load_library().moe_forward_timed(ctypes.byref(cfg), _ptr(x), ctypes.byref(wst), _ptr(y),
                                            None, None, _ptr(ws), ws.numel(), _stream(),
                                            events_array))


# ------------------------------------------------------------- dense operators in 8 bits

_ACT = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}


def _raw_stream(dev: int) -> int:
    """The current stream of device `dev` (what _stream() gives, at a tenth of its cost)."""
    return torch._C._cuda_getCurrentRawStream(dev)


def _device() -> int:
    """The current device's index (-2, which no tensor has, before there is one)."""
    return torch._C._cuda_getDevice() if torch.cuda._initialized else -2


def _arg(name: str, t: torch.Tensor, shape: tuple, dtype: torch.dtype, dev: int) -> int:
    """Device pointer of a contiguous tensor of exactly this shape and type on the current
    device (the library launches on that device and checks nothing behind a pointer).  A call
    makes up to seven of these checks beside a launch of a few microseconds, so they use the
    cheapest accessors there are (get_device() of a host tensor is -1)."""
    if (t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous()):
        return t.data_ptr()
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name}: expected {dtype} {shape}, got {t.dtype} {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: expected a tensor on the current device, got {t.device}")
    raise ValueError(f"{name}: contiguous tensors only")


def _act_dtype(name: str, dtype: torch.dtype) -> int:
    if dtype not in _ACT:
        raise ValueError(f"{name}: float32 or bfloat16 only, got {dtype}")
    return _ACT[dtype]


def _rows_of(name: str, t: torch.Tensor):
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name}: expected [rows, width], got {tuple(shape)}")
    return shape


def norm_quant_rows(x, fmt: str, norm_weight: Optional[torch.Tensor] = None,
                    residual: Optional[torch.Tensor] = None, eps: float = 1e-6,
                    x_sum: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                    scales: Optional[torch.Tensor] = None):
    """Residual add, RMSNorm and output format of rows in one kernel (moe_norm_quant_rows).
    `fmt`: "rows" (x's type), "i8" (int8 codes, fp32 scale per row), "e4m3" (uint8 codes, fp32
    scale per 128 columns) or "mxfp8" (uint8 codes, uint8 E8M0 scale per 32).  Without
    norm_weight the (summed) rows themselves are converted.  x_sum may be x or residual, a
    "rows" out too.  Returns (out, scales or None, x_sum or None)."""
    T, H = _rows_of("x", x)
    dev = _device()
    act = _act_dtype("x", x.dtype)
    if fmt not in ROW_FORMATS:
        raise ValueError(f"fmt: one of {tuple(ROW_FORMATS)}, got {fmt!r}")
    xp = _arg("x", x, (T, H), x.dtype, dev)
    rp = sp = cp = gp = None
    if norm_weight is not None:
        gp = _arg("norm_weight", norm_weight, (H,), x.dtype, dev)
    if residual is not None:
        rp = _arg("residual", residual, (T, H), x.dtype, dev)
        if x_sum is None:
            x_sum = x.new_empty((T, H))
            sp = x_sum.data_ptr()
        else:
            sp = _arg("x_sum", x_sum, (T, H), x.dtype, dev)
    else:
        x_sum = None
    odt = x.dtype if fmt == "rows" else torch.int8 if fmt == "i8" else torch.uint8
    if out is None:
        out = x.new_empty((T, H), dtype=odt)
        op = out.data_ptr()
    else:
        op = _arg("out", out, (T, H), odt, dev)
    if fmt == "rows":
        scales = None
    else:
        shape = (T,) if fmt == "i8" else (T, H // 128) if fmt == "e4m3" else (T, H // 32)
        sdt = torch.uint8 if fmt == "mxfp8" else torch.float32
        if scales is None:
            scales = x.new_empty(shape, dtype=sdt)
            cp = scales.data_ptr()
        else:
            cp = _arg("scales", scales, shape, sdt, dev)
    _check(load_library().moe_norm_quant_rows(T, H, act, ROW_FORMATS[fmt], xp, rp, gp, eps, sp, op,
                                              cp, _raw_stream(dev)))
    return out, scales, x_sum


def linear_i8(x_codes, x_scales, w_codes, w_scales, out_dtype=torch.bfloat16,
              residual: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None):
    """y = (x_codes @ w_codes.T) * x_scales[:, None] * w_scales (+ residual): int8 [T, K] and
    [N, K] codes, fp32 scales per token and per channel, y [T, N] bf16 or fp32
    (moe_linear_i8).  residual may be y itself."""
    T, K = _rows_of("x_codes", x_codes)
    N = _rows_of("w_codes", w_codes)[0]
    dev = _device()
    out = _act_dtype("out_dtype", out_dtype)
    xp = _arg("x_codes", x_codes, (T, K), torch.int8, dev)
    sp = _arg("x_scales", x_scales, (T,), torch.float32, dev)
    wp = _arg("w_codes", w_codes, (N, K), torch.int8, dev)
    cp = _arg("w_scales", w_scales, (N,), torch.float32, dev)
    rp = None if residual is None else _arg("residual", residual, (T, N), out_dtype, dev)
    if y is None:
        y = x_codes.new_empty((T, N), dtype=out_dtype)
        yp = y.data_ptr()
    else:
        yp = _arg("y", y, (T, N), out_dtype, dev)
    _check(load_library().moe_linear_i8(T, K, N, out, xp, sp, wp, cp, rp, yp, _raw_stream(dev)))
    return y


def glu_i8(x_codes, x_scales, w_gate, s_gate, w_up, s_up, out_dtype=torch.bfloat16,
           h: Optional[torch.Tensor] = None):
    """h = silu(g) * u with g and u the two 8-bit products of linear_i8, in one kernel
    (moe_glu_i8).  Returns h [T, N] bf16 or fp32."""
    T, K = _rows_of("x_codes", x_codes)
    N = _rows_of("w_gate", w_gate)[0]
    dev = _device()
    out = _act_dtype("out_dtype", out_dtype)
    xp = _arg("x_codes", x_codes, (T, K), torch.int8, dev)
    sp = _arg("x_scales", x_scales, (T,), torch.float32, dev)
    gp = _arg("w_gate", w_gate, (N, K), torch.int8, dev)
    gs = _arg("s_gate", s_gate, (N,), torch.float32, dev)
    up = _arg("w_up", w_up, (N, K), torch.int8, dev)
    us = _arg("s_up", s_up, (N,), torch.float32, dev)
    if h is None:
        h = x_codes.new_empty((T, N), dtype=out_dtype)
        hp = h.data_ptr()
    else:
        hp = _arg("h", h, (T, N), out_dtype, dev)
    _check(load_library().moe_glu_i8(T, K, N, out, xp, sp, gp, gs, up, us, hp, _raw_stream(dev)))
    return h


def make_dense_config(T: int, H: int, I: int, act: str = "bf16") -> DenseConfig:
    return DenseConfig(T, H, I, _DTYPES[act])


def dense_workspace_size(cfg: DenseConfig) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().moe_dense_workspace_size(ctypes.byref(cfg), ctypes.byref(n)))
    return int(n.value)


def alloc_dense_workspace(cfg: DenseConfig, device="cuda") -> torch.Tensor:
    return torch.empty(max(dense_workspace_size(cfg), 256), dtype=torch.uint8, device=device)


def dense_weights_struct(w: dict) -> DenseWeights:
    """Weight struct of a dict of CUDA tensors: w_gate, w_up [I, H] and w_down [H, I] int8,
    s_gate, s_up [I] and s_down [H] fp32.  It holds pointers only: keep the tensors alive.  Its
    sizes and device stay with it, for dense_residual_i8 to compare."""
    I, H = _rows_of("w_gate", w["w_gate"])
    dev = _device()
    shapes = {"w_gate": (I, H), "w_up": (I, H), "w_down": (H, I), "s_gate": (I,), "s_up": (I,),
              "s_down": (H,)}
    wst = DenseWeights(*[_arg(n, w[n], shapes[n], torch.int8 if n[0] == "w" else torch.float32, dev)
                         for n, _ in DenseWeights._fields_])
    wst.made_for = (H, I, dev)
    return wst


def dense_residual_i8(cfg: DenseConfig, x, norm_weight, wst: DenseWeights, ws,
                      x_out: Optional[torch.Tensor] = None, eps: float = 1e-6):
    """A dense decoder layer's feed-forward block in 8 bits: x_out = x + down(i8(glu(i8(
    RMSNorm(x) * norm_weight)))) (moe_dense_residual_i8).  x_out may be x itself."""
    T, H = cfg.num_tokens, cfg.hidden
    dev = _device()
    dtype = torch.float32 if cfg.act_dtype == MOE_F32 else torch.bfloat16
    xp = _arg("x", x, (T, H), dtype, dev)
    gp = _arg("norm_weight", norm_weight, (H,), dtype, dev)
    if x_out is None:
        x_out = x.new_empty((T, H))
        op = x_out.data_ptr()
    else:
        op = _arg("x_out", x_out, (T, H), dtype, dev)
    wp = _arg("ws", ws, (ws.numel(),), torch.uint8, dev)
    if getattr(wst, "made_for", (H, cfg.intermediate, dev)) != (H, cfg.intermediate, dev):
        raise ValueError(f"wst: made for (hidden, intermediate, device) {wst.made_for}, the call "
                         f"has {(H, cfg.intermediate, dev)}")
    _check(load_library().moe_dense_residual_i8(ctypes.byref(cfg), xp, gp, eps, ctypes.byref(wst),
                                                op, wp, ws.numel(), _raw_stream(dev)))
    return x_out
