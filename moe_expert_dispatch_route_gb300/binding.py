"""Python binding of libmoe_gb300 (ctypes): the C ABI's calls under the same names.

Argument marshalling only -- every step of the layer runs in the library's CUDA
kernels.  Tensors are torch CUDA tensors (PyTorch supplies device memory and
streams); a call returns after enqueueing, like the C call.  A non-zero
``moe_status`` raises :class:`MoeError`.  Importing this module loads the in-tree
shared library and fails loudly when it is missing or cannot be built.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import build as _build

F32, BF16, FP8_E4M3 = 0, 1, 2
GATE_SOFTMAX, GATE_SIGMOID_GROUPED, GATE_SQRT_SOFTPLUS = 0, 1, 2
STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_ALIGNMENT",
          4: "MOE_ERR_WORKSPACE", 5: "MOE_ERR_CUDA", 6: "MOE_ERR_CAPACITY", 7: "MOE_ERR_BAD_INDEX",
          8: "MOE_ERR_TIMEOUT"}
OPS = {0: "route", 1: "plan", 2: "dispatch", 3: "ffn", 4: "combine", 5: "record", 6: "wait", 7: "standin"}


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        super().__init__(f"{where}: {STATUS.get(self.status, self.status)}")


class MoeConfig(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("num_experts", ctypes.c_int32), ("num_shared", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("gate", ctypes.c_int32),
                ("renormalize", ctypes.c_int32), ("n_group", ctypes.c_int32),
                ("topk_group", ctypes.c_int32), ("routed_scale", ctypes.c_float),
                ("dtype", ctypes.c_int32)]


class MoeStackArgs(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("out", ctypes.c_void_p), ("logits", ctypes.c_void_p),
                ("bias", ctypes.c_void_p), ("wa", ctypes.c_void_p), ("w13", ctypes.c_void_p),
                ("w13_scale", ctypes.c_void_p), ("w2", ctypes.c_void_p), ("w2_scale", ctypes.c_void_p),
                ("err_flag", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t)]


class MoeLayerArgs(ctypes.Structure):
    _fields_ = [("logits", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("x", ctypes.c_void_p),
                ("w13", ctypes.c_void_p), ("w13_scale", ctypes.c_void_p), ("w2", ctypes.c_void_p),
                ("w2_scale", ctypes.c_void_p), ("y", ctypes.c_void_p), ("topk_ids", ctypes.c_void_p),
                ("topk_w", ctypes.c_void_p), ("err_flag", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


class MoeKvCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("num_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("stride_page", ctypes.c_int64), ("stride_head", ctypes.c_int64), ("stride_token", ctypes.c_int64)]


class MoeAttnArgs(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("o", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("q_ld", ctypes.c_int64), ("q_head_stride", ctypes.c_int64), ("o_ld", ctypes.c_int64),
                ("o_head_stride", ctypes.c_int64), ("cu_q", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("table_ld", ctypes.c_int32), ("T", ctypes.c_int32),
                ("B", ctypes.c_int32), ("max_q", ctypes.c_int32), ("max_kv", ctypes.c_int32),
                ("num_q_heads", ctypes.c_int32), ("scale", ctypes.c_float), ("causal", ctypes.c_int32),
                ("window", ctypes.c_int32), ("err_flag", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t)]


class MoeLatentCache(ctypes.Structure):
    _fields_ = [("kv", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("latent", ctypes.c_int32), ("rope", ctypes.c_int32),
                ("stride_page", ctypes.c_int64), ("stride_token", ctypes.c_int64)]


class MoeAttnExpandedArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "k", "k_rope", "v", "o", "lse")] + \
               [(n, ctypes.c_int64) for n in ("q_ld", "q_head_stride", "k_ld", "k_head_stride", "rope_ld", "v_ld",
                                              "v_head_stride", "o_ld", "o_head_stride")] + \
               [("cu_q", ctypes.c_void_p), ("cu_kv", ctypes.c_void_p), ("T", ctypes.c_int32), ("S", ctypes.c_int32),
                ("B", ctypes.c_int32), ("max_q", ctypes.c_int32), ("max_kv", ctypes.c_int32),
                ("num_heads", ctypes.c_int32), ("scale", ctypes.c_float), ("causal", ctypes.c_int32),
                ("err_flag", ctypes.c_void_p), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


class MoeNormArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("y", "post_weight", "gate", "resid", "resid_out", "pre_weight", "out")] + \
               [(n, ctypes.c_int32) for n in ("T", "hidden", "dtype", "resid_dtype", "gate_rows")] + \
               [("scale", ctypes.c_float), ("eps", ctypes.c_float)]


def config(hidden, inter, num_experts, num_shared, top_k, gate=GATE_SOFTMAX, renormalize=1,
           n_group=1, topk_group=1, routed_scale=1.0, dtype=BF16) -> MoeConfig:
    return MoeConfig(hidden, inter, num_experts, num_shared, top_k, gate, int(renormalize), n_group,
                     topk_group, float(routed_scale), dtype)


def config_of(wl) -> MoeConfig:
    """MoeConfig of a workloads.Workload."""
    gate = {"softmax": GATE_SOFTMAX, "sigmoid_grouped": GATE_SIGMOID_GROUPED, "sqrt_softplus": GATE_SQRT_SOFTPLUS}
    return config(wl.hidden, wl.inter, wl.num_experts, wl.num_shared, wl.top_k, gate[wl.gate],
                  int(wl.renormalize), wl.n_group, wl.topk_group, wl.routed_scale,
                  {"f32": F32, "bf16": BF16, "fp8": FP8_E4M3}[wl.dtype])


_P, _I32, _I64, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
_CFG = ctypes.POINTER(MoeConfig)
_CACHE = ctypes.POINTER(MoeKvCache)
_LATENT = ctypes.POINTER(MoeLatentCache)
_SIGS = {
    "moe_route": (_I32, [_CFG, _I32, _P, _P, _P, _P, _I32, _P]),
    "moe_route_hash": (_I32, [_CFG, _I32, _P, _P, _P, _I32, _P, _P, _I32, _P]),
    "moe_plan_rows": (_SZ, [_CFG, _I32, _I32, _I32]),
    "moe_plan_workspace_size": (_SZ, [_CFG, _I32]),
    "moe_plan": (_I32, [_CFG, _I32, _P, _I32, _I32, _P, _P, _P, _P, _P, _P, _SZ, _I32, _P]),
    "moe_plan_noalloc": (_I32, [_CFG, _I32, _P, _I32, _I32, _P, _P, _P, _P, _P, _I32, _P]),
    "moe_dispatch": (_I32, [_CFG, _I32, _P, _P, _P, _P, _I64, _I32, _P]),
    "moe_ffn_workspace_size": (_SZ, [_CFG, _I64]),
    "moe_expert_ffn": (_I32, [_CFG, _P, _P, _I64, _P, _P, _I64, _P, _P, _P, _P, _P, _P, _SZ, _P, _I32, _P]),
    "moe_combine": (_I32, [_CFG, _I32, _P, _P, _P, _P, _I32, _P]),
    "moe_dbo_create": (_I32, [ctypes.POINTER(_P)]),
    "moe_dbo_destroy": (None, [_P]),
    "moe_layer_workspace_size": (_SZ, [_CFG, _I32, _I32, _I32]),
    "moe_layer_dbo": (_I32, [_P, _CFG, ctypes.POINTER(MoeLayerArgs), _I32, _I32, _I32, _I32, _I32, _I32,
                             _P, _P]),
    "moe_dbo_schedule": (_I32, [_I32, _P, _I32]),
    "moe_layer_dbo_ex": (_I32, [_P, _CFG, ctypes.POINTER(MoeLayerArgs), _I32, _I32, _I32, _I32, _I32, _I32, _I32,
                                _P, _P]),
    "moe_dbo_schedule_ex": (_I32, [_I32, _I32, _P, _I32]),
    "moe_stack_workspace_size": (_SZ, [_CFG, _I32, _I32, _I32]),
    "moe_stack_dbo": (_I32, [_P, _CFG, ctypes.POINTER(MoeStackArgs), _I32, _I32, _I32, _I32, _I32, _I32, _I32,
                             _I32, _P, _P]),
    "moe_stack_schedule": (_I32, [_I32, _I32, _I32, _P, _I32]),
    "moe_status_string": (ctypes.c_char_p, [_I32]),
    "moe_debug_inject_wait": (_I32, [_I32, _I64]),
    "moe_comm_error": (_I32, [_P, _I32]),
    "moe_kv_write": (_I32, [_CACHE, _I32, _P, _P, _I64, _I64, _I64, _P, _P, _I32, _P]),
    "moe_kv_read": (_I32, [_CACHE, _I32, _I32, _P, _I32, _P, _P, _P, _P, _P, _I32, _P]),
    "moe_attn_workspace_size": (_SZ, [_CACHE, _I32]),
    "moe_attn_paged": (_I32, [_CACHE, ctypes.POINTER(MoeAttnArgs), _I32, _P]),
    "moe_attn_tree": (_I32, [_CACHE, ctypes.POINTER(MoeAttnArgs), _P, _I32, _P]),
    "moe_latent_write": (_I32, [_LATENT, _I32, _P, _I64, _P, _I64, _P, ctypes.c_float, _P, _P, _I32, _P]),
    "moe_attn_latent_workspace_size": (_SZ, [_LATENT, _I32]),
    "moe_attn_latent": (_I32, [_LATENT, ctypes.POINTER(MoeAttnArgs), _P, _I32, _P]),
    "moe_attn_expanded_workspace_size": (_SZ, [_I32]),
    "moe_attn_expanded": (_I32, [ctypes.POINTER(MoeAttnExpandedArgs), _I32, _P]),
    "moe_block_norm": (_I32, [ctypes.POINTER(MoeNormArgs), _I32, _P]),
    "moe_draft_verify": (_I32, [_I32, _I32, _I32, _I32, _P, _I64, _P, _I64, _P, _P, _P, _P, _P, _P, _P, _I32, _P]),
    "moe_draft_verify_ex": (_I32, [_I32, _I32, _I32, _I32, _I32, _P, _I64, _P, _I64, _P, _P, _P, _P, _P, _P, _P, _I32,
                                   _P]),
}
EXPORTS = tuple(_SIGS)

_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libmoe_gb300 (built in-tree on first use if stale or missing)."""
    global _lib
    if _lib is None:
        path = _build.build()
        if not os.path.exists(path):
            raise ImportError(f"libmoe_gb300 not found at {path}")
        L = ctypes.CDLL(path)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def library_path() -> str:
    return _build.LIB


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(s):
    if s is None:  # torch.cuda.current_stream().cuda_stream, without the Stream object (3 us)
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(st: int, where: str):
    if st != 0:
        raise MoeError(st, where)


def moe_route(cfg, T, logits, bias, topk_ids, topk_w, max_ctas=0, stream=None):
    _check(lib().moe_route(ctypes.byref(cfg), T, _ptr(logits), _ptr(bias), _ptr(topk_ids), _ptr(topk_w),
                           max_ctas, _stream(stream)), "moe_route")


def moe_route_hash(cfg, T, logits, token_ids, table, topk_ids, topk_w, max_ctas=0, stream=None):
    vocab = table.shape[0] if table is not None else 0
    _check(lib().moe_route_hash(ctypes.byref(cfg), T, _ptr(logits), _ptr(token_ids), _ptr(table), vocab,
                                _ptr(topk_ids), _ptr(topk_w), max_ctas, _stream(stream)), "moe_route_hash")


def moe_plan_rows(cfg, T, capacity=0, align=1) -> int:
    return int(lib().moe_plan_rows(ctypes.byref(cfg), T, capacity, align))


def moe_plan_workspace_size(cfg, T) -> int:
    return int(lib().moe_plan_workspace_size(ctypes.byref(cfg), T))


def moe_plan(cfg, T, topk_ids, capacity, align, counts, offsets, slot_of, token_of, err_flag, ws=None,
             ws_bytes=0, max_ctas=0, stream=None):
    if ws is not None and not ws_bytes:
        ws_bytes = ws.numel() * ws.element_size()
    _check(lib().moe_plan(ctypes.byref(cfg), T, _ptr(topk_ids), capacity, align, _ptr(counts), _ptr(offsets),
                          _ptr(slot_of), _ptr(token_of), _ptr(err_flag), _ptr(ws), ws_bytes, max_ctas,
                          _stream(stream)), "moe_plan")


def moe_plan_noalloc(cfg, T, topk_ids, capacity, align, counts, offsets, slot_of, token_of, err_flag,
                     max_ctas=0, stream=None):
    """moe_plan without a workspace (scratch lives in the library; see moe.h for the limit)."""
    _check(lib().moe_plan_noalloc(ctypes.byref(cfg), T, _ptr(topk_ids), capacity, align, _ptr(counts),
                                  _ptr(offsets), _ptr(slot_of), _ptr(token_of), _ptr(err_flag), max_ctas,
                                  _stream(stream)), "moe_plan_noalloc")


def moe_dispatch(cfg, T, x, slot_of, xe, xe_scale=None, max_ctas=0, stream=None, xe_scale_ld=0):
    _check(lib().moe_dispatch(ctypes.byref(cfg), T, _ptr(x), _ptr(slot_of), _ptr(xe), _ptr(xe_scale),
                              xe_scale_ld, max_ctas, _stream(stream)), "moe_dispatch")


def moe_ffn_workspace_size(cfg, max_rows) -> int:
    return int(lib().moe_ffn_workspace_size(ctypes.byref(cfg), max_rows))


def moe_expert_ffn(cfg, counts, offsets, max_rows, xe, xe_scale, w13, w13_scale, w2, w2_scale, ye, ws,
                   ws_bytes=0, err_flag=None, max_ctas=0, stream=None, xe_scale_ld=0):
    if ws is not None and not ws_bytes:
        ws_bytes = ws.numel() * ws.element_size()
    _check(lib().moe_expert_ffn(ctypes.byref(cfg), _ptr(counts), _ptr(offsets), max_rows, _ptr(xe),
                                _ptr(xe_scale), xe_scale_ld, _ptr(w13), _ptr(w13_scale), _ptr(w2), _ptr(w2_scale),
                                _ptr(ye), _ptr(ws), ws_bytes, _ptr(err_flag), max_ctas, _stream(stream)),
           "moe_expert_ffn")


def moe_combine(cfg, T, ye, topk_w, slot_of, y, max_ctas=0, stream=None):
    _check(lib().moe_combine(ctypes.byref(cfg), T, _ptr(ye), _ptr(topk_w), _ptr(slot_of), _ptr(y), max_ctas,
                             _stream(stream)), "moe_combine")


def moe_dbo_create() -> int:
    h = ctypes.c_void_p()
    _check(lib().moe_dbo_create(ctypes.byref(h)), "moe_dbo_create")
    return h.value


def moe_dbo_destroy(h: int):
    lib().moe_dbo_destroy(h)


def moe_layer_workspace_size(cfg, T, capacity=0, align=128) -> int:
    return int(lib().moe_layer_workspace_size(ctypes.byref(cfg), T, capacity, align))


def moe_layer_dbo(handle, cfg, args: MoeLayerArgs, T, split=0, min_tokens=4, capacity=0, align=128,
                  comm_sms=0, compute=None, comm=None):
    cs = _stream(compute)
    ms = _stream(comm) if comm is not None else cs
    _check(lib().moe_layer_dbo(handle, ctypes.byref(cfg), ctypes.byref(args), T, split, min_tokens, capacity,
                               align, comm_sms, cs, ms), "moe_layer_dbo")


LAYER_FUSED_GATHER, LAYER_FUSED_COMBINE, LAYER_FUSED = 1, 2, 3


def moe_layer_dbo_ex(handle, cfg, args: MoeLayerArgs, T, split=0, min_tokens=4, capacity=0, align=128,
                     comm_sms=0, flags=0, compute=None, comm=None):
    cs = _stream(compute)
    ms = _stream(comm) if comm is not None else cs
    _check(lib().moe_layer_dbo_ex(handle, ctypes.byref(cfg), ctypes.byref(args), T, split, min_tokens, capacity,
                                  align, comm_sms, flags, cs, ms), "moe_layer_dbo_ex")


def moe_dbo_schedule(two_ubatches: bool, flags: int = 0):
    n = lib().moe_dbo_schedule_ex(int(two_ubatches), flags, None, 0)
    buf = (ctypes.c_int32 * (4 * n))()
    lib().moe_dbo_schedule_ex(int(two_ubatches), flags, buf, n)
    return [tuple(buf[4 * i:4 * i + 4]) for i in range(n)]


def moe_debug_inject_wait(enable: bool, timeout_ns: int = 0):
    """Test hook: FFN and combine kernels launched while enabled let a bounded wait run
    out (see moe.h)."""
    _check(lib().moe_debug_inject_wait(int(enable), int(timeout_ns)), "moe_debug_inject_wait")


def moe_comm_error(clear: bool = False) -> int:
    """The sticky error word of moe_combine (synchronises the device)."""
    code = ctypes.c_int32(0)
    _check(lib().moe_comm_error(ctypes.byref(code), int(clear)), "moe_comm_error")
    return int(code.value)


def moe_status_string(st: int) -> str:
    return lib().moe_status_string(st).decode()


def layer_args(logits, x, weights: dict, y, topk_ids, topk_w, workspace, bias=None, err_flag=None):
    """MoeLayerArgs from tensors (weights: {"w13","w2"} or {"w13_q","w13_s","w2_q","w2_s"})."""
    w13 = weights.get("w13", weights.get("w13_q"))
    w2 = weights.get("w2", weights.get("w2_q"))
    return MoeLayerArgs(_ptr(logits), _ptr(bias), _ptr(x), _ptr(w13), _ptr(weights.get("w13_s")), _ptr(w2),
                        _ptr(weights.get("w2_s")), _ptr(y), _ptr(topk_ids), _ptr(topk_w), _ptr(err_flag),
                        _ptr(workspace), workspace.numel() * workspace.element_size())


def moe_stack_workspace_size(cfg, T, capacity=0, align=128) -> int:
    return int(lib().moe_stack_workspace_size(ctypes.byref(cfg), T, capacity, align))


class StackArgs:
    """moe_stack_args from tensors; keeps the host pointer arrays alive.
    layers: list of dicts with "logits", "wa" and the weights ({"w13","w2"} or fp8 keys)."""

    def __init__(self, x, out, layers, workspace, bias=None, err_flag=None):
        L = len(layers)
        arr = lambda vals: (ctypes.c_void_p * L)(*[_ptr(v) for v in vals])
        self._keep = [arr([ly["logits"] for ly in layers]), arr([ly["wa"] for ly in layers]),
                      arr([ly.get("w13", ly.get("w13_q")) for ly in layers]),
                      arr([ly.get("w13_s") for ly in layers]),
                      arr([ly.get("w2", ly.get("w2_q")) for ly in layers]),
                      arr([ly.get("w2_s") for ly in layers])]
        lg, wa, w13, w13s, w2, w2s = self._keep
        self.c = MoeStackArgs(_ptr(x), _ptr(out), ctypes.cast(lg, ctypes.c_void_p), _ptr(bias),
                              ctypes.cast(wa, ctypes.c_void_p), ctypes.cast(w13, ctypes.c_void_p),
                              ctypes.cast(w13s, ctypes.c_void_p), ctypes.cast(w2, ctypes.c_void_p),
                              ctypes.cast(w2s, ctypes.c_void_p), _ptr(err_flag), _ptr(workspace),
                              workspace.numel() * workspace.element_size())
        self.L = L


def moe_stack_dbo(handle, cfg, args: StackArgs, T, split=0, min_tokens=4, capacity=0, align=128, comm_sms=0,
                  event_before_yield=1, compute=None, comm=None):
    cs = _stream(compute)
    ms = _stream(comm) if comm is not None else cs
    _check(lib().moe_stack_dbo(handle, ctypes.byref(cfg), ctypes.byref(args.c), args.L, T, split, min_tokens,
                               capacity, align, comm_sms, int(event_before_yield), cs, ms), "moe_stack_dbo")


def moe_stack_schedule(layers: int, two_ubatches: bool = True, event_before_yield: bool = True):
    n = lib().moe_stack_schedule(layers, int(two_ubatches), int(event_before_yield), None, 0)
    buf = (ctypes.c_int32 * (4 * n))()
    lib().moe_stack_schedule(layers, int(two_ubatches), int(event_before_yield), buf, n)
    return [tuple(buf[4 * i:4 * i + 4]) for i in range(n)]


# ---------------------------------------------------------------- serving around the layer
def _same(what, *pairs):
    """Raises ValueError unless every (got, want) pair agrees: shapes and types that the C call,
    which sees pointers only, cannot check."""
    for got, want in pairs:
        if got != want:
            raise ValueError(f"{what}: got {got}, expected {want}")


def _vector(what, t, dtype, n):
    if t.dtype is not dtype or t.dim() != 1 or t.size(0) != n or not t.is_contiguous():
        raise ValueError(f"{what}: a packed {dtype} vector of {n} is expected, got {t.dtype} {tuple(t.shape)}")


def kv_cache(k, v, k_scale=None, v_scale=None) -> MoeKvCache:
    """The cache in pools k and v [pages][heads][page_size][head_dim] (any strides, head_dim
    contiguous: a pool kept as [pages][page_size][heads][head_dim] is passed transposed).  bf16,
    or float8_e4m3fn / uint8 codes with packed uint8 scale exponents [pages][heads][page_size].
    The tensors must outlive the cache."""
    fp8 = k.dtype in (torch.float8_e4m3fn, torch.uint8)
    if not fp8 and k.dtype != torch.bfloat16:
        raise ValueError(f"kv_cache: bf16 or e4m3 pools are expected, got {k.dtype}")
    if k.dim() != 4 or k.stride(3) != 1:
        raise ValueError("kv_cache: pools are [pages][heads][page_size][head_dim] with head_dim contiguous")
    _same("kv_cache: v", (v.dtype, k.dtype), (v.shape, k.shape), (v.stride(), k.stride()))
    if fp8 != (k_scale is not None) or fp8 != (v_scale is not None):
        raise ValueError("kv_cache: e4m3 pools come with scales, bf16 pools without")
    for s in (k_scale, v_scale):
        if s is not None:
            _same("kv_cache: scales", (s.dtype, torch.uint8), (s.shape, k.shape[:3]), (s.is_contiguous(), True))
    return MoeKvCache(_ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale), FP8_E4M3 if fp8 else BF16, k.shape[0],
                      k.shape[2], k.shape[1], k.shape[3], k.stride(0), k.stride(1), k.stride(2))


def moe_kv_write(cache: MoeKvCache, k, v, slots, err_flag=None, max_ctas=0, stream=None):
    """Stores k, v [T][heads][head_dim] (bf16, any token and head strides) at slots int64 [T]."""
    shape = k.shape
    T = shape[0]
    if shape != (T, cache.num_heads, cache.head_dim) or v.shape != shape or not (k.dtype is v.dtype is torch.bfloat16):
        raise ValueError(f"moe_kv_write: k and v are bf16 {(T, cache.num_heads, cache.head_dim)}, got {k.dtype} "
                         f"{tuple(shape)} and {v.dtype} {tuple(v.shape)}")
    k0, k1, k2 = k.stride()
    v0, v1, v2 = v.stride()
    if k2 != 1 or v2 != 1 or k1 != v1:
        raise ValueError("moe_kv_write: head_dim is contiguous and the head stride the same for k and v")
    _vector("moe_kv_write: slots", slots, torch.int64, T)
    _check(lib().moe_kv_write(ctypes.byref(cache), T, k.data_ptr(), v.data_ptr(), k0, v0, k1, slots.data_ptr(),
                              _ptr(err_flag), max_ctas, _stream(stream)), "moe_kv_write")


def moe_kv_read(cache: MoeKvCache, block_table, start, cu_len, k_out, v_out, err_flag=None, max_ctas=0, stream=None):
    """Cached tokens [start[b], start[b] + n_b) of every request to rows of k_out, v_out (bf16)."""
    B, shape = start.size(0), k_out.shape
    if shape != (shape[0], cache.num_heads, cache.head_dim) or v_out.shape != shape or \
            not (k_out.dtype is v_out.dtype is torch.bfloat16) or not (k_out.is_contiguous() and v_out.is_contiguous()):
        raise ValueError(f"moe_kv_read: outputs are packed bf16 [rows][{cache.num_heads}][{cache.head_dim}], got "
                         f"{k_out.dtype} {tuple(shape)} and {v_out.dtype} {tuple(v_out.shape)}")
    _table_ok("moe_kv_read", block_table, B)
    _vector("moe_kv_read: start", start, torch.int32, B)
    _vector("moe_kv_read: cu_len", cu_len, torch.int32, B + 1)
    _check(lib().moe_kv_read(ctypes.byref(cache), B, shape[0], block_table.data_ptr(), block_table.size(1),
                             start.data_ptr(), cu_len.data_ptr(), k_out.data_ptr(), v_out.data_ptr(), _ptr(err_flag),
                             max_ctas, _stream(stream)), "moe_kv_read")


def _table_ok(where, t, B):
    if t.dtype is not torch.int32 or t.dim() != 2 or t.size(0) != B or not t.is_contiguous():
        raise ValueError(f"{where}: the block table is packed int32 [{B}][pages], got {t.dtype} {tuple(t.shape)}")


def _strides(t):
    """Row and head strides of t [rows][heads][width].  That of an index with one value is not used, and may be any
    number: the packed one is passed on."""
    rows, heads, width = t.shape
    head = t.stride(1) if heads > 1 else width
    return t.stride(0) if rows > 1 else heads * head, head


def moe_attn_workspace_size(cache: MoeKvCache, num_q_heads: int) -> int:
    return int(lib().moe_attn_workspace_size(ctypes.byref(cache), num_q_heads))


def attn_args(q, o, cu_q, kv_len, block_table, max_q, max_kv, scale, causal=True, window=0, lse=None,
              workspace=None, err_flag=None) -> MoeAttnArgs:
    """MoeAttnArgs from tensors: q, o bf16 [T][heads][head_dim] (any token and head strides), lse
    fp32 [T][heads]; workspace: moe_attn_workspace_size bytes, zeroed once before its first use."""
    _same("attn_args: o", (o.shape, q.shape))
    return _attn_args("attn_args", q, o, cu_q, kv_len, block_table, max_q, max_kv, scale, causal, window, lse,
                      workspace, err_flag)


def _attn_args(where, q, o, cu_q, kv_len, block_table, max_q, max_kv, scale, causal, window, lse, workspace, err_flag):
    T, H, D = q.shape
    B = kv_len.shape[0]
    _same(f"{where}: q, o", (o.dtype, torch.bfloat16), (q.dtype, torch.bfloat16))
    if q.stride(2) != 1 or o.stride(2) != 1:
        raise ValueError(f"{where}: head_dim is contiguous in q and o")
    _vector(f"{where}: cu_q", cu_q, torch.int32, B + 1)
    _vector(f"{where}: kv_len", kv_len, torch.int32, B)
    _table_ok(where, block_table, B)
    if lse is not None:
        _same(f"{where}: lse", (lse.shape, (T, H)), (lse.dtype, torch.float32), (lse.is_contiguous(), True))
    size = workspace.numel() * workspace.element_size() if workspace is not None else 0
    args = MoeAttnArgs(_ptr(q), _ptr(o), _ptr(lse), *_strides(q), *_strides(o), _ptr(cu_q), _ptr(kv_len),
                       _ptr(block_table), block_table.shape[1], T, B, max_q, max_kv, H, float(scale), int(causal), window,
                       _ptr(err_flag), _ptr(workspace), size)
    args.head_dim = D  # the C structure has no field for it: the cache's is meant
    args.keep = (q, o, lse, cu_q, kv_len, block_table, err_flag, workspace)  # it holds their addresses
    return args


def moe_attn_paged(cache: MoeKvCache, args: MoeAttnArgs, max_ctas=0, stream=None):
    if getattr(args, "head_dim", cache.head_dim) != cache.head_dim:  # a structure filled by hand has none
        raise ValueError(f"moe_attn_paged: q and o have heads of {args.head_dim}, the cache of {cache.head_dim}")
    _check(lib().moe_attn_paged(ctypes.byref(cache), ctypes.byref(args), max_ctas, _stream(stream)),
           "moe_attn_paged")


def _branches(where, tree, args):
    if tree.dtype not in (torch.int64, torch.uint64) or tree.shape != (args.T,) or not tree.is_contiguous():
        raise ValueError(f"{where}: tree is a packed vector of {args.T} 64-bit integers, got {tree.dtype} "
                         f"{tuple(tree.shape)}")
    return tree.data_ptr()


def moe_attn_tree(cache: MoeKvCache, args: MoeAttnArgs, tree, max_ctas=0, stream=None):
    """moe_attn_paged for trees of drafted tokens: tree int64 (or uint64) [T], bit j of a row's for its
    request's j-th new token (at most 64), itself included or not; args with causal, without a window."""
    if getattr(args, "head_dim", cache.head_dim) != cache.head_dim:
        raise ValueError(f"moe_attn_tree: q and o have heads of {args.head_dim}, the cache of {cache.head_dim}")
    _check(lib().moe_attn_tree(ctypes.byref(cache), ctypes.byref(args), _branches("moe_attn_tree", tree, args), max_ctas,
                               _stream(stream)), "moe_attn_tree")


# ---------------------------------------------------------------- latent attention
LATENT, ROPE, HEAD = 512, 64, 128  # numbers of a latent vector, of a rotary key, of an expanded key or value


def latent_cache(pool) -> MoeLatentCache:
    """The cache in a bf16 pool [pages][page_size][576] (any strides, the 576 numbers contiguous: 512 of the
    latent vector, 64 of the rotary key).  The pool must outlive the cache."""
    if pool.dtype != torch.bfloat16 or pool.dim() != 3 or pool.shape[2] != LATENT + ROPE or pool.stride(2) != 1:
        raise ValueError(f"latent_cache: a bf16 pool [pages][page_size][{LATENT + ROPE}] with contiguous rows is "
                         f"expected, got {pool.dtype} {tuple(pool.shape)}")
    return MoeLatentCache(_ptr(pool), BF16, pool.shape[0], pool.shape[1], LATENT, ROPE, pool.stride(0), pool.stride(1))


def moe_latent_write(cache: MoeLatentCache, c, k_rope, slots, weight=None, eps=1e-6, err_flag=None, max_ctas=0,
                     stream=None):
    """Stores c [T][512] (normed with weight [512] where given) and k_rope [T][64] (bf16, any row strides) at
    slots int64 [T]."""
    T = c.size(0)
    bf16 = torch.bfloat16
    if c.shape != (T, cache.latent) or k_rope.shape != (T, cache.rope) or not (c.dtype is k_rope.dtype is bf16):
        raise ValueError(f"moe_latent_write: c and k_rope are bf16 [{T}][{cache.latent}] and [{T}][{cache.rope}], got "
                         f"{c.dtype} {tuple(c.shape)} and {k_rope.dtype} {tuple(k_rope.shape)}")
    c0, c1 = c.stride()
    r0, r1 = k_rope.stride()
    if c1 != 1 or r1 != 1:
        raise ValueError("moe_latent_write: the rows of c and k_rope are contiguous")
    if weight is not None:
        _vector("moe_latent_write: weight", weight, bf16, cache.latent)
    _vector("moe_latent_write: slots", slots, torch.int64, T)
    # the stride of a single row is not used, and may be any number
    _check(lib().moe_latent_write(ctypes.byref(cache), T, c.data_ptr(), c0 if T > 1 else cache.latent,
                                  k_rope.data_ptr(), r0 if T > 1 else cache.rope, _ptr(weight), eps, slots.data_ptr(),
                                  _ptr(err_flag), max_ctas, _stream(stream)), "moe_latent_write")


def moe_attn_latent_workspace_size(cache: MoeLatentCache, num_q_heads: int) -> int:
    return int(lib().moe_attn_latent_workspace_size(ctypes.byref(cache), num_q_heads))


def attn_latent_args(q, o, cu_q, kv_len, block_table, max_q, max_kv, scale, causal=True, window=0, lse=None,
                     workspace=None, err_flag=None) -> MoeAttnArgs:
    """attn_args of moe_attn_latent: q bf16 [T][heads][576], o bf16 [T][heads][512]; workspace:
    moe_attn_latent_workspace_size bytes, zeroed once before its first use."""
    _same("attn_latent_args: q, o", (q.dim(), 3), (q.shape[2:], (LATENT + ROPE,)), (o.shape, (*q.shape[:2], LATENT)))
    return _attn_args("attn_latent_args", q, o, cu_q, kv_len, block_table, max_q, max_kv, scale, causal, window, lse,
                      workspace, err_flag)


def moe_attn_latent(cache: MoeLatentCache, args: MoeAttnArgs, tree=None, max_ctas=0, stream=None):
    """Absorbed latent attention; tree as for moe_attn_tree."""
    width = cache.latent + cache.rope
    if getattr(args, "head_dim", width) != width:  # a structure filled by hand has none
        raise ValueError(f"moe_attn_latent: q has rows of {args.head_dim}, the cache of {width} (attn_latent_args)")
    _check(lib().moe_attn_latent(ctypes.byref(cache), ctypes.byref(args),
                                 None if tree is None else _branches("moe_attn_latent", tree, args), max_ctas,
                                 _stream(stream)), "moe_attn_latent")


def moe_attn_expanded_workspace_size(num_heads: int) -> int:
    return int(lib().moe_attn_expanded_workspace_size(num_heads))


def attn_expanded_args(q, k, k_rope, v, o, cu_q, cu_kv, max_q, max_kv, scale, causal=True, lse=None, workspace=None,
                       err_flag=None) -> MoeAttnExpandedArgs:
    """MoeAttnExpandedArgs from bf16 tensors q [T][heads][192], k and v [S][heads][128], k_rope [S][64],
    o [T][heads][128] (any row and head strides); lse fp32 [T][heads]; workspace:
    moe_attn_expanded_workspace_size bytes, zeroed once before its first use."""
    T, H, _ = q.shape
    S, B = k_rope.shape[0], cu_q.shape[0] - 1
    _same("attn_expanded_args: shapes", (q.shape, (T, H, HEAD + ROPE)), (k.shape, (S, H, HEAD)),
          (k_rope.shape, (S, ROPE)), (v.shape, (S, H, HEAD)), (o.shape, (T, H, HEAD)))
    for t in (q, k, k_rope, v, o):
        _same("attn_expanded_args: types", (t.dtype, torch.bfloat16))
        if t.stride(-1) != 1:
            raise ValueError("attn_expanded_args: rows are contiguous")
    _vector("attn_expanded_args: cu_q", cu_q, torch.int32, B + 1)
    _vector("attn_expanded_args: cu_kv", cu_kv, torch.int32, B + 1)
    if lse is not None:
        _same("attn_expanded_args: lse", (lse.shape, (T, H)), (lse.dtype, torch.float32), (lse.is_contiguous(), True))
    size = workspace.numel() * workspace.element_size() if workspace is not None else 0
    args = MoeAttnExpandedArgs(_ptr(q), _ptr(k), _ptr(k_rope), _ptr(v), _ptr(o), _ptr(lse), *_strides(q), *_strides(k),
                               k_rope.stride(0) if S > 1 else ROPE, *_strides(v), *_strides(o), _ptr(cu_q), _ptr(cu_kv),
                               T, S, B, max_q, max_kv, H, float(scale), int(causal), _ptr(err_flag), _ptr(workspace),
                               size)
    args.keep = (q, k, k_rope, v, o, lse, cu_q, cu_kv, err_flag, workspace)  # it holds their addresses
    return args


def moe_attn_expanded(args: MoeAttnExpandedArgs, max_ctas=0, stream=None):
    _check(lib().moe_attn_expanded(ctypes.byref(args), max_ctas, _stream(stream)), "moe_attn_expanded")


# ---------------------------------------------------------------- between two blocks
_FLOATS = {torch.float32: F32, torch.bfloat16: BF16}


def moe_block_norm(y, out=None, pre_weight=None, resid=None, resid_out=None, post_weight=None, gate=None, scale=1.0,
                   eps=1e-6, max_ctas=0, stream=None):
    """x = norm(y) with post_weight [H], or y; resid_out = resid + scale * gate * x; out = norm(resid_out) with
    pre_weight [H].  y, out, weights and gate ([T][H], or [1][H] for all tokens) fp32 or bf16, the residual
    either; packed rows.  resid_out may be resid, and out may be y."""
    shape, dtype = y.shape, y.dtype
    T, H = shape
    rdtype = dtype if resid is None and resid_out is None else (resid if resid is not None else resid_out).dtype
    kind, rkind = _FLOATS.get(dtype), _FLOATS.get(rdtype)
    if kind is None or rkind is None or not y.is_contiguous():
        raise ValueError(f"moe_block_norm: packed rows of fp32 or bf16 are expected, got {dtype} and {rdtype}")
    y_at, out_at, resid_at = y.data_ptr(), _rows_at(out, shape, dtype), _rows_at(resid, shape, rdtype)
    resid_out_at = resid_at if resid_out is resid else _rows_at(resid_out, shape, rdtype)
    post_at = pre_at = gate_at = None
    if post_weight is not None:
        _vector("moe_block_norm: post_weight", post_weight, dtype, H)
        post_at = post_weight.data_ptr()
    if pre_weight is not None:
        _vector("moe_block_norm: pre_weight", pre_weight, dtype, H)
        pre_at = pre_weight.data_ptr()
    rows = 1
    if gate is not None:
        rows = gate.size(0)
        if gate.dtype is not dtype or gate.shape != (rows, H) or rows not in (1, T) or not gate.is_contiguous():
            raise ValueError(f"moe_block_norm: gate is packed {dtype} [1 or {T}][{H}], got {gate.dtype} {tuple(gate.shape)}")
        gate_at = gate.data_ptr()
    args = MoeNormArgs(y_at, post_at, gate_at, resid_at, resid_out_at, pre_at, out_at, T, H, kind, rkind, rows, scale, eps)
    _check(lib().moe_block_norm(ctypes.byref(args), max_ctas, _stream(stream)), "moe_block_norm")


def _rows_at(t, shape, dtype):
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"moe_block_norm: packed {dtype} rows {tuple(shape)} are expected, got {t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


def moe_draft_verify(target, draft, cu_draft, ids, u, u_draw, out_ids, out_len, err_flag=None, max_ctas=0,
                     stream=None):
    """Drafted tokens ids against target [N + B][vocab] and draft [N][vocab] (or None) probabilities
    (fp32 or bf16, rows at any stride) from uniform numbers u [N], u_draw [B]; see moe.h."""
    i32, f32 = torch.int32, torch.float32
    B, (rows, V), dtype = out_len.size(0), target.shape, target.dtype
    N = ids.size(0) if ids is not None else 0
    target_ld, one = target.stride()
    if one != 1 or rows != N + B or (dtype is not f32 and dtype is not torch.bfloat16):
        raise ValueError(f"moe_draft_verify: target is fp32 or bf16 [{N + B}][vocab], got {dtype} {tuple(target.shape)}")
    q, draft_ld = None, 0
    if draft is not None:
        draft_ld, one = draft.stride()
        if one != 1 or draft.dtype is not dtype or draft.shape != (N, V):
            raise ValueError(f"moe_draft_verify: draft is {dtype} [{N}][{V}], got {draft.dtype} {tuple(draft.shape)}")
        if N:
            q = draft.data_ptr()
    _vector("moe_draft_verify: cu_draft", cu_draft, i32, B + 1)
    _vector("moe_draft_verify: u_draw", u_draw, f32, B)
    _vector("moe_draft_verify: out_len", out_len, i32, B)
    if N:
        _vector("moe_draft_verify: ids", ids, i32, N)
        _vector("moe_draft_verify: u", u, f32, N)
    if out_ids.dtype is not i32 or out_ids.dim() != 2 or out_ids.size(0) != B or not out_ids.is_contiguous():
        raise ValueError(f"moe_draft_verify: out_ids is packed int32 [{B}][max_draft + 1]")
    # the stride of a single row is not used, and may be any number
    _check(lib().moe_draft_verify_ex(B, N, V, out_ids.size(1) - 1, F32 if dtype is f32 else BF16, target.data_ptr(),
                                     target_ld if rows > 1 else V, q, draft_ld if N > 1 else V, cu_draft.data_ptr(),
                                     ids.data_ptr() if N else None, u.data_ptr() if N else None, u_draw.data_ptr(),
                                     out_ids.data_ptr(), out_len.data_ptr(), _ptr(err_flag), max_ctas,
                                     _stream(stream)), "moe_draft_verify")
