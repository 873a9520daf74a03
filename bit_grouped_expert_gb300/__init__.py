"""Python binding of libmoe.so (the sm_103a MoE expert layer).

Argument marshalling only: every function forwards to the C entry point of
the same name in ``include/moe.h``; all of the layer's work runs in the
library's CUDA kernels.  Tensors are passed by device pointer
(``tensor.data_ptr()``) and must already live on the GPU; the stream defaults
to PyTorch's current stream.  There is no fallback: if ``libmoe.so`` has not
been built (``python -m bit_grouped_expert_gb300.build``) the import of the
library raises.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

MOE_OK = 0
MOE_ERR_INVALID_ARGUMENT = 1
MOE_ERR_UNSUPPORTED = 2
MOE_ERR_MISALIGNED = 3
MOE_ERR_WORKSPACE_TOO_SMALL = 4
MOE_ERR_TOO_MANY_TOKENS = 5
MOE_ERR_CUDA = 6
MOE_ERR_DEVICE_TIMEOUT = 7
MOE_ERR_NONFINITE = 8
MOE_ERR_DEVICE_BOUNDS = 9
MOE_ERR_OUT_OF_PAGES = 10

MOE_BF16 = 0
MOE_FP16 = 1

MOE_FLAG_DEBUG_CHECKS = 0x1
MOE_FLAG_FORCE_GROUPED = 0x2
MOE_FLAG_SIMT_EXPERTS = 0x4
MOE_FLAG_TILE_ROWS_64 = 0x8
MOE_FLAG_PRENORM = 0x10
MOE_FLAG_TRACE = 0x20
MOE_FLAG_TEST_WITHHOLD = 0x40
MOE_TRACE_CTAS = 256
MOE_TRACE_SLOTS = 32

EXPORTS = ("moe_plan", "moe_plan_destroy", "moe_workspace_bytes", "moe_workspace_init", "moe_route",
           "moe_route_from_logits", "moe_route_from_ids", "moe_forward", "moe_prefill_stack", "moe_router_split_bytes",
           "moe_router_split", "moe_route_view", "moe_rmsnorm", "moe_dequant",
           "moe_device_status", "moe_last_launch_count", "moe_status_str", "moe_profile_events", "moe_profile_stride",
           "moe_last_cuda_error",
           "moe_decode_static", "moe_decode_stack", "gdn_scan", "attn_decode_workspace_bytes", "attn_decode",
           "attn_cache_append_workspace_bytes", "attn_cache_append", "attn_cache_fork_workspace_bytes",
           "attn_cache_fork", "attn_cache_trim", "attn_tree_workspace_bytes", "attn_tree", "moe_draft_verify",
           "attn_rotary_plan", "attn_rotary", "attn_cache_append_rotary", "attn_qcache_append_workspace_bytes",
           "attn_qcache_append", "attn_qcache_fork_workspace_bytes", "attn_qcache_fork", "attn_qcache_trim",
           "attn_qcache_attend_workspace_bytes", "attn_qcache_attend")

MOE_DECODE_STATIC_SCRATCH_BYTES = 65536

MOE_KERNEL_ROUTER = 1
MOE_KERNEL_TOPK = 2
MOE_KERNEL_SCATTER = 3
MOE_KERNEL_GATEUP = 4
MOE_KERNEL_DOWN = 5
MOE_KERNEL_COMBINE = 6
MOE_KERNEL_DECODE_LAYER = 7
MOE_KERNEL_RMSNORM = 10
MOE_KERNEL_GATHER = 11
MOE_KERNEL_GDN_SCAN = 12
MOE_KERNEL_ATTN_DECODE = 13
MOE_KERNEL_ATTN_TREE = 14
MOE_KERNEL_DRAFT_VERIFY = 15
MOE_KERNEL_CACHE_COPY = 16
MOE_KERNEL_ATTN_QCACHE = 17


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        msg = f"{fn}: {status_str(status)} ({status})"
        if status == MOE_ERR_CUDA:
            msg += ": " + lib().moe_last_cuda_error().decode()
        super().__init__(msg)


class moe_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("hidden", "n_experts", "top_k", "inter", "n_shared", "group_size")]


class moe_weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("router_d", "gate_q_d", "up_q_d", "gate_s_d", "gate_b_d", "up_s_d",
                                               "up_b_d", "down_q_d", "down_s_d", "down_b_d", "shared_gate_d",
                                               "router_split_d")]


class moe_route_ptrs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("keys_d", "topk_id_d", "topk_w_d", "counts_d", "offsets_d", "perm_d",
                                               "inv_d", "blockmap_d", "n_tiles_d", "h_d", "y_d", "status_d",
                                               "trace_d")] + \
               [("max_tiles", ctypes.c_int32), ("block_rows", ctypes.c_int32), ("blockmap2_d", ctypes.c_void_p),
                ("n_tiles2_d", ctypes.c_void_p), ("max_tiles2", ctypes.c_int32), ("block_rows2", ctypes.c_int32)]


class attn_cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_d", "v_d", "refs_d", "table_d", "lens_d", "status_d")] + \
               [(n, ctypes.c_int32) for n in ("n_layers", "n_pages", "page_size", "n_kv_heads", "head_dim", "n_slots",
                                              "max_pages", "dtype")]


class attn_qcache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_d", "v_d", "k_scale_d", "v_scale_d", "refs_d", "table_d", "lens_d",
                                               "status_d")] + \
               [(n, ctypes.c_int32) for n in ("n_layers", "n_pages", "page_size", "n_kv_heads", "head_dim", "n_slots",
                                              "max_pages", "reserved")]


class attn_rotary_config(ctypes.Structure):
    _fields_ = [("dim", ctypes.c_int32), ("interleaved", ctypes.c_int32)] + \
               [(n, ctypes.c_double) for n in ("base", "stretch", "low_turns", "high_turns", "original_len")] + \
               [("factor", ctypes.c_float)]


class attn_rotary_table(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_uint64 * 128), ("dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("factor", ctypes.c_float), ("reserved", ctypes.c_int32)]


_lib = None


def lib():
    """Load libmoe.so (raises OSError if it is missing: no fallback path)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise OSError(f"libmoe.so not built at {LIB_PATH}; run bit_grouped_expert_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, u32, sz, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint32, ctypes.c_size_t, ctypes.c_float
        L.moe_plan.restype = i32
        L.moe_plan.argtypes = [ctypes.POINTER(moe_config), i32, u32, ctypes.POINTER(vp)]
        L.moe_plan_destroy.restype = None
        L.moe_plan_destroy.argtypes = [vp]
        L.moe_workspace_bytes.restype = sz
        L.moe_workspace_bytes.argtypes = [vp]
        L.moe_workspace_init.restype = i32
        L.moe_workspace_init.argtypes = [vp, vp, sz, vp]
        L.moe_route.restype = i32
        L.moe_route.argtypes = [vp, vp, i32, vp, vp, vp, sz, vp]
        L.moe_route_from_logits.restype = i32
        L.moe_route_from_logits.argtypes = [vp, vp, i32, vp, sz, vp]
        L.moe_route_from_ids.restype = i32
        L.moe_route_from_ids.argtypes = [vp, vp, vp, i32, vp, sz, vp]
        L.moe_forward.restype = i32
        L.moe_forward.argtypes = [vp, vp, vp, i32, ctypes.POINTER(moe_weights), vp, vp, vp, sz, vp]
        L.moe_prefill_stack.restype = i32
        L.moe_prefill_stack.argtypes = [vp, vp, i32, i32, ctypes.POINTER(moe_weights), ctypes.POINTER(vp), vp, sz,
                                        vp]
        L.moe_router_split_bytes.restype = sz
        L.moe_router_split_bytes.argtypes = [i32, i32]
        L.moe_router_split.restype = i32
        L.moe_router_split.argtypes = [vp, i32, i32, vp, sz, vp]
        L.moe_route_view.restype = i32
        L.moe_route_view.argtypes = [vp, vp, i32, ctypes.POINTER(moe_route_ptrs)]
        L.moe_rmsnorm.restype = i32
        L.moe_rmsnorm.argtypes = [vp, i32, i32, f32, vp, vp]
        L.moe_dequant.restype = i32
        L.moe_dequant.argtypes = [vp, vp, vp, i32, i32, i32, vp, vp]
        L.moe_device_status.restype = i32
        L.moe_device_status.argtypes = [vp, vp, vp, ctypes.POINTER(i32), i32]
        L.moe_last_launch_count.restype = i32
        L.moe_last_launch_count.argtypes = []
        L.moe_profile_events.restype = i32
        L.moe_profile_events.argtypes = [i32, ctypes.POINTER(vp), ctypes.POINTER(vp), i32]
        L.moe_profile_stride.restype = i32
        L.moe_profile_stride.argtypes = [i32, i32]
        L.moe_last_cuda_error.restype = ctypes.c_char_p
        L.moe_last_cuda_error.argtypes = []
        L.moe_status_str.restype = ctypes.c_char_p
        L.moe_status_str.argtypes = [i32]
        L.moe_decode_stack.restype = i32
        L.moe_decode_stack.argtypes = [vp, vp, i32, ctypes.POINTER(moe_weights), ctypes.POINTER(vp), vp, sz, vp]
        L.moe_decode_static.restype = i32
        L.moe_decode_static.argtypes = [ctypes.POINTER(moe_config), vp, vp, ctypes.POINTER(moe_weights), vp, vp, vp,
                                        u32, vp]
        L.gdn_scan.restype = i32
        L.gdn_scan.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp]
        L.attn_decode_workspace_bytes.restype = sz
        L.attn_decode_workspace_bytes.argtypes = [i32, i32, i32]
        L.attn_decode.restype = i32
        L.attn_decode.argtypes = [vp, vp, vp, i32, i32, i32, i32, f32, vp, sz, vp, vp]
        cache = ctypes.POINTER(attn_cache)
        L.attn_cache_append_workspace_bytes.restype = sz
        L.attn_cache_append_workspace_bytes.argtypes = [cache, i32, i32]
        L.attn_cache_append.restype = i32
        L.attn_cache_append.argtypes = [cache, vp, vp, vp, vp, vp, vp, i32, i32, i32, vp, sz, vp]
        L.attn_cache_fork_workspace_bytes.restype = sz
        L.attn_cache_fork_workspace_bytes.argtypes = [cache, i32]
        L.attn_cache_fork.restype = i32
        L.attn_cache_fork.argtypes = [cache, vp, vp, i32, vp, sz, vp]
        L.attn_cache_trim.restype = i32
        L.attn_cache_trim.argtypes = [cache, vp, vp, i32, vp]
        L.attn_tree_workspace_bytes.restype = sz
        L.attn_tree_workspace_bytes.argtypes = [cache, i32, i32, i32, i32]
        L.attn_tree.restype = i32
        L.attn_tree.argtypes = [cache, i32, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, f32, vp, sz, vp, vp]
        L.moe_draft_verify.restype = i32
        L.moe_draft_verify.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, vp, i32, vp, vp, vp, vp]
        table, qcache, i64 = ctypes.POINTER(attn_rotary_table), ctypes.POINTER(attn_qcache), ctypes.c_int64
        L.attn_rotary_plan.restype = i32
        L.attn_rotary_plan.argtypes = [ctypes.POINTER(attn_rotary_config), table]
        L.attn_rotary.restype = i32
        L.attn_rotary.argtypes = [table, vp, i64, i32, vp, i32, i32, i32, vp, i64, vp]
        L.attn_cache_append_rotary.restype = i32
        L.attn_cache_append_rotary.argtypes = [cache, table, vp, vp, vp, vp, vp, vp, i32, i32, i32, vp, sz, vp]
        L.attn_qcache_append_workspace_bytes.restype = sz
        L.attn_qcache_append_workspace_bytes.argtypes = [qcache, i32, i32]
        L.attn_qcache_append.restype = i32
        L.attn_qcache_append.argtypes = [qcache, table, vp, vp, i32, vp, vp, vp, vp, i32, i32, i32, vp, sz, vp]
        L.attn_qcache_fork_workspace_bytes.restype = sz
        L.attn_qcache_fork_workspace_bytes.argtypes = [qcache, i32]
        L.attn_qcache_fork.restype = i32
        L.attn_qcache_fork.argtypes = [qcache, vp, vp, i32, vp, sz, vp]
        L.attn_qcache_trim.restype = i32
        L.attn_qcache_trim.argtypes = [qcache, vp, vp, i32, vp]
        L.attn_qcache_attend_workspace_bytes.restype = sz
        L.attn_qcache_attend_workspace_bytes.argtypes = [qcache, i32, i32, i32, i32]
        L.attn_qcache_attend.restype = i32
        L.attn_qcache_attend.argtypes = [qcache, i32, vp, i32, vp, vp, i32, i32, i32, i32, f32, vp, sz, vp, vp]
        _lib = L
    return _lib


def status_str(status: int) -> str:
    return lib().moe_status_str(int(status)).decode()


def _ptr(t):
    """Device pointer of a tensor (or an int address, or None)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _nbytes(t):
    return t.numel() * t.element_size()


def _check(fn, status):
    if status != MOE_OK:
        raise MoeError(fn, status)


class Plan:
    """Owns a moe_plan_t (host memory only)."""

    def __init__(self, handle: int, cfg: moe_config, max_tokens: int, flags: int):
        self.handle = handle
        self.cfg = cfg
        self.max_tokens = max_tokens
        self.flags = flags

    def __del__(self):
        if getattr(self, "handle", None) and _lib is not None:
            _lib.moe_plan_destroy(self.handle)
            self.handle = None


def make_config(hidden=2048, n_experts=256, top_k=8, inter=512, n_shared=1, group_size=64) -> moe_config:
    return moe_config(hidden, n_experts, top_k, inter, n_shared, group_size)


def moe_plan(cfg: moe_config, max_tokens: int, flags: int = 0) -> Plan:
    h = ctypes.c_void_p()
    _check("moe_plan", lib().moe_plan(ctypes.byref(cfg), int(max_tokens), int(flags), ctypes.byref(h)))
    return Plan(h.value, cfg, max_tokens, flags)


def moe_workspace_bytes(plan: Plan) -> int:
    return int(lib().moe_workspace_bytes(plan.handle))


def moe_workspace_init(plan: Plan, ws, stream=None):
    _check("moe_workspace_init", lib().moe_workspace_init(plan.handle, _ptr(ws), _nbytes(ws), _stream(stream)))


def make_weights(w: dict) -> moe_weights:
    """moe_weights from a dict of device tensors (keys: router, gate_q, ...;
    shared_gate and router_split optional).  The caller keeps the tensors
    alive."""
    return moe_weights(*[_ptr(w.get(n[:-2])) for n, _ in moe_weights._fields_])


def moe_route(plan: Plan, x, T: int, router, logit_bias, ws, stream=None):
    _check("moe_route", lib().moe_route(plan.handle, _ptr(x), int(T), _ptr(router), _ptr(logit_bias), _ptr(ws),
                                        _nbytes(ws), _stream(stream)))


def moe_route_from_logits(plan: Plan, keys, T: int, ws, stream=None):
    _check("moe_route_from_logits", lib().moe_route_from_logits(plan.handle, _ptr(keys), int(T), _ptr(ws),
                                                                _nbytes(ws), _stream(stream)))


def moe_route_from_ids(plan: Plan, ids, w, T: int, ws, stream=None):
    _check("moe_route_from_ids", lib().moe_route_from_ids(plan.handle, _ptr(ids), _ptr(w), int(T), _ptr(ws),
                                                          _nbytes(ws), _stream(stream)))


def moe_router_split_bytes(E: int, H: int) -> int:
    return int(lib().moe_router_split_bytes(int(E), int(H)))


def moe_router_split(router, E: int, H: int, split, stream=None):
    """The router's three bf16 parts into ``split`` (a device tensor of
    moe_router_split_bytes(E, H) bytes), for the ``router_split`` weight."""
    _check("moe_router_split", lib().moe_router_split(_ptr(router), int(E), int(H), _ptr(split), _nbytes(split),
                                                      _stream(stream)))


def _weights_array(weights):
    n = len(weights)
    return (moe_weights * max(n, 1))(*[w if isinstance(w, moe_weights) else make_weights(w) for w in weights])


def _bias_array(logit_bias, n):
    if logit_bias is None:
        return None
    if len(logit_bias) != n:
        raise ValueError("one logit bias (or None) per layer")
    return (ctypes.c_void_p * max(n, 1))(*[_ptr(b) for b in logit_bias])


def moe_prefill_stack(plan: Plan, r, T: int, weights, logit_bias=None, ws=None, stream=None):
    """T tokens of the residual stream ``r`` through len(weights) pre-norm
    layers in chunks of the plan's max_tokens (chunk-major), in place."""
    n = len(weights)
    _check("moe_prefill_stack", lib().moe_prefill_stack(plan.handle, _ptr(r), int(T), n, _weights_array(weights),
                                                        _bias_array(logit_bias, n), _ptr(ws), _nbytes(ws),
                                                        _stream(stream)))


def moe_forward(plan: Plan, x, residual, T: int, weights, logit_bias, out, ws, stream=None):
    cw = weights if isinstance(weights, moe_weights) else make_weights(weights)
    _check("moe_forward", lib().moe_forward(plan.handle, _ptr(x), _ptr(residual), int(T), ctypes.byref(cw),
                                            _ptr(logit_bias), _ptr(out), _ptr(ws), _nbytes(ws), _stream(stream)))


def moe_decode_stack(plan: Plan, r, weights, logit_bias=None, ws=None, stream=None):
    """Single-token decode through len(weights) pre-norm layers, r updated in
    place.  ``weights``: list of weight dicts (or moe_weights); ``logit_bias``:
    None or a list of per-layer bias tensors (entries may be None)."""
    n = len(weights)
    _check("moe_decode_stack", lib().moe_decode_stack(plan.handle, _ptr(r), n, _weights_array(weights),
                                                      _bias_array(logit_bias, n), _ptr(ws), _nbytes(ws),
                                                      _stream(stream)))


def moe_decode_static(cfg: moe_config, x, residual, weights, logit_bias, out, status=None, flags: int = 0,
                      stream=None):
    """One token through the layer with no device allocation (library-owned
    static scratch; see the header).  ``status``: optional device int32."""
    cw = weights if isinstance(weights, moe_weights) else make_weights(weights)
    _check("moe_decode_static", lib().moe_decode_static(ctypes.byref(cfg), _ptr(x), _ptr(residual), ctypes.byref(cw),
                                                        _ptr(logit_bias), _ptr(out), _ptr(status), int(flags),
                                                        _stream(stream)))


def gdn_scan(q, k, v, alpha, beta, state, o, T: int, Hk: int, Hv: int, dk: int = 128, dv: int = 128, stream=None):
    """Gated DeltaNet scan of one sequence (gdn.h): q, k [T, Hk, dk] and v
    [T, Hv, dv] bf16, alpha, beta [T, Hv] fp32, state [Hv, dk, dv] fp32
    (updated in place), o [T, Hv, dv] bf16 (written)."""
    _check("gdn_scan", lib().gdn_scan(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(state), _ptr(o),
                                      int(T), int(Hk), int(Hv), int(dk), int(dv), _stream(stream)))


def attn_decode_workspace_bytes(L: int, Hq: int = 16, D: int = 256) -> int:
    return int(lib().attn_decode_workspace_bytes(int(L), int(Hq), int(D)))


def attn_decode(q, k, v, L: int, Hq: int, Hkv: int, D: int, ws, o, scale: float = 0.0, stream=None):
    """One query token against a KV cache (attn.h): q [Hq, D], k, v [L, Hkv, D]
    bf16, ws a uint8 device tensor of attn_decode_workspace_bytes(L, Hq, D)
    bytes or more, o [Hq, D] bf16 (written)."""
    _check("attn_decode", lib().attn_decode(_ptr(q), _ptr(k), _ptr(v), int(L), int(Hq), int(Hkv), int(D),
                                            float(scale), _ptr(ws), _nbytes(ws) if not isinstance(ws, int) else 0,
                                            _ptr(o), _stream(stream)))


def _given(name, t, dtype, device, shape):
    """Address of a tensor argument of the paged-cache and drafting operators,
    whose sizes come from their tensors: dense, of the type and shape asked
    for, on the call's device."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != device:
        raise ValueError(f"{name}: a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{device} wanted, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}{'' if t.is_contiguous() else ' (not contiguous)'}")
    return t.data_ptr()


def _here(name, device):
    """Refuse a call whose tensors are not on the current device (kernels launch there)."""
    import torch
    current = torch._C._cuda_getDevice() if device >= 0 else None  # CUDA is up: a tensor lives there
    if device != current:
        raise ValueError(f"{name}: on {'the host' if device < 0 else f'cuda:{device}'}, not on the current device")


def _scratch(ws, device):
    """Address and bytes of a workspace tensor on the call's device."""
    if ws.get_device() != device or not ws.is_contiguous():
        raise ValueError(f"ws: a contiguous tensor on cuda:{device} wanted, got one on {ws.device}")
    return ws.data_ptr(), ws.nbytes


def _raw_stream(stream, device):
    """As _stream, without making a Stream object for the current one."""
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(device)
    return _stream(stream)


class Rotary:
    """The rates of rotary positions (rotary.h): an attn_rotary_table on the host."""

    def __init__(self, struct: attn_rotary_table):
        self.struct = struct
        self.ref = ctypes.byref(struct)


def make_rotary(dim: int, base: float = 10000.0, interleaved: bool = False, stretch: float = 1.0,
                low_turns: float = 0.0, high_turns: float = 0.0, original_len: float = 0.0,
                factor: float = 1.0) -> Rotary:
    """The rates of the first ``dim`` values of a head: base^(-2i/dim), slowed
    by ``stretch`` for pairs that turn less than ``high_turns`` times over
    ``original_len`` positions (fully below ``low_turns``; with both 0 all of them)."""
    cfg = attn_rotary_config(int(dim), int(interleaved), base, stretch, low_turns, high_turns, original_len, factor)
    table = attn_rotary_table()
    _check("attn_rotary_plan", lib().attn_rotary_plan(ctypes.byref(cfg), ctypes.byref(table)))
    return Rotary(table)


def _kind(name, dtype):
    """MOE_BF16 or MOE_FP16 of a torch type."""
    import torch
    if dtype is torch.bfloat16:
        return MOE_BF16
    if dtype is torch.float16:
        return MOE_FP16
    raise ValueError(f"{name}: bf16 or fp16 wanted, got {dtype}")


def _rows_given(name, t, dtype, device, shape):
    """Address and row stride of rows [n, H, D] whose heads lie one after another."""
    n, H, D = shape
    strides = t.stride()
    if (t.dtype is dtype and t.shape == shape and t.get_device() == device and
            (strides[2] == 1 and (H == 1 or strides[1] == D) or not t.numel())):
        return t.data_ptr(), strides[0] if n > 1 else H * D
    raise ValueError(f"{name}: a {dtype} tensor of shape {tuple(shape)} on cuda:{device} wanted, each row's heads one "
                     f"after another, got {t.dtype} {tuple(t.shape)} with strides {strides} on {t.device}")


def attn_rotary(rotary: Rotary, x, positions, o, stream=None):
    """Rows turned by their positions (rotary.h): x, o [n, H, D] bf16 or fp16
    (rows may lie apart; o may be x), positions int32 [n]."""
    import torch
    dev, shape, dtype = x.get_device(), x.shape, x.dtype
    _here("x", dev)
    if len(shape) != 3:
        raise ValueError(f"x: [n, H, D] wanted, got {tuple(shape)}")
    n, H, D = shape
    kind = MOE_BF16 if dtype is torch.bfloat16 else _kind("x", dtype)
    x_at, x_stride = _rows_given("x", x, dtype, dev, shape)
    o_at, o_stride = (x_at, x_stride) if o is x else _rows_given("o", o, dtype, dev, shape)
    _check("attn_rotary", lib().attn_rotary(
        rotary.ref, x_at, x_stride, kind, _given("positions", positions, torch.int32, dev, (n,)), n, H, D, o_at, o_stride,
        _raw_stream(stream, dev)))


class AttnCache:
    """A paged KV cache (cache.h): the attn_cache struct and the tensors behind it."""

    def __init__(self, struct: attn_cache, tensors: dict):
        import torch
        self.struct = struct
        self.ref = ctypes.byref(struct)
        self.tensors = tensors
        self.dtype = tensors["k"].dtype
        self.i32 = torch.int32
        self.device = tensors["k"].get_device()
        self.layers, self.heads, self.dim = struct.n_layers, struct.n_kv_heads, struct.head_dim


def make_attn_cache(k, v, refs, table, lens, status) -> AttnCache:
    """The cache over the caller's tensors: k, v [n_layers, n_pages, page_size,
    Hkv, D] (bf16 or fp16), refs [n_pages], table [n_slots, max_pages], lens
    [n_slots], status [>= 1] int32, all contiguous on one device.  A new cache
    starts with refs, lens and status zero and table -1."""
    import torch
    kinds = {torch.bfloat16: MOE_BF16, torch.float16: MOE_FP16}
    if k.dtype not in kinds or k.dim() != 5 or table.dim() != 2 or lens.dim() != 1 or status.dim() != 1:
        raise ValueError(f"k: bf16 or fp16 [layers, pages, page_size, heads, dim], table of 2, lens and status of 1 "
                         f"dimensions wanted, got k {k.dtype} {tuple(k.shape)}")
    layers, pages, page, heads, dim = k.shape
    dev, ints = k.get_device(), torch.int32
    st = attn_cache(_given("k", k, k.dtype, dev, k.shape), _given("v", v, k.dtype, dev, k.shape),
                    _given("refs", refs, ints, dev, (pages,)),
                    _given("table", table, ints, dev, (lens.shape[0], table.shape[1])),
                    _given("lens", lens, ints, dev, lens.shape), _given("status", status, ints, dev, status.shape),
                    layers, pages, page, heads, dim, lens.shape[0], table.shape[1], kinds[k.dtype])
    return AttnCache(st, dict(k=k, v=v, refs=refs, table=table, lens=lens, status=status))


def attn_cache_append_workspace_bytes(cache: AttnCache, B: int, n_rows: int) -> int:
    return int(lib().attn_cache_append_workspace_bytes(cache.ref, int(B), int(n_rows)))


def _append_given(cache, dtype, k_new, v_new, offsets, B, ws, slots, path, n_keep):
    """The arguments that every append shares, in the entry points' order, up to the stream."""
    dev, i32, n_rows = cache.device, cache.i32, k_new.shape[1]
    _here("cache", dev)
    shape, stride = (cache.layers, n_rows, cache.heads, cache.dim), 0 if path is None else path.shape[-1]
    return ((_given("k_new", k_new, dtype, dev, shape), _given("v_new", v_new, dtype, dev, shape)),
            (None if slots is None else _given("slots", slots, i32, dev, (B,)),
             _given("offsets", offsets, i32, dev, (B + 1,)),
             None if n_keep is None else _given("n_keep", n_keep, i32, dev, (B,)),
             None if path is None else _given("path", path, i32, dev, (B, stride)), stride, B, n_rows,
             *_scratch(ws, dev)))


def attn_cache_append(cache: AttnCache, k_new, v_new, offsets, B: int, ws, slots=None, path=None, n_keep=None,
                      stream=None):
    """Append the kept rows of B sequences, in all layers: k_new, v_new
    [n_layers, n_rows, Hkv, D], offsets int32 [B + 1], slots int32 [B] or None
    (0 .. B-1), path int32 [B, stride] and n_keep int32 [B] as moe_draft_verify
    leaves them, or None (every row, in order)."""
    rows, rest = _append_given(cache, cache.dtype, k_new, v_new, offsets, int(B), ws, slots, path, n_keep)
    _check("attn_cache_append", lib().attn_cache_append(cache.ref, *rows, *rest, _raw_stream(stream, cache.device)))


def attn_cache_append_rotary(cache: AttnCache, rotary: Rotary, k_new, v_new, offsets, B: int, ws, slots=None, path=None,
                             n_keep=None, stream=None):
    """As attn_cache_append, every K row turned by the position it is stored at (rotary.h)."""
    rows, rest = _append_given(cache, cache.dtype, k_new, v_new, offsets, int(B), ws, slots, path, n_keep)
    _check("attn_cache_append_rotary", lib().attn_cache_append_rotary(cache.ref, rotary.ref, *rows, *rest,
                                                                      _raw_stream(stream, cache.device)))


def attn_cache_fork_workspace_bytes(cache: AttnCache, n: int) -> int:
    return int(lib().attn_cache_fork_workspace_bytes(cache.ref, int(n)))


def attn_cache_fork(cache: AttnCache, src, dst, n: int, ws, stream=None):
    """Slot dst[i] (empty) becomes a copy of slot src[i]: full pages shared, the
    partly filled last page copied.  src, dst int32 [n]."""
    dev, n = cache.device, int(n)
    _here("cache", dev)
    _check("attn_cache_fork", lib().attn_cache_fork(
        cache.ref, _given("src", src, cache.i32, dev, (n,)), _given("dst", dst, cache.i32, dev, (n,)), n,
        *_scratch(ws, dev), _raw_stream(stream, dev)))


def attn_cache_trim(cache: AttnCache, slots, new_lens, n: int, stream=None):
    """Cut n sequences to new_lens (0 frees one); slots int32 [n], or None for 0 .. n-1."""
    dev, n = cache.device, int(n)
    _here("cache", dev)
    _check("attn_cache_trim", lib().attn_cache_trim(
        cache.ref, None if slots is None else _given("slots", slots, cache.i32, dev, (n,)),
        _given("new_lens", new_lens, cache.i32, dev, (n,)), n, _raw_stream(stream, dev)))


def attn_tree_workspace_bytes(cache: AttnCache, B: int, n_nodes: int, max_nodes: int, Hq: int) -> int:
    return int(lib().attn_tree_workspace_bytes(cache.ref, int(B), int(n_nodes), int(max_nodes), int(Hq)))


def attn_tree(cache: AttnCache, layer: int, q, k_new, v_new, offsets, parent, B: int, max_nodes: int, ws, o,
              slots=None, scale: float = 0.0, stream=None):
    """Attention of B drafted trees over the cache's layer (tree.h): q, o
    [n_nodes, Hq, D], k_new, v_new [n_nodes, Hkv, D] of the cache's type, offsets int32
    [B + 1], parent int32 [n_nodes], slots int32 [B] or None (0 .. B-1), ws a
    uint8 device tensor of attn_tree_workspace_bytes bytes or more."""
    dev, dt, i32 = cache.device, cache.dtype, cache.i32
    _here("cache", dev)
    n, Hq, _ = q.shape
    layer, B, max_nodes = int(layer), int(B), int(max_nodes)
    rows, heads = (n, cache.heads, cache.dim), (n, Hq, cache.dim)
    _check("attn_tree", lib().attn_tree(
        cache.ref, layer, _given("q", q, dt, dev, heads), _given("k_new", k_new, dt, dev, rows),
        _given("v_new", v_new, dt, dev, rows), None if slots is None else _given("slots", slots, i32, dev, (B,)),
        _given("offsets", offsets, i32, dev, (B + 1,)), _given("parent", parent, i32, dev, (n,)), B, n, max_nodes, Hq,
        scale, *_scratch(ws, dev), _given("o", o, dt, dev, heads), _raw_stream(stream, dev)))


def moe_draft_verify(p, q, tokens, parent, offsets, u_accept, u_sample, B: int, path, n_path, next_token, status,
                     stream=None):
    """Verify B drafted trees (tree.h): p fp32 [n_nodes, V], q the same or
    None, tokens, parent int32 [n_nodes], offsets int32 [B + 1], u_accept fp32
    [n_nodes], u_sample fp32 [B]; written: path int32 [B, stride], n_path,
    next_token int32 [B], status int32 [>= 1] (on an error)."""
    import torch
    f32, i32, dev = torch.float32, torch.int32, p.get_device()
    _here("p", dev)
    n, V = p.shape
    B, stride = int(B), path.shape[-1]
    _check("moe_draft_verify", lib().moe_draft_verify(
        _given("p", p, f32, dev, (n, V)), None if q is None else _given("q", q, f32, dev, (n, V)),
        _given("tokens", tokens, i32, dev, (n,)), _given("parent", parent, i32, dev, (n,)),
        _given("offsets", offsets, i32, dev, (B + 1,)), _given("u_accept", u_accept, f32, dev, (n,)),
        _given("u_sample", u_sample, f32, dev, (B,)), B, n, V, _given("path", path, i32, dev, (B, stride)), stride,
        _given("n_path", n_path, i32, dev, (B,)), _given("next_token", next_token, i32, dev, (B,)),
        _given("status", status, i32, dev, status.shape), _raw_stream(stream, dev)))


class AttnQCache:
    """An 8-bit paged KV cache (qcache.h): the attn_qcache struct and the tensors behind it."""

    def __init__(self, struct: attn_qcache, tensors: dict):
        import torch
        self.struct = struct
        self.ref = ctypes.byref(struct)
        self.tensors = tensors
        self.i32 = torch.int32
        self.device = tensors["k"].get_device()
        self.layers, self.heads, self.dim = struct.n_layers, struct.n_kv_heads, struct.head_dim


def make_attn_qcache(k, v, k_scale, v_scale, refs, table, lens, status) -> AttnQCache:
    """The cache over the caller's tensors: k, v float8_e4m3fn [n_layers,
    n_pages, page_size, Hkv, D], k_scale, v_scale fp32 [n_layers, n_pages, Hkv], the
    others as for make_attn_cache.  A new cache starts with refs, lens and
    status zero and table -1."""
    import torch
    if k.dtype is not torch.float8_e4m3fn or k.dim() != 5 or table.dim() != 2 or lens.dim() != 1 or status.dim() != 1:
        raise ValueError(f"k: float8_e4m3fn [layers, pages, page_size, heads, dim], table of 2, lens and status of 1 "
                         f"dimensions wanted, got k {k.dtype} {tuple(k.shape)}")
    layers, pages, page, heads, dim = k.shape
    dev, ints, scales = k.get_device(), torch.int32, (layers, pages, heads)
    st = attn_qcache(_given("k", k, k.dtype, dev, k.shape), _given("v", v, k.dtype, dev, k.shape),
                     _given("k_scale", k_scale, torch.float32, dev, scales),
                     _given("v_scale", v_scale, torch.float32, dev, scales),
                     _given("refs", refs, ints, dev, (pages,)),
                     _given("table", table, ints, dev, (lens.shape[0], table.shape[1])),
                     _given("lens", lens, ints, dev, lens.shape), _given("status", status, ints, dev, status.shape),
                     layers, pages, page, heads, dim, lens.shape[0], table.shape[1], 0)
    return AttnQCache(st, dict(k=k, v=v, k_scale=k_scale, v_scale=v_scale, refs=refs, table=table, lens=lens,
                               status=status))


def attn_qcache_append_workspace_bytes(cache: AttnQCache, B: int, n_rows: int) -> int:
    return int(lib().attn_qcache_append_workspace_bytes(cache.ref, int(B), int(n_rows)))


def attn_qcache_append(cache: AttnQCache, rotary, k_new, v_new, offsets, B: int, ws, slots=None, path=None, n_keep=None,
                       stream=None):
    """As attn_cache_append, into e4m3 codes (qcache.h); k_new, v_new bf16 or fp16.
    ``rotary``: K rows are turned by the position they are stored at; None: not."""
    kind = _kind("k_new", k_new.dtype)
    rows, rest = _append_given(cache, k_new.dtype, k_new, v_new, offsets, int(B), ws, slots, path, n_keep)
    _check("attn_qcache_append", lib().attn_qcache_append(cache.ref, None if rotary is None else rotary.ref, *rows, kind,
                                                          *rest, _raw_stream(stream, cache.device)))


def attn_qcache_fork_workspace_bytes(cache: AttnQCache, n: int) -> int:
    return int(lib().attn_qcache_fork_workspace_bytes(cache.ref, int(n)))


def attn_qcache_fork(cache: AttnQCache, src, dst, n: int, ws, stream=None):
    """As attn_cache_fork; a copied page brings its scales."""
    dev, n = cache.device, int(n)
    _here("cache", dev)
    _check("attn_qcache_fork", lib().attn_qcache_fork(
        cache.ref, _given("src", src, cache.i32, dev, (n,)), _given("dst", dst, cache.i32, dev, (n,)), n,
        *_scratch(ws, dev), _raw_stream(stream, dev)))


def attn_qcache_trim(cache: AttnQCache, slots, new_lens, n: int, stream=None):
    """As attn_cache_trim."""
    dev, n = cache.device, int(n)
    _here("cache", dev)
    _check("attn_qcache_trim", lib().attn_qcache_trim(
        cache.ref, None if slots is None else _given("slots", slots, cache.i32, dev, (n,)),
        _given("new_lens", new_lens, cache.i32, dev, (n,)), n, _raw_stream(stream, dev)))


def attn_qcache_attend_workspace_bytes(cache: AttnQCache, B: int, n_rows: int, max_rows: int, Hq: int) -> int:
    return int(lib().attn_qcache_attend_workspace_bytes(cache.ref, int(B), int(n_rows), int(max_rows), int(Hq)))


def attn_qcache_attend(cache: AttnQCache, layer: int, q, offsets, B: int, max_rows: int, ws, o, slots=None,
                       scale: float = 0.0, stream=None):
    """Attention of the last rows of B sequences over the 8-bit cache's layer
    (qcache.h): q, o [n_rows, Hq, D] bf16 or fp16, offsets int32 [B + 1], slots
    int32 [B] or None (0 .. B-1), ws a uint8 device tensor of
    attn_qcache_attend_workspace_bytes bytes or more."""
    dev, i32 = cache.device, cache.i32
    _here("cache", dev)
    n, Hq, _ = q.shape
    layer, B, max_rows, shape = int(layer), int(B), int(max_rows), (n, Hq, cache.dim)
    kind = _kind("q", q.dtype)
    _check("attn_qcache_attend", lib().attn_qcache_attend(
        cache.ref, layer, _given("q", q, q.dtype, dev, shape), kind,
        None if slots is None else _given("slots", slots, i32, dev, (B,)), _given("offsets", offsets, i32, dev, (B + 1,)),
        B, n, max_rows, Hq, scale, *_scratch(ws, dev), _given("o", o, q.dtype, dev, shape), _raw_stream(stream, dev)))


def moe_route_view(plan: Plan, ws, T: int) -> moe_route_ptrs:
    r = moe_route_ptrs()
    _check("moe_route_view", lib().moe_route_view(plan.handle, _ptr(ws), int(T), ctypes.byref(r)))
    return r


def workspace_tensor(ws, ptr: int, numel: int, dtype):
    """A typed view of ``numel`` elements of the workspace tensor ``ws`` (a
    uint8 tensor) starting at device address ``ptr`` (from moe_route_view)."""
    off = int(ptr) - ws.data_ptr()
    nbytes = numel * _itemsize(dtype)
    if off < 0 or off + nbytes > _nbytes(ws):
        raise ValueError("pointer range outside the workspace")
    return ws[off:off + nbytes].view(dtype)


def _itemsize(dtype):
    import torch
    return torch.empty((), dtype=dtype).element_size()


def moe_rmsnorm(r, T: int, H: int, eps: float, x, stream=None):
    _check("moe_rmsnorm", lib().moe_rmsnorm(_ptr(r), int(T), int(H), float(eps), _ptr(x), _stream(stream)))


def moe_dequant(q, s, b, rows: int, K: int, G: int, w, stream=None):
    _check("moe_dequant", lib().moe_dequant(_ptr(q), _ptr(s), _ptr(b), int(rows), int(K), int(G), _ptr(w),
                                            _stream(stream)))


def moe_device_status(plan: Plan, ws, stream=None, reset: bool = True) -> int:
    st = ctypes.c_int32(-1)
    _check("moe_device_status", lib().moe_device_status(plan.handle, _ptr(ws), _stream(stream), ctypes.byref(st),
                                                        int(bool(reset))))
    return int(st.value)


def moe_last_launch_count() -> int:
    return int(lib().moe_last_launch_count())


def moe_profile_events(kernel: int, start_events=(), stop_events=()):
    """Bracket the i-th later launch of ``kernel`` on this thread with
    ``start_events[i % n]`` / ``stop_events[i % n]`` (torch.cuda.Event objects
    created with enable_timing=True); empty lists turn the hook off."""
    n = len(start_events)
    if n != len(stop_events):
        raise ValueError("start and stop event lists differ in length")
    for e in list(start_events) + list(stop_events):
        if not e.cuda_event:  # torch creates the CUDA event lazily, on its first record
            e.record()
    arr = ctypes.c_void_p * max(n, 1)
    a = arr(*[e.cuda_event for e in start_events]) if n else None
    b = arr(*[e.cuda_event for e in stop_events]) if n else None
    _check("moe_profile_events", lib().moe_profile_events(int(kernel), a, b, n))


def moe_profile_stride(kernel: int, stride: int):
    """Bracket only every ``stride``-th launch of ``kernel`` from now on."""
    _check("moe_profile_stride", lib().moe_profile_stride(int(kernel), int(stride)))
