"""Python binding of libmoe_mxfp4 (the MXFP4 MoE expert FFN on MI355X).

Argument marshalling only: every step of the forward path runs in the HIP
kernels behind the C ABI in ``include/moe_mxfp4.h``.  PyTorch supplies device
memory and the current stream; nothing here computes any part of the method,
and there is no CPU fallback -- if the library is missing, loading fails.

Names follow the C ABI: ``MoeMxfp4`` wraps ``moe_mxfp4_create / _forward /
_destroy / _workspace_bytes / _debug_dequant``; ``quantize_weights`` wraps
``moe_mxfp4_quantize_weights``; ``dflash_accept`` wraps
``moe_mxfp4_dflash_accept`` (the rejection-sampling pass of a verify step).
The attention half of the step: ``KvCache`` (a paged cache's buffers),
``cache_plan``, ``qk_norm_rope``, ``attention`` and ``kv_read`` wrap the
entries of the same names.
"""
from __future__ import annotations

import collections
import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_mxfp4.so")

MOE_OK = 0
STATUS_NAMES = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED_SHAPE",
                3: "MOE_ERR_CAPACITY", 4: "MOE_ERR_ALIGNMENT", 5: "MOE_ERR_WORKSPACE",
                6: "MOE_ERR_HIP", 7: "MOE_ERR_INTERNAL"}
ACT_BF16, ACT_MXFP8_E4M3 = 0, 1
OUT_BF16, OUT_F32 = 0, 1
KV_BF16, KV_MXFP4 = 0, 1

# Every symbol include/moe_mxfp4.h declares.
EXPORTS = ("moe_mxfp4_status_string", "moe_mxfp4_abi_version", "moe_mxfp4_create",
           "moe_mxfp4_destroy", "moe_mxfp4_workspace_bytes", "moe_mxfp4_forward",
           "moe_mxfp4_debug_dequant", "moe_mxfp4_quantize_weights", "moe_mxfp4_stage_timing",
           "moe_mxfp4_stage_times", "moe_mxfp4_tiled_scale_bytes", "moe_mxfp4_tile_weights",
           "moe_mxfp4_quantize_act_mxfp8", "moe_mxfp4_router_logits", "moe_mxfp4_forward_hidden",
           "moe_mxfp4_dflash_workspace_bytes", "moe_mxfp4_dflash_accept", "moe_mxfp4_probe",
           "moe_mxfp4_forward_noalloc", "moe_mxfp4_device_status", "moe_mxfp4_debug_hidden",
           "moe_mxfp4_kv_cache_bytes", "moe_mxfp4_cache_plan", "moe_mxfp4_qk_norm_rope", "moe_mxfp4_kv_read",
           "moe_mxfp4_attention_workspace_bytes", "moe_mxfp4_attention")
# Scratch bytes moe_mxfp4_forward_noalloc holds per GPU (MOE_MXFP4_NOALLOC_SCRATCH_BYTES).
NOALLOC_SCRATCH_BYTES = 64 << 20
# Largest batch (tokens x top_k) the fused path runs (MOE_MXFP4_FUSED_MAX_PAIRS);
# larger ones take the per-phase launches.
FUSED_MAX_PAIRS = 8192
NUM_STAGES = 6
STAGES = ("route", "sort", "quant", "gateup", "down", "combine")


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


class Config(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("num_experts", ctypes.c_int32),
                ("d_model", ctypes.c_int32), ("d_ff", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("max_tokens", ctypes.c_int32), ("act_mode", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class Weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("w_gate", "w_gate_scale", "w_up", "w_up_scale",
                                               "w_down", "w_down_scale")]


class Routing(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("topk_ids", "topk_w", "expert_offsets",
                                               "sorted_pairs")]


class KvCacheStruct(ctypes.Structure):
    _fields_ = ([("struct_size", ctypes.c_uint32)] +
                [(n, ctypes.c_int32) for n in ("format", "num_pages", "page_size", "kv_heads", "head_dim")] +
                [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale")])


class PlanArgs(ctypes.Structure):
    _fields_ = ([("struct_size", ctypes.c_uint32)] +
                [(n, ctypes.c_int32) for n in ("batch", "num_tokens", "max_blocks", "page_size", "num_pages")] +
                [(n, ctypes.c_void_p) for n in ("ctx_lens", "new_lens", "block_table", "held", "held_out", "free_ring",
                                                "free_state", "free_state_out", "cu_q", "kv_lens", "slots",
                                                "positions", "refused")])


class RopeArgs(ctypes.Structure):
    _fields_ = ([("struct_size", ctypes.c_uint32)] +
                [(n, ctypes.c_int32) for n in ("num_tokens", "heads", "kv_heads", "head_dim", "rot_dim",
                                               "interleaved")] + [("eps", ctypes.c_float)] +
                [(n, ctypes.c_int64) for n in ("q_stride", "k_stride", "v_stride")] +
                [(n, ctypes.c_void_p) for n in ("q", "k", "v", "q_weight", "k_weight", "inv_freq", "positions",
                                                "slots", "q_out", "k_out")])


class AttnArgs(ctypes.Structure):
    _fields_ = ([("struct_size", ctypes.c_uint32)] +
                [(n, ctypes.c_int32) for n in ("batch", "num_tokens", "heads", "max_q", "max_kv", "max_blocks",
                                               "causal", "window", "sinks")] + [("scale", ctypes.c_float)] +
                [(n, ctypes.c_int64) for n in ("q_stride", "out_stride")] +
                [(n, ctypes.c_void_p) for n in ("q", "out", "block_table", "cu_q", "kv_lens")])


_lib = None


def lib():
    """Load the HIP library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              f"`python -m mxfp4_expert_ffn_amd.build` (hipcc, gfx950)")
        L = ctypes.CDLL(LIB_PATH)
        P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        L.moe_mxfp4_status_string.argtypes = [ctypes.c_int]
        L.moe_mxfp4_status_string.restype = ctypes.c_char_p
        L.moe_mxfp4_abi_version.argtypes = []
        L.moe_mxfp4_abi_version.restype = i32
        L.moe_mxfp4_create.argtypes = [ctypes.POINTER(Config), ctypes.POINTER(Weights),
                                       ctypes.POINTER(P)]
        L.moe_mxfp4_create.restype = ctypes.c_int
        L.moe_mxfp4_destroy.argtypes = [P]
        L.moe_mxfp4_destroy.restype = ctypes.c_int
        L.moe_mxfp4_workspace_bytes.argtypes = [P, i32]
        L.moe_mxfp4_workspace_bytes.restype = sz
        L.moe_mxfp4_forward.argtypes = [P, P, P, i32, P, P, sz, P, ctypes.POINTER(Routing)]
        L.moe_mxfp4_forward.restype = ctypes.c_int
        L.moe_mxfp4_forward_noalloc.argtypes = [P, P, P, i32, P, P, ctypes.POINTER(Routing)]
        L.moe_mxfp4_forward_noalloc.restype = ctypes.c_int
        L.moe_mxfp4_debug_hidden.argtypes = [P, P, i32, P, P, P]
        L.moe_mxfp4_debug_hidden.restype = ctypes.c_int
        L.moe_mxfp4_device_status.argtypes = [P, P, i32, ctypes.POINTER(i32), P]
        L.moe_mxfp4_device_status.restype = ctypes.c_int
        L.moe_mxfp4_forward_hidden.argtypes = [P, P, P, i32, P, P, sz, P, ctypes.POINTER(Routing)]
        L.moe_mxfp4_forward_hidden.restype = ctypes.c_int
        L.moe_mxfp4_router_logits.argtypes = [P, P, P, i32, P, P]
        L.moe_mxfp4_router_logits.restype = ctypes.c_int
        L.moe_mxfp4_debug_dequant.argtypes = [P, i32, i32, i32, i32, P, P]
        L.moe_mxfp4_debug_dequant.restype = ctypes.c_int
        L.moe_mxfp4_quantize_weights.argtypes = [P, i64, i64, P, P, P]
        L.moe_mxfp4_quantize_weights.restype = ctypes.c_int
        L.moe_mxfp4_quantize_act_mxfp8.argtypes = [P, i64, i64, P, P, P]
        L.moe_mxfp4_quantize_act_mxfp8.restype = ctypes.c_int
        L.moe_mxfp4_tiled_scale_bytes.argtypes = [i64, i64]
        L.moe_mxfp4_tiled_scale_bytes.restype = sz
        L.moe_mxfp4_tile_weights.argtypes = [P, P, i64, i64, P, P, P]
        L.moe_mxfp4_tile_weights.restype = ctypes.c_int
        L.moe_mxfp4_dflash_workspace_bytes.argtypes = [i32, i32]
        L.moe_mxfp4_dflash_workspace_bytes.restype = sz
        L.moe_mxfp4_dflash_accept.argtypes = [i32, i32, i32, P, P, P, P, P, P, P, P, sz, P]
        L.moe_mxfp4_dflash_accept.restype = ctypes.c_int
        L.moe_mxfp4_kv_cache_bytes.argtypes = [ctypes.POINTER(KvCacheStruct), ctypes.POINTER(sz), ctypes.POINTER(sz)]
        L.moe_mxfp4_kv_cache_bytes.restype = ctypes.c_int
        L.moe_mxfp4_cache_plan.argtypes = [ctypes.POINTER(PlanArgs), P]
        L.moe_mxfp4_cache_plan.restype = ctypes.c_int
        L.moe_mxfp4_qk_norm_rope.argtypes = [ctypes.POINTER(RopeArgs), ctypes.POINTER(KvCacheStruct), P]
        L.moe_mxfp4_qk_norm_rope.restype = ctypes.c_int
        L.moe_mxfp4_kv_read.argtypes = [ctypes.POINTER(KvCacheStruct), P, i32, P, P, P]
        L.moe_mxfp4_kv_read.restype = ctypes.c_int
        L.moe_mxfp4_attention_workspace_bytes.argtypes = [ctypes.POINTER(AttnArgs), ctypes.POINTER(KvCacheStruct)]
        L.moe_mxfp4_attention_workspace_bytes.restype = sz
        L.moe_mxfp4_attention.argtypes = [ctypes.POINTER(AttnArgs), ctypes.POINTER(KvCacheStruct), P, sz, P]
        L.moe_mxfp4_attention.restype = ctypes.c_int
        L.moe_mxfp4_probe.argtypes = [i32, P, sz, i32, P, ctypes.POINTER(ctypes.c_double), P]
        L.moe_mxfp4_probe.restype = ctypes.c_int
        L.moe_mxfp4_stage_timing.argtypes = [P, i32]
        L.moe_mxfp4_stage_timing.restype = ctypes.c_int
        L.moe_mxfp4_stage_times.argtypes = [P, ctypes.POINTER(ctypes.c_float),
                                            ctypes.POINTER(i32)]
        L.moe_mxfp4_stage_times.restype = ctypes.c_int
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().moe_mxfp4_status_string(status).decode()


def _check(status: int, where: str):
    if status != MOE_OK:
        raise MoeError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _require(t, dtype, shape, name):
    """Argument check of the binding: a contiguous CUDA tensor of this dtype and shape."""
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous CUDA {dtype} tensor of shape {tuple(shape)}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")


def _torch_stream(stream=None):
    import torch
    return torch.cuda.current_stream() if stream is None else stream


def _stream(stream=None):
    return ctypes.c_void_p(_torch_stream(stream).cuda_stream)


ROUTING_FIELDS = ("topk_ids", "topk_w", "expert_offsets", "sorted_pairs")


def _routing_struct(routing, T, k, E):
    """Routing outputs (dict of optional CUDA tensors) -> the C struct, after
    checking each tensor's dtype, size and contiguity."""
    import torch
    if routing is None:
        return None
    unknown = set(routing) - set(ROUTING_FIELDS)
    if unknown:
        raise ValueError(f"routing: unknown outputs {sorted(unknown)}")
    want = {"topk_ids": (torch.int32, T * k), "topk_w": (torch.float32, T * k),
            "expert_offsets": (torch.int32, E + 1), "sorted_pairs": (torch.int32, T * k)}
    for n, t in routing.items():
        if t is None:
            continue
        dt, numel = want[n]
        if t.dtype != dt or t.numel() < numel or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"routing[{n!r}]: expected a contiguous CUDA {dt} tensor of at least {numel} "
                             f"elements, got {t.dtype} {tuple(t.shape)} on {t.device}")
    return Routing(*[_ptr(routing.get(n)) for n in ROUTING_FIELDS])


def make_config(num_experts, d_model, d_ff, top_k, max_tokens, act_mode=ACT_BF16,
                out_dtype=OUT_BF16, flags=0) -> Config:
    return Config(ctypes.sizeof(Config), num_experts, d_model, d_ff, top_k, max_tokens,
                  act_mode, out_dtype, flags)


class MoeMxfp4:
    """One expert layer: borrowed packed weights + configuration.

    ``weights``: dict of uint8 CUDA tensors in the TILED layout of the C
    header (``tile_expert_weights`` converts the row-major form): ``w_gate``,
    ``w_gate_scale``, ``w_up``, ``w_up_scale``, ``w_down``, ``w_down_scale``.
    References are kept for the life of this object.
    """

    def __init__(self, weights: dict, num_experts: int, d_model: int, d_ff: int, top_k: int,
                 max_tokens: int, act_mode: int = ACT_BF16, out_dtype: int = OUT_BF16):
        self.cfg = make_config(num_experts, d_model, d_ff, top_k, max_tokens, act_mode, out_dtype)
        self.weights = dict(weights)
        self.out_dtype = out_dtype
        w = Weights(*[_ptr(self.weights[n]) for n in ("w_gate", "w_gate_scale", "w_up",
                                                      "w_up_scale", "w_down", "w_down_scale")])
        h = ctypes.c_void_p()
        _check(lib().moe_mxfp4_create(ctypes.byref(self.cfg), ctypes.byref(w), ctypes.byref(h)),
               "moe_mxfp4_create")
        self._ctx = h
        self._ws = {}            # cached workspace per stream handle

    def close(self):
        if getattr(self, "_ctx", None) is not None and self._ctx.value:
            lib().moe_mxfp4_destroy(self._ctx)
            self._ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def workspace_bytes(self, num_tokens: int) -> int:
        return lib().moe_mxfp4_workspace_bytes(self._ctx, num_tokens)

    def workspace(self, num_tokens: int, stream=None):
        """A cached uint8 workspace large enough for ``num_tokens``, one per
        stream (calls that may run at the same time need distinct
        workspaces).  It is allocated on that stream, so the caching
        allocator reuses its memory only after the stream's queued work."""
        import torch
        s = _torch_stream(stream)
        need = self.workspace_bytes(num_tokens)
        ws = self._ws.get(s.cuda_stream)
        if ws is None or ws.numel() < need:
            with torch.cuda.stream(s):
                ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
            self._ws[s.cuda_stream] = ws
        return ws

    def _out(self, out, T, device, stream):
        import torch
        dt = torch.bfloat16 if self.out_dtype == OUT_BF16 else torch.float32
        if out is None:
            with torch.cuda.stream(_torch_stream(stream)):
                return torch.empty((T, self.cfg.d_model), dtype=dt, device=device)
        _require(out, dt, (T, self.cfg.d_model), "out")
        return out

    def forward(self, hidden, logits, out=None, workspace=None, routing: dict | None = None,
                stream=None, w_router=None):
        """hidden: bf16 [T, d] CUDA; logits: float32 [T, E] CUDA -> out [T, d].

        With ``w_router`` (bf16 [E, d] CUDA) and ``logits=None`` the logits are
        projected from ``hidden`` inside the call (moe_mxfp4_forward_hidden).
        """
        import torch
        if (logits is None) == (w_router is None):
            raise ValueError("pass exactly one of logits and w_router")
        T = hidden.shape[0]
        E, d = self.cfg.num_experts, self.cfg.d_model
        _require(hidden, torch.bfloat16, (T, d), "hidden")
        if logits is not None:
            _require(logits, torch.float32, (T, E), "logits")
        else:
            _require(w_router, torch.bfloat16, (E, d), "w_router")
        out = self._out(out, T, hidden.device, stream)
        ws = self.workspace(T, stream) if workspace is None else workspace
        r = _routing_struct(routing, T, self.cfg.top_k, E)
        fn, name = ((lib().moe_mxfp4_forward, "moe_mxfp4_forward") if w_router is None else
                    (lib().moe_mxfp4_forward_hidden, "moe_mxfp4_forward_hidden"))
        st = fn(self._ctx, _ptr(hidden), _ptr(logits if w_router is None else w_router), T, _ptr(out),
                _ptr(ws), ws.numel() if ws is not None else 0, _stream(stream),
                ctypes.byref(r) if r is not None else None)
        _check(st, name)
        return out

    __call__ = forward

    def forward_noalloc(self, hidden, logits, out, routing: dict | None = None, stream=None):
        """moe_mxfp4_forward_noalloc: as ``forward`` with the logits given,
        but on the library's own per-GPU scratch (no workspace, nothing
        allocated); ``out`` must be given.  Calls on one GPU share the
        scratch, so they must not overlap in time."""
        import torch
        T = hidden.shape[0]
        _require(hidden, torch.bfloat16, (T, self.cfg.d_model), "hidden")
        _require(logits, torch.float32, (T, self.cfg.num_experts), "logits")
        out = self._out(out, T, hidden.device, stream)
        r = _routing_struct(routing, T, self.cfg.top_k, self.cfg.num_experts)
        _check(lib().moe_mxfp4_forward_noalloc(self._ctx, _ptr(hidden), _ptr(logits), T, _ptr(out), _stream(stream),
                                               ctypes.byref(r) if r is not None else None),
               "moe_mxfp4_forward_noalloc")
        return out

    def device_status(self, num_tokens: int, workspace=None, stream=None) -> int:
        """The fused kernels' error word of the last call with ``num_tokens``
        tokens: on ``stream`` where the expert launch routes a verify block itself,
        else on ``workspace`` (default: this object's cached workspace for
        ``stream``); waits for the stream.  0 = no device-side wait gave up."""
        ws = self.workspace(num_tokens, stream) if workspace is None else workspace
        st = ctypes.c_int32()
        _check(lib().moe_mxfp4_device_status(self._ctx, _ptr(ws), num_tokens, ctypes.byref(st), _stream(stream)),
               "moe_mxfp4_device_status")
        return st.value

    def debug_hidden(self, num_tokens: int, workspace=None, stream=None):
        """h of the last call with ``num_tokens`` tokens on ``workspace``
        (default: the cached one), rows in expert-sorted order: MXFP8 mode
        (uint8 codes [P, d_ff], uint8 E8M0 scales [P, d_ff/32]); bf16 mode
        (bf16 [P, d_ff], None)."""
        import torch
        ws = self.workspace(num_tokens, stream) if workspace is None else workspace
        P, f = num_tokens * self.cfg.top_k, self.cfg.d_ff
        if self.cfg.act_mode == ACT_MXFP8_E4M3:
            h = torch.empty((P, f), dtype=torch.uint8, device="cuda")
            sc = torch.empty((P, f // 32), dtype=torch.uint8, device="cuda")
        else:
            h, sc = torch.empty((P, f), dtype=torch.bfloat16, device="cuda"), None
        _check(lib().moe_mxfp4_debug_hidden(self._ctx, _ptr(ws), num_tokens, _ptr(h), _ptr(sc), _stream(stream)),
               "moe_mxfp4_debug_hidden")
        return h, sc

    def router_logits(self, hidden, w_router, out=None, stream=None):
        """hidden: bf16 [T, d]; w_router: bf16 [E, d] -> float32 logits [T, E]."""
        import torch
        T = hidden.shape[0]
        _require(hidden, torch.bfloat16, (T, self.cfg.d_model), "hidden")
        _require(w_router, torch.bfloat16, (self.cfg.num_experts, self.cfg.d_model), "w_router")
        if out is None:
            out = torch.empty((T, self.cfg.num_experts), dtype=torch.float32, device=hidden.device)
        _check(lib().moe_mxfp4_router_logits(self._ctx, _ptr(hidden), _ptr(w_router), T, _ptr(out),
                                             _stream(stream)), "moe_mxfp4_router_logits")
        return out

    def stage_timing(self, capacity: int):
        """Record HIP events around each stage of the next forward calls."""
        _check(lib().moe_mxfp4_stage_timing(self._ctx, capacity), "moe_mxfp4_stage_timing")

    def stage_times(self):
        """(per-stage summed ms as a dict, number of calls) since the last read."""
        ms = (ctypes.c_float * NUM_STAGES)()
        n = ctypes.c_int32()
        _check(lib().moe_mxfp4_stage_times(self._ctx, ms, ctypes.byref(n)), "moe_mxfp4_stage_times")
        return dict(zip(STAGES, list(ms))), n.value

    def debug_dequant(self, expert: int, matrix: int, row0: int, nrows: int, out=None, stream=None):
        import torch
        K = self.cfg.d_ff if matrix == 2 else self.cfg.d_model
        if out is None:
            out = torch.empty((nrows, K), dtype=torch.float32, device="cuda")
        _check(lib().moe_mxfp4_debug_dequant(self._ctx, expert, matrix, row0, nrows, _ptr(out),
                                             _stream(stream)), "moe_mxfp4_debug_dequant")
        return out


def quantize_weights(w, packed=None, scales=None, stream=None):
    """float32 CUDA [rows, K] -> (packed uint8 [rows, K/2], scales uint8 [rows, K/32])."""
    import torch
    rows, K = w.shape
    if packed is None:
        packed = torch.empty((rows, K // 2), dtype=torch.uint8, device=w.device)
    if scales is None:
        scales = torch.empty((rows, K // 32), dtype=torch.uint8, device=w.device)
    _check(lib().moe_mxfp4_quantize_weights(_ptr(w), rows, K, _ptr(packed), _ptr(scales),
                                            _stream(stream)), "moe_mxfp4_quantize_weights")
    return packed, scales


def tiled_scale_bytes(rows: int, K: int) -> int:
    return lib().moe_mxfp4_tiled_scale_bytes(rows, K)


def tile_weights(packed, scales, stream=None):
    """Row-major packed [rows, K/2] + scales [rows, K/32] (uint8 CUDA) -> tiled
    (packed uint8 [rows*K/2], scales uint8 [tiled_scale_bytes(rows, K)])."""
    import torch
    rows, K = packed.shape[0], packed.shape[1] * 2
    tp = torch.empty(rows * K // 2, dtype=torch.uint8, device=packed.device)
    ts = torch.empty(tiled_scale_bytes(rows, K), dtype=torch.uint8, device=packed.device)
    _check(lib().moe_mxfp4_tile_weights(_ptr(packed), _ptr(scales), rows, K, _ptr(tp), _ptr(ts),
                                        _stream(stream)), "moe_mxfp4_tile_weights")
    return tp, ts


def tile_expert_weights(rowmajor: dict, stream=None) -> dict:
    """Row-major expert weights (uint8 CUDA tensors shaped [E, N, K/2] and
    [E, N, K/32]) -> the tiled dict the forward path takes."""
    out = {}
    for name in ("w_gate", "w_up", "w_down"):
        p, sc = rowmajor[name], rowmajor[name + "_scale"]
        E, N, half = p.shape
        tp, ts = tile_weights(p.reshape(E * N, half), sc.reshape(E * N, sc.shape[2]), stream)
        out[name], out[name + "_scale"] = tp, ts
    return out


def quantize_act_mxfp8(x, codes=None, scales=None, stream=None):
    """bf16 CUDA [rows, K] -> (E4M3 codes uint8 [rows, K], E8M0 scales uint8 [rows, K/32])."""
    import torch
    rows, K = x.shape
    if codes is None:
        codes = torch.empty((rows, K), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((rows, K // 32), dtype=torch.uint8, device=x.device)
    _check(lib().moe_mxfp4_quantize_act_mxfp8(_ptr(x), rows, K, _ptr(codes), _ptr(scales),
                                              _stream(stream)), "moe_mxfp4_quantize_act_mxfp8")
    return codes, scales


def dflash_workspace_bytes(batch: int, vocab: int) -> int:
    return lib().moe_mxfp4_dflash_workspace_bytes(batch, vocab)


def dflash_accept(draft, p_draft, p_target, u, r, n_accepted=None, next_token=None, workspace=None,
                  stream=None):
    """Rejection-sampling acceptance of drafted blocks (moe_mxfp4_dflash_accept).

    draft int32 [B, G], p_draft float32 [B, G, V], p_target float32 [B, G+1, V],
    u float32 [B, G], r float32 [B], all contiguous CUDA tensors ->
    (n_accepted int32 [B], next_token int32 [B]).
    """
    import torch
    B, G = draft.shape
    V = p_target.shape[2]
    if p_target.shape != (B, G + 1, V) or p_draft.shape != (B, G, V) or u.shape != (B, G) or r.shape != (B,):
        raise ValueError("dflash_accept: inconsistent shapes")
    want = ((draft, torch.int32), (p_draft, torch.float32), (p_target, torch.float32), (u, torch.float32),
            (r, torch.float32))
    for t, dt in want:
        if t.dtype != dt or not t.is_cuda or not t.is_contiguous():
            raise ValueError("dflash_accept: draft must be int32 and the rest float32, all contiguous CUDA tensors")
    if n_accepted is None:
        n_accepted = torch.empty(B, dtype=torch.int32, device=p_target.device)
    if next_token is None:
        next_token = torch.empty(B, dtype=torch.int32, device=p_target.device)
    if workspace is None:
        workspace = torch.empty(max(dflash_workspace_bytes(B, V), 256), dtype=torch.uint8,
                                device=p_target.device)
    _check(lib().moe_mxfp4_dflash_accept(B, G, V, _ptr(draft), _ptr(p_draft), _ptr(p_target), _ptr(u),
                                         _ptr(r), _ptr(n_accepted), _ptr(next_token), _ptr(workspace),
                                         workspace.numel(), _stream(stream)), "moe_mxfp4_dflash_accept")
    return n_accepted, next_token


def _like(t, dtype, shape, device, name):
    """Argument check: a contiguous tensor of this dtype and shape on this CUDA device."""
    if t.dtype != dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")


def _heads(t, D, device, name):
    """Argument check: bf16 [T, heads, D] on this CUDA device whose heads of a token are contiguous; its token stride."""
    import torch
    if t.dtype == torch.bfloat16 and t.device == device and t.dim() == 3:
        n, h, d = t.shape
        token, head, element = t.stride()
        if d == D and (element == 1 and (head == D or h == 1) or n == 0 or h == 0):
            # the stride between tokens is of no account where there are not two
            return token if n > 1 else h * D
    raise ValueError(f"{name}: expected bfloat16 [T, heads, {D}] on {device} with contiguous heads, got {t.dtype} "
                     f"{tuple(t.shape)} with strides {t.stride()} on {t.device}")


def _handle_on(device, stream):
    """The stream's handle where it and the device are current (``stream`` None: the device's current one), else
    None: then the call has to be made again inside ``_made_current``."""
    import torch
    if device.type != "cuda":
        raise ValueError(f"expected CUDA tensors, got {device}")
    if torch._C._cuda_getDevice() != device.index:
        return None
    # the current stream's handle as it is: a stream object for it costs as much as a launch
    own = torch._C._cuda_getCurrentRawStream(device.index)
    return own if stream is None or (stream.device == device and stream.cuda_stream == own) else None


def _made_current(device, stream):
    """The context in which the stream (None: the device's current one) and the device are current."""
    import torch
    if stream is not None and stream.device != device:
        raise ValueError(f"stream of {stream.device} for tensors on {device}")
    return torch.cuda.stream(torch.cuda.current_stream(device) if stream is None else stream)


class KvCache:
    """A paged key/value cache of ``num_pages`` pages of ``page_size`` tokens.

    ``fmt``: ``KV_MXFP4`` (uint8 codes and E8M0 scale bytes) or ``KV_BF16``.
    The buffers ``k``, ``v`` [pages, kv_heads, page_size, D/2 or D] and
    ``k_scale``, ``v_scale`` [pages, kv_heads, page_size, D/32] (None for
    bf16) have the layout of the C header; they start zeroed.  ``wrap`` takes
    existing buffers.
    """

    def __init__(self, num_pages: int, page_size: int, kv_heads: int, head_dim: int, fmt: int = KV_MXFP4,
                 device="cuda"):
        import torch
        if fmt not in (KV_BF16, KV_MXFP4):
            raise ValueError(f"fmt: expected KV_BF16 or KV_MXFP4, got {fmt}")
        shape = (num_pages, kv_heads, page_size)
        if fmt == KV_BF16:
            k, v = (torch.zeros((*shape, head_dim), dtype=torch.bfloat16, device=device) for _ in range(2))
            self._take(k, v, None, None)
        else:
            k, v = (torch.zeros((*shape, head_dim // 2), dtype=torch.uint8, device=device) for _ in range(2))
            ks, vs = (torch.zeros((*shape, head_dim // 32), dtype=torch.uint8, device=device) for _ in range(2))
            self._take(k, v, ks, vs)

    @classmethod
    def wrap(cls, k, v, k_scale=None, v_scale=None):
        self = cls.__new__(cls)
        self._take(k, v, k_scale, v_scale)
        return self

    def _take(self, k, v, k_scale, v_scale):
        import torch
        fp4 = k_scale is not None
        if k.dim() != 4:
            raise ValueError(f"k: expected 4 dimensions, got {tuple(k.shape)}")
        pages, heads, ps, width = k.shape
        D = width * 2 if fp4 else width
        dt = torch.uint8 if fp4 else torch.bfloat16
        _like(k, dt, k.shape, k.device, "k")
        _like(v, dt, k.shape, k.device, "v")
        if fp4:
            _like(k_scale, torch.uint8, (pages, heads, ps, D // 32), k.device, "k_scale")
            _like(v_scale, torch.uint8, (pages, heads, ps, D // 32), k.device, "v_scale")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.fmt = KV_MXFP4 if fp4 else KV_BF16
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = pages, heads, ps, D
        self.device = k.device
        self.struct = KvCacheStruct(ctypes.sizeof(KvCacheStruct), self.fmt, pages, ps, heads, D, k.data_ptr(), v.data_ptr(),
                                    k_scale.data_ptr() if fp4 else None, v_scale.data_ptr() if fp4 else None)
        self.ref = ctypes.byref(self.struct)
        data, scale = ctypes.c_size_t(), ctypes.c_size_t()
        _check(lib().moe_mxfp4_kv_cache_bytes(self.ref, ctypes.byref(data), ctypes.byref(scale)),
               "moe_mxfp4_kv_cache_bytes")


CachePlan = collections.namedtuple("CachePlan", "cu_q kv_lens slots positions refused held free_state")


def cache_plan(ctx_lens, new_lens, block_table, held, free_ring, free_state, *, page_size: int, num_tokens: int,
               held_out=None, free_out=None, out: CachePlan | None = None, stream=None) -> CachePlan:
    """Block tables and slot map of a step, from request lengths (moe_mxfp4_cache_plan).

    int32 CUDA tensors: ctx_lens, new_lens, held [B], block_table [B, max_blocks]
    and free_ring [num_pages] (both updated), free_state [2].  ``held_out``
    and ``free_out`` receive the state after the call and must not be the
    inputs; ``out``: an earlier result whose tensors are used again.
    """
    import torch
    i32, dev = torch.int32, block_table.device
    B, W = block_table.shape
    N = free_ring.numel()
    for t, shape, name in ((ctx_lens, (B,), "ctx_lens"), (new_lens, (B,), "new_lens"), (held, (B,), "held"),
                           (block_table, (B, W), "block_table"), (free_ring, (N,), "free_ring"),
                           (free_state, (2,), "free_state")):
        _like(t, i32, shape, dev, name)
    st = _handle_on(dev, stream)
    if st is None:
        with _made_current(dev, stream):
            return cache_plan(ctx_lens, new_lens, block_table, held, free_ring, free_state, page_size=page_size,
                              num_tokens=num_tokens, held_out=held_out, free_out=free_out, out=out)
    if out is None:
        # one allocation, cut up on 16-byte boundaries
        T, pb = num_tokens, -(B + 1) % 4
        parts = torch.empty(2 * (B + T) + 20, dtype=i32, device=dev).split_with_sizes(
            (1, 3, B + 1, pb, B, -B % 4, T, -T % 4, T, 15 - pb - -B % 4 - -T % 4))
        cu_q, kv_lens, slots, positions, refused = parts[2], parts[4], parts[6], parts[8], parts[0]
        held_out = torch.empty(B, dtype=i32, device=dev) if held_out is None else held_out
        free_out = torch.empty(2, dtype=i32, device=dev) if free_out is None else free_out
    else:
        cu_q, kv_lens, slots, positions, refused = out[:5]
        held_out = out.held if held_out is None else held_out
        free_out = out.free_state if free_out is None else free_out
        for t, n, name in ((cu_q, B + 1, "cu_q"), (kv_lens, B, "kv_lens"), (slots, num_tokens, "slots"),
                           (positions, num_tokens, "positions"), (refused, 1, "refused")):
            _like(t, i32, (n,), dev, name)
    _like(held_out, i32, (B,), dev, "held_out")
    _like(free_out, i32, (2,), dev, "free_out")
    args = PlanArgs(ctypes.sizeof(PlanArgs), B, num_tokens, W, page_size, N, ctx_lens.data_ptr(), new_lens.data_ptr(),
                    block_table.data_ptr(), held.data_ptr(), held_out.data_ptr(), free_ring.data_ptr(),
                    free_state.data_ptr(), free_out.data_ptr(), cu_q.data_ptr(), kv_lens.data_ptr(), slots.data_ptr(),
                    positions.data_ptr(), refused.data_ptr())
    _check(lib().moe_mxfp4_cache_plan(ctypes.byref(args), st), "moe_mxfp4_cache_plan")
    return CachePlan(cu_q, kv_lens, slots, positions, refused, held_out, free_out)


def qk_norm_rope(q, k, v, positions, inv_freq, *, q_weight=None, k_weight=None, eps: float = 1e-6,
                 interleaved: bool = False, cache: KvCache | None = None, slots=None, q_out=None, k_out=None,
                 stream=None):
    """Per-head norms, rotation and cache write (moe_mxfp4_qk_norm_rope) -> (q_out, k_out).

    q [T, heads, D], k, v [T, kv_heads, D]: bf16 CUDA, tokens at any stride
    that is a multiple of 8.  inv_freq: float64 [rot_dim/2].  With ``cache``
    the key and value go to ``slots`` (int32 [T]) and k_out is None unless
    given; without one, v and slots are ignored.
    """
    import torch
    dev = q.device
    T, H, D = q.shape
    HK = k.shape[1]
    qs, ks = _heads(q, D, dev, "q"), _heads(k, D, dev, "k")
    vs, v_ptr, slots_ptr, cache_ref = 0, None, None, None
    if k.shape[0] != T:
        raise ValueError(f"k: {k.shape[0]} tokens, q has {T}")
    _like(positions, torch.int32, (T,), dev, "positions")
    _like(inv_freq, torch.float64, (inv_freq.numel(),), dev, "inv_freq")
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None:
            _like(w, torch.bfloat16, (D,), dev, name)
    if cache is not None:
        vs = _heads(v, D, dev, "v")
        if v.shape != k.shape or slots is None:
            raise ValueError("a cache write needs v of k's shape, and slots")
        _like(slots, torch.int32, (T,), dev, "slots")
        if cache.device != dev:
            raise ValueError(f"cache on {cache.device}, q on {dev}")
        v_ptr, slots_ptr, cache_ref = v.data_ptr(), slots.data_ptr(), cache.ref
    st = _handle_on(dev, stream)
    if st is None:
        with _made_current(dev, stream):
            return qk_norm_rope(q, k, v, positions, inv_freq, q_weight=q_weight, k_weight=k_weight, eps=eps,
                                interleaved=interleaved, cache=cache, slots=slots, q_out=q_out, k_out=k_out)
    if q_out is None:
        q_out = q.new_empty((T, H, D))
    else:
        _like(q_out, torch.bfloat16, (T, H, D), dev, "q_out")
    if k_out is not None:
        _like(k_out, torch.bfloat16, (T, HK, D), dev, "k_out")
    elif cache is None:
        k_out = q.new_empty((T, HK, D))
    args = RopeArgs(ctypes.sizeof(RopeArgs), T, H, HK, D, 2 * inv_freq.numel(), int(interleaved), eps, qs, ks, vs,
                    q.data_ptr(), k.data_ptr(), v_ptr, None if q_weight is None else q_weight.data_ptr(),
                    None if k_weight is None else k_weight.data_ptr(), inv_freq.data_ptr(), positions.data_ptr(),
                    slots_ptr, q_out.data_ptr(), None if k_out is None else k_out.data_ptr())
    _check(lib().moe_mxfp4_qk_norm_rope(ctypes.byref(args), cache_ref, st), "moe_mxfp4_qk_norm_rope")
    return q_out, k_out


def kv_read(cache: KvCache, slots, stream=None):
    """The values a cache holds at ``slots`` (int32 [n]): (k, v) bf16 [n, kv_heads, D] (moe_mxfp4_kv_read)."""
    import torch
    n, dev = slots.numel(), cache.device
    _like(slots, torch.int32, (n,), dev, "slots")
    st = _handle_on(dev, stream)
    if st is None:
        with _made_current(dev, stream):
            return kv_read(cache, slots)
    k, v = torch.empty((2, n, cache.kv_heads, cache.head_dim), dtype=torch.bfloat16, device=dev).unbind()
    _check(lib().moe_mxfp4_kv_read(cache.ref, slots.data_ptr(), n, k.data_ptr(), v.data_ptr(), st), "moe_mxfp4_kv_read")
    return k, v


def attention(q, cache: KvCache, block_table, cu_q, kv_lens, *, max_q: int, max_kv: int, scale: float | None = None,
              causal: bool = True, window: int = 0, sinks: int = 0, out=None, workspace=None, stream=None):
    """Attention of packed rows over a paged cache (moe_mxfp4_attention) -> out [T, heads, D] bf16.

    q bf16 [T, heads, D]; block_table int32 [B, max_blocks], cu_q int32 [B+1],
    kv_lens int32 [B], all CUDA.  ``max_q`` and ``max_kv``: the longest
    sequences the caller expects (longer ones are slower, not wrong).
    ``scale``: 1/sqrt(D) by default.  ``window`` > 0: only the last ``window``
    keys, and the first ``sinks``, are visible.  Rows of ``out`` past cu_q[B]
    are not written (unspecified where ``out`` is made here).
    """
    import torch
    dev = q.device
    T, H, D = q.shape
    B, W = block_table.shape
    qs = _heads(q, D, dev, "q")
    _like(block_table, torch.int32, (B, W), dev, "block_table")
    _like(cu_q, torch.int32, (B + 1,), dev, "cu_q")
    _like(kv_lens, torch.int32, (B,), dev, "kv_lens")
    if cache.head_dim != D or cache.device != dev:
        raise ValueError(f"q has heads of {D} on {dev}, the cache of {cache.head_dim} on {cache.device}")
    st = _handle_on(dev, stream)
    if st is None:
        with _made_current(dev, stream):
            return attention(q, cache, block_table, cu_q, kv_lens, max_q=max_q, max_kv=max_kv, scale=scale, causal=causal,
                             window=window, sinks=sinks, out=out, workspace=workspace)
    if out is None:
        out, os_ = q.new_empty((T, H, D)), H * D
    else:
        if out.shape != q.shape:
            raise ValueError(f"out: expected {tuple(q.shape)}, got {tuple(out.shape)}")
        os_ = _heads(out, D, dev, "out")
    args = ctypes.byref(AttnArgs(ctypes.sizeof(AttnArgs), B, T, H, max_q, max_kv, W, int(causal), window, sinks,
                                 D ** -0.5 if scale is None else scale, qs, os_, q.data_ptr(), out.data_ptr(),
                                 block_table.data_ptr(), cu_q.data_ptr(), kv_lens.data_ptr()))
    L = lib()
    if workspace is None:
        need = L.moe_mxfp4_attention_workspace_bytes(args, cache.ref)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace: expected a contiguous tensor on {dev}, got strides {workspace.stride()} on "
                         f"{workspace.device}")
    if workspace is None:
        status = L.moe_mxfp4_attention(args, cache.ref, None, 0, st)
    else:
        status = L.moe_mxfp4_attention(args, cache.ref, workspace.data_ptr(),
                                       workspace.numel() * workspace.element_size(), st)
    _check(status, "moe_mxfp4_attention")
    return out


def attention_workspace_bytes(cache: KvCache, num_tokens: int, heads: int, batch: int, *, max_q: int, max_kv: int,
                              window: int = 0, sinks: int = 0) -> int:
    """Bytes of workspace an ``attention`` call of these sizes needs (0: none)."""
    row = heads * cache.head_dim
    args = AttnArgs(ctypes.sizeof(AttnArgs), batch, num_tokens, heads, max_q, max_kv, 1, 1, window, sinks, 1.0, row, row)
    return lib().moe_mxfp4_attention_workspace_bytes(ctypes.byref(args), ctypes.byref(cache.struct))


PROBE_STREAM, PROBE_MFMA_BF16, PROBE_MFMA_FP8_FP4, PROBE_MFMA_FP4_FP4 = 0, 1, 2, 3
# the same instructions on random operands that change every MFMA
PROBE_MFMA_BF16_RANDOM, PROBE_MFMA_FP8_FP4_RANDOM, PROBE_MFMA_FP4_FP4_RANDOM = 4, 5, 6


def probe(kind: int, src=None, reps: int = 0, sink=None, stream=None) -> float:
    """Launch one measurement probe (moe_mxfp4_probe); returns the bytes or
    flops it does.  ``src``: a CUDA tensor to read (kind 0)."""
    import torch
    if sink is None:
        sink = torch.zeros(1, dtype=torch.int32, device="cuda")
    work = ctypes.c_double()
    nbytes = 0 if src is None else src.numel() * src.element_size()
    _check(lib().moe_mxfp4_probe(kind, _ptr(src), nbytes, reps, _ptr(sink), ctypes.byref(work), _stream(stream)),
           "moe_mxfp4_probe")
    return work.value
