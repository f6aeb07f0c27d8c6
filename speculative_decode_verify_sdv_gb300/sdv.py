"""Thin Python binding of libsdv (include/sdv.h): argument marshalling only.

Every function has the name of the C entry point it calls and takes torch
tensors where the C function takes device pointers.  All arithmetic happens
in the library's CUDA kernels; there is no Python or CPU fallback: if the
shared library is missing or a GPU is absent the calls raise.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsdv.so")

SDV_OK, SDV_ERR_INVALID_ARG, SDV_ERR_UNSUPPORTED, SDV_ERR_CUDA, SDV_ERR_TIMEOUT, SDV_ERR_WORKSPACE = range(6)
SDV_Q8, SDV_Q4, SDV_F4 = 8, 4, 2
SDV_F16, SDV_BF16 = 16, 17
SDV_OP_QLINEAR, SDV_OP_QLINEAR_SWIGLU, SDV_OP_VERIFY_HEAD, SDV_OP_MOE, SDV_OP_VERIFY_SAMPLE = 1, 2, 3, 4, 5

EXPORTED = (
    "sdv_quantize_block32", "sdv_qlinear", "sdv_qlinear_swiglu", "sdv_verify_head",
    "sdv_greedy_accept", "sdv_moe_gather_qmm", "sdv_workspace_bytes", "sdv_workspace_init",
    "sdv_last_device_status", "sdv_device_status", "sdv_noalloc_device_status", "sdv_status_string", "sdv_version", "sdv_launch_count", "sdv_verify_head_noalloc", "sdv_set_gemm_path",
    "sdv_moe_route", "sdv_verify_sample", "sdv_tree_accept", "sdv_debug_fault",
    "sdv_ngram_create", "sdv_ngram_destroy", "sdv_ngram_append", "sdv_ngram_propose",
    "sdv_kv_append", "sdv_paged_attn", "sdv_paged_attn_workspace_bytes", "sdv_linear_attn",
    "sdv_linear_attn_workspace_bytes",
)


class SdvError(RuntimeError):
    def __init__(self, fn: str, status: int, text: str):
        super().__init__(f"{fn} failed: {text} ({status})")
        self.status = status


class sdv_qweight(ctypes.Structure):
    _fields_ = [("qtype", ctypes.c_int32), ("n", ctypes.c_int32), ("k", ctypes.c_int32),
                ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class sdv_kvcache(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("n_pages", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("dim", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("table", ctypes.c_void_p)]


_lib = None


def load() -> ctypes.CDLL:
    """Load libsdv.so (built in-tree by ``build.build()``); raise if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libsdv.so not found at {LIB_PATH}; run __graft_entry__.build() first")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    i64, f32 = ctypes.c_int64, ctypes.c_float
    kvc = ctypes.POINTER(sdv_kvcache)
    qw = ctypes.POINTER(sdv_qweight)
    sig = {
        "sdv_quantize_block32": ([vp, i32, i32, i32, vp, vp, vp], i32),
        "sdv_qlinear": ([qw, vp, i32, vp, vp, sz, vp], i32),
        "sdv_qlinear_swiglu": ([qw, qw, vp, i32, vp, vp, sz, vp], i32),
        "sdv_verify_head": ([qw, vp, i32, vp, i32, vp, vp, vp, vp, vp, sz, vp], i32),
        "sdv_verify_head_noalloc": ([qw, vp, i32, vp, i32, vp, vp, vp, vp, vp], i32),
        "sdv_verify_sample": ([qw, vp, i32, vp, i32, ctypes.c_float, ctypes.c_uint64, ctypes.c_uint64, vp, vp, vp,
                               vp, vp, sz, vp], i32),
        "sdv_greedy_accept": ([vp, i32, vp, i32, vp, vp, vp], i32),
        "sdv_tree_accept": ([vp, i32, vp, vp, vp, vp, vp, vp], i32),
        "sdv_moe_gather_qmm": ([qw, qw, qw, i32, i32, i32, i32, vp, vp, i32, vp, vp, vp, vp, sz, vp], i32),
        "sdv_moe_route": ([vp, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp], i32),
        "sdv_workspace_bytes": ([i32, i32, i32, i32, i32, i32], sz),
        "sdv_workspace_init": ([vp, sz, vp], i32),
        "sdv_last_device_status": ([vp, vp], i32),
        "sdv_device_status": ([vp, vp], i32),
        "sdv_noalloc_device_status": ([vp], i32),
        "sdv_status_string": ([i32], ctypes.c_char_p),
        "sdv_version": ([], i32),
        "sdv_launch_count": ([], ctypes.c_uint64),
        "sdv_set_gemm_path": ([i32], i32),
        "sdv_debug_fault": ([i32, ctypes.c_uint64], i32),
        "sdv_ngram_create": ([i32, ctypes.POINTER(vp)], i32),
        "sdv_ngram_destroy": ([vp], i32),
        "sdv_ngram_append": ([vp, vp, i32], i32),
        "sdv_ngram_propose": ([vp, i32, vp, ctypes.POINTER(i32)], i32),
        "sdv_kv_append": ([kvc, vp, vp, i64, i64, i32, i32, vp, vp, vp, vp], i32),
        "sdv_paged_attn": ([kvc, vp, i64, i32, i32, i32, vp, vp, vp, f32, vp, vp, vp, sz, vp], i32),
        "sdv_paged_attn_workspace_bytes": ([i32, i32, i32, i32, i32], sz),
        "sdv_linear_attn": ([i32, vp, vp, vp, i64, i64, i64, vp, i32, f32, i32, i32, i32, i32, i32, i32, vp, vp, vp,
                             vp, vp, sz, vp], i32),
        "sdv_linear_attn_workspace_bytes": ([i32, i32, i32, i32, i32], sz),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    _lib = lib
    return lib


def _check(fn: str, status: int) -> None:
    if status != SDV_OK:
        raise SdvError(fn, status, load().sdv_status_string(status).decode())


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return ctypes.c_void_p(t.data_ptr())


def _want(t, dtype, name):
    if t is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


class QWeight:
    """A per-block-32 quantised weight: codes (int8 [n, k] or uint8 [n, k/2]),
    fp16 scales [n, k/32], on the GPU."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, bits: int, n: int, k: int):
        self.codes, self.scales, self.bits, self.n, self.k = codes, scales, bits, n, k

    def c(self) -> sdv_qweight:
        return sdv_qweight(self.bits, self.n, self.k, _ptr(self.codes), _ptr(self.scales))


def sdv_launch_count() -> int:
    """Kernels the library has launched in this process (see the header)."""
    return int(load().sdv_launch_count())


def sdv_version() -> int:
    return int(load().sdv_version())


SDV_PATH_AUTO, SDV_PATH_MMA_SYNC, SDV_PATH_TCGEN05, SDV_PATH_GEMV = 0, 1, 2, 3


def sdv_set_gemm_path(path: int) -> int:
    """Select the GEMM implementation (0 auto, 1 mma.sync, 2 tcgen05, 3 CUDA-core GEMV for S <= 2);
    returns the previous one."""
    prev = int(load().sdv_set_gemm_path(path))
    if prev < 0:
        raise ValueError(f"invalid GEMM path {path}")
    return prev


def sdv_debug_fault(withhold_stage: int, wait_limit_ns: int) -> None:
    """Timeout-path test hook: withhold one weight stage of every tcgen05 launch
    and shorten the bounded waits (-1, 0 switches it off)."""
    _check("sdv_debug_fault", load().sdv_debug_fault(withhold_stage, wait_limit_ns))


def sdv_status_string(status: int) -> str:
    return load().sdv_status_string(status).decode()


def sdv_workspace_bytes(op: int, n: int, k: int, S: int, E: int = 0, top_k: int = 0) -> int:
    return int(load().sdv_workspace_bytes(op, n, k, S, E, top_k))


def sdv_workspace_init(ws: torch.Tensor, stream=None) -> None:
    _check("sdv_workspace_init", load().sdv_workspace_init(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def sdv_last_device_status(ws: torch.Tensor, stream=None) -> int:
    """Synchronise and return (and clear) the workspace's device status."""
    return int(load().sdv_last_device_status(_ptr(ws), _stream(stream)))


def sdv_device_status(ws: torch.Tensor, stream=None) -> int:
    """The same as ``sdv_last_device_status`` (the earlier name)."""
    return int(load().sdv_device_status(_ptr(ws), _stream(stream)))


def sdv_noalloc_device_status(stream=None) -> int:
    """Synchronise and return (and clear) the status of the no-workspace head's fixed scratch."""
    return int(load().sdv_noalloc_device_status(_stream(stream)))


def sdv_quantize_block32(w: torch.Tensor, bits: int, codes: torch.Tensor, scales: torch.Tensor,
                         stream=None) -> None:
    _want(w, torch.float32, "w")
    _want(scales, torch.float16, "scales")
    n, k = w.shape
    _check("sdv_quantize_block32", load().sdv_quantize_block32(
        _ptr(w), n, k, bits, _ptr(codes), _ptr(scales), _stream(stream)))


def sdv_qlinear(w: QWeight, x: torch.Tensor, S: int, y: torch.Tensor, ws: torch.Tensor, stream=None) -> None:
    _want(x, torch.float16, "x")
    _want(y, torch.float32, "y")
    cw = w.c()
    _check("sdv_qlinear", load().sdv_qlinear(ctypes.byref(cw), _ptr(x), S, _ptr(y), _ptr(ws),
                                             ws.numel() * ws.element_size(), _stream(stream)))


def sdv_qlinear_swiglu(gate: QWeight, up: QWeight, x: torch.Tensor, S: int, h: torch.Tensor,
                       ws: torch.Tensor, stream=None) -> None:
    _want(x, torch.float16, "x")
    _want(h, torch.float16, "h")
    cg, cu = gate.c(), up.c()
    _check("sdv_qlinear_swiglu", load().sdv_qlinear_swiglu(
        ctypes.byref(cg), ctypes.byref(cu), _ptr(x), S, _ptr(h), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def sdv_verify_head(head: QWeight, x: torch.Tensor, S: int, drafts, n_valid: int, logits,
                    argmax: torch.Tensor, accepted: torch.Tensor, next_a0: torch.Tensor,
                    ws: torch.Tensor, stream=None) -> None:
    _want(x, torch.float16, "x")
    _want(drafts, torch.int32, "drafts")
    _want(logits, torch.float32, "logits")
    for t, nm in ((argmax, "argmax"), (accepted, "accepted"), (next_a0, "next_a0")):
        _want(t, torch.int32, nm)
    cw = head.c()
    _check("sdv_verify_head", load().sdv_verify_head(
        ctypes.byref(cw), _ptr(x), S, _ptr(drafts), n_valid, _ptr(logits), _ptr(argmax),
        _ptr(accepted), _ptr(next_a0), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def sdv_verify_sample(head: QWeight, x: torch.Tensor, S: int, drafts, n_valid: int, temperature: float,
                      seed: int, counter: int, logits, samples: torch.Tensor, accepted: torch.Tensor,
                      next_token: torch.Tensor, ws: torch.Tensor, stream=None) -> None:
    _want(x, torch.float16, "x")
    _want(drafts, torch.int32, "drafts")
    _want(logits, torch.float32, "logits")
    for t, nm in ((samples, "samples"), (accepted, "accepted"), (next_token, "next_token")):
        _want(t, torch.int32, nm)
    cw = head.c()
    _check("sdv_verify_sample", load().sdv_verify_sample(
        ctypes.byref(cw), _ptr(x), S, _ptr(drafts), n_valid, float(temperature), seed % 2**64, counter % 2**64,
        _ptr(logits), _ptr(samples), _ptr(accepted), _ptr(next_token), _ptr(ws), ws.numel() * ws.element_size(),
        _stream(stream)))


def sdv_verify_head_noalloc(head: QWeight, x: torch.Tensor, S: int, drafts, n_valid: int, logits,
                            argmax: torch.Tensor, accepted: torch.Tensor, next_a0: torch.Tensor,
                            stream=None) -> None:
    """sdv_verify_head with the library's own fixed device scratch (no workspace)."""
    _want(x, torch.float16, "x")
    _want(drafts, torch.int32, "drafts")
    _want(logits, torch.float32, "logits")
    for t, nm in ((argmax, "argmax"), (accepted, "accepted"), (next_a0, "next_a0")):
        _want(t, torch.int32, nm)
    cw = head.c()
    _check("sdv_verify_head_noalloc", load().sdv_verify_head_noalloc(
        ctypes.byref(cw), _ptr(x), S, _ptr(drafts), n_valid, _ptr(logits), _ptr(argmax),
        _ptr(accepted), _ptr(next_a0), _stream(stream)))


def sdv_tree_accept(argmax: torch.Tensor, S: int, tokens, parent, path, accepted: torch.Tensor,
                    next_a0: torch.Tensor, stream=None) -> None:
    for t, nm in ((argmax, "argmax"), (tokens, "tokens"), (parent, "parent"), (path, "path"),
                  (accepted, "accepted"), (next_a0, "next_a0")):
        _want(t, torch.int32, nm)
    _check("sdv_tree_accept", load().sdv_tree_accept(
        _ptr(argmax), S, _ptr(tokens), _ptr(parent), _ptr(path), _ptr(accepted), _ptr(next_a0), _stream(stream)))


def sdv_greedy_accept(argmax: torch.Tensor, S: int, drafts, n_valid: int, accepted: torch.Tensor,
                      next_a0: torch.Tensor, stream=None) -> None:
    for t, nm in ((argmax, "argmax"), (drafts, "drafts"), (accepted, "accepted"), (next_a0, "next_a0")):
        _want(t, torch.int32, nm)
    _check("sdv_greedy_accept", load().sdv_greedy_accept(
        _ptr(argmax), S, _ptr(drafts), n_valid, _ptr(accepted), _ptr(next_a0), _stream(stream)))


def sdv_moe_gather_qmm(gate: QWeight, up: QWeight, down: QWeight, E: int, I: int, H: int, top_k: int,
                       x: torch.Tensor, router_logits: torch.Tensor, S: int, out: torch.Tensor,
                       topk_ids, topk_w, ws: torch.Tensor, stream=None) -> None:
    _want(x, torch.float16, "x")
    _want(router_logits, torch.float32, "router_logits")
    _want(out, torch.float32, "out")
    cg, cu, cd = gate.c(), up.c(), down.c()
    _check("sdv_moe_gather_qmm", load().sdv_moe_gather_qmm(
        ctypes.byref(cg), ctypes.byref(cu), ctypes.byref(cd), E, I, H, top_k, _ptr(x),
        _ptr(router_logits), S, _ptr(out), _ptr(topk_ids), _ptr(topk_w), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def sdv_moe_route(router_logits: torch.Tensor, S: int, E: int, top_k: int, ids: torch.Tensor,
                  weights: torch.Tensor, offsets: torch.Tensor, pair_rows: torch.Tensor,
                  n_hit: torch.Tensor, hit: torch.Tensor, stream=None) -> None:
    _want(router_logits, torch.float32, "router_logits")
    _want(weights, torch.float32, "weights")
    for t, nm in ((ids, "ids"), (offsets, "offsets"), (pair_rows, "pair_rows"), (n_hit, "n_hit"), (hit, "hit")):
        _want(t, torch.int32, nm)
    _check("sdv_moe_route", load().sdv_moe_route(
        _ptr(router_logits), S, E, top_k, _ptr(ids), _ptr(weights), _ptr(offsets), _ptr(pair_rows),
        _ptr(n_hit), _ptr(hit), _stream(stream)))


# ---- token mixing: paged cache, its attention, linear attention ------------------

_DTYPES = {torch.float16: SDV_F16, torch.bfloat16: SDV_BF16}


def _addr(t, dtype, name, shape=None):
    """Device address of a contiguous CUDA tensor (None for None)."""
    if t is None:
        return None
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _rows(t, dtype, name, B, T, heads, dim):
    """(address, token stride) of [B, T, heads, dim] rows: heads and dim contiguous,
    the tokens of all sequences at one stride (the slices of a fused projection)."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.shape != (B, T, heads, dim):
        raise ValueError(f"{name} must be {(B, T, heads, dim)}, got {tuple(t.shape)}")
    sb, st, sh, sd = t.stride()
    if T == 1:
        st = sb if B > 1 else heads * dim
    if sd != 1 or (heads > 1 and sh != dim) or (B > 1 and sb != T * st):
        raise ValueError(f"{name}: heads and dim must be contiguous and its tokens evenly strided")
    return t.data_ptr(), st


def _kvcache(k_pages, v_pages, table):
    dt = k_pages.dtype
    if dt not in _DTYPES:
        raise TypeError(f"a cache is float16 or bfloat16, got {dt}")
    if k_pages.dim() != 4 or table.dim() != 2:
        raise ValueError("k_pages and v_pages are [n_pages, heads, page_size, dim], table is [B, max_pages]")
    n, heads, page, dim = k_pages.shape
    return sdv_kvcache(_DTYPES[dt], n, heads, page, dim, table.shape[1], _addr(k_pages, dt, "k_pages"),
                       _addr(v_pages, dt, "v_pages", k_pages.shape), _addr(table, torch.int32, "table"))


# the current stream's handle without building a Stream object (a third of a small call's host time)
_current_raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(stream, device):
    if stream is not None:
        return stream.cuda_stream
    if _current_raw is not None and device.index is not None:
        return _current_raw(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def sdv_paged_attn_workspace_bytes(B: int, S: int, Hq: int, heads: int, dim: int) -> int:
    return int(load().sdv_paged_attn_workspace_bytes(B, S, Hq, heads, dim))


def sdv_linear_attn_workspace_bytes(B: int, T: int, H: int, Dk: int, Dv: int) -> int:
    return int(load().sdv_linear_attn_workspace_bytes(B, T, H, Dk, Dv))


def sdv_kv_append(k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                  table: torch.Tensor, ctx: torch.Tensor, n_rows, ws, stream=None) -> None:
    """Rows k, v [B, T, heads, dim] into the cache behind ctx [B]; n_rows [B] or
    None (all T); ws: a workspace for the device status, or None."""
    c = _kvcache(k_pages, v_pages, table)
    B, T = k.shape[:2]
    i32 = torch.int32
    dt = k_pages.dtype
    ka, ks = _rows(k, dt, "k", B, T, c.heads, c.dim)
    va, vs = _rows(v, dt, "v", B, T, c.heads, c.dim)
    if table.shape[0] != B:
        raise ValueError(f"table must have {B} rows, got {table.shape[0]}")
    if ws is not None and ws.numel() * ws.element_size() < 256:
        raise ValueError("ws must hold at least 256 bytes")
    st = load().sdv_kv_append(ctypes.byref(c), ka, va, ks, vs, B, T, _addr(ctx, i32, "ctx", (B,)),
                              _addr(n_rows, i32, "n_rows", (B,)), None if ws is None else _addr(ws, ws.dtype, "ws"),
                              _raw_stream(stream, k.device))
    if st:
        _check("sdv_kv_append", st)


def sdv_paged_attn(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, table: torch.Tensor,
                   ctx: torch.Tensor, n_rows, mask, scale: float, out: torch.Tensor, lse, ws: torch.Tensor,
                   stream=None) -> None:
    """Attention of the window rows q [B, S, Hq, dim] over the cache; mask: int32
    [B, S] visibility words or None (causal); lse: fp32 [B, S, Hq] or None."""
    c = _kvcache(k_pages, v_pages, table)
    B, S, hq = q.shape[:3]
    i32 = torch.int32
    dt = k_pages.dtype
    qa, qs = _rows(q, dt, "q", B, S, hq, c.dim)
    if table.shape[0] != B:
        raise ValueError(f"table must have {B} rows, got {table.shape[0]}")
    st = load().sdv_paged_attn(
        ctypes.byref(c), qa, qs, B, S, hq, _addr(ctx, i32, "ctx", (B,)), _addr(n_rows, i32, "n_rows", (B,)),
        _addr(mask, i32, "mask", (B, S)), scale, _addr(out, dt, "out", q.shape),
        _addr(lse, torch.float32, "lse", (B, S, hq)), _addr(ws, ws.dtype, "ws"), ws.nbytes,
        _raw_stream(stream, q.device))
    if st:
        _check("sdv_paged_attn", st)


def sdv_linear_attn(q, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, scale: float, n_tokens,
                    state_in, state_out, o, ws: torch.Tensor, stream=None) -> None:
    """Linear attention with a decay per head: q, k [B, T, Hqk, Dk], v [B, T, H, Dv],
    log_decay fp32 [B, T, H] or [H], states fp32 [B, H, Dk, Dv], o [B, T, H, Dv];
    n_tokens int32 [B], state_in, state_out, o (and then q) may be None."""
    if k.dtype not in _DTYPES:
        raise TypeError(f"q, k and v are float16 or bfloat16, got {k.dtype}")
    B, T, hqk, dk = k.shape
    H, dv = v.shape[2:]
    dt, f32 = k.dtype, torch.float32
    ka, ks = _rows(k, dt, "k", B, T, hqk, dk)
    va, vs = _rows(v, dt, "v", B, T, H, dv)
    qa, qs = (None, 0) if q is None else _rows(q, dt, "q", B, T, hqk, dk)
    per_token = log_decay.dim() == 3
    state = (B, H, dk, dv)
    st = load().sdv_linear_attn(
        _DTYPES[dt], qa, ka, va, qs, ks, vs, _addr(log_decay, f32, "log_decay", (B, T, H) if per_token else (H,)),
        1 if per_token else 0, scale, B, T, H, hqk, dk, dv, _addr(n_tokens, torch.int32, "n_tokens", (B,)),
        _addr(state_in, f32, "state_in", state), _addr(state_out, f32, "state_out", state),
        _addr(o, dt, "o", (B, T, H, dv)), _addr(ws, ws.dtype, "ws"), ws.nbytes,
        _raw_stream(stream, k.device))
    if st:
        _check("sdv_linear_attn", st)


# ---- host n-gram drafter (host pointers; no GPU involved) -------------------------

def sdv_ngram_create(m: int) -> int:
    """A native drafter of order m; returns its opaque handle."""
    h = ctypes.c_void_p()
    _check("sdv_ngram_create", load().sdv_ngram_create(m, ctypes.byref(h)))
    return h.value


def sdv_ngram_destroy(handle: int) -> None:
    _check("sdv_ngram_destroy", load().sdv_ngram_destroy(ctypes.c_void_p(handle)))


def sdv_ngram_append(handle: int, tokens) -> None:
    arr = (ctypes.c_int32 * len(tokens))(*[int(t) for t in tokens])
    _check("sdv_ngram_append", load().sdv_ngram_append(ctypes.c_void_p(handle), arr, len(tokens)))


def sdv_ngram_propose(handle: int, k: int) -> list[int]:
    """Up to k drafts continuing the stream's last m tokens (empty when none)."""
    buf = (ctypes.c_int32 * max(k, 1))()
    count = ctypes.c_int32(0)
    _check("sdv_ngram_propose", load().sdv_ngram_propose(ctypes.c_void_p(handle), k, buf, ctypes.byref(count)))
    return list(buf[:count.value])


# ---- small allocation helpers (torch owns the memory) ---------------------------

def workspace(op: int, n: int, k: int, S: int, E: int = 0, top_k: int = 0, device="cuda") -> torch.Tensor:
    """A zero-filled workspace of the size the operation needs."""
    nbytes = max(sdv_workspace_bytes(op, n, k, S, E, top_k), 256)
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


def quantize(w: torch.Tensor, bits: int) -> QWeight:
    """Quantise an fp32 [n, k] CUDA tensor with sdv_quantize_block32."""
    n, k = w.shape
    codes = torch.empty((n, k if bits == 8 else k // 2), dtype=torch.int8 if bits == 8 else torch.uint8,
                        device=w.device)
    scales = torch.empty((n, k // 32), dtype=torch.float16, device=w.device)
    sdv_quantize_block32(w.contiguous(), bits, codes, scales)
    return QWeight(codes, scales, bits, n, k)


def paged_attn_workspace(q: torch.Tensor, k_pages: torch.Tensor, table: torch.Tensor) -> torch.Tensor:
    """A zero-filled workspace for sdv_paged_attn calls of up to S rows of this shape (q [B, S, Hq, dim])."""
    B, S, hq, dim = q.shape
    nbytes = max(sdv_paged_attn_workspace_bytes(B, S, hq, k_pages.shape[1], dim), 256)
    return torch.zeros(nbytes, dtype=torch.uint8, device=q.device)


def linear_attn_workspace(k: torch.Tensor, v: torch.Tensor) -> torch.Tensor:
    """A zero-filled workspace for sdv_linear_attn calls of this shape and of fewer tokens or sequences
    (k [B, T, Hqk, Dk], v [B, T, H, Dv])."""
    B, T = k.shape[:2]
    nbytes = max(sdv_linear_attn_workspace_bytes(B, T, v.shape[2], k.shape[3], v.shape[3]), 256)
    return torch.zeros(nbytes, dtype=torch.uint8, device=k.device)
