"""Python binding of the C ABI: argument marshalling over torch CUDA tensors.

Every function here checks shapes/dtypes, passes raw device pointers and the
current torch stream to libtokengate.so, and raises TokenGateError on a non-OK
status. All arithmetic happens in the CUDA kernels.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
from typing import Optional, Sequence

import torch

from . import _lib
from ._lib import TokenGateError, check

TG_F32, TG_BF16, TG_I8, TG_E4M3 = 0, 1, 2, 3
_DT = {torch.float32: TG_F32, torch.bfloat16: TG_BF16}
_CODE_DT = {torch.int8: TG_I8, torch.float8_e4m3fn: TG_E4M3}


def _stream(stream=None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(s.cuda_stream)


def _cuda(t: torch.Tensor, name: str, dtype=None) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TokenGateError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise TokenGateError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TokenGateError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _numel(t: torch.Tensor, n: int, name: str) -> None:
    if t.numel() != n:
        raise TokenGateError(f"{name} must have {n} elements, got {t.numel()}")


def _shape(t: torch.Tensor, shape, name: str, dtype=None) -> None:
    if t.shape != shape:
        raise TokenGateError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TokenGateError(f"{name} must be {dtype}, got {t.dtype}")


_CURRENT = contextlib.nullcontext()


def _on(stream):
    """Where a call on a given stream allocates: with that stream current, so that the
    allocator hands out blocks whose earlier use is over when the call's kernels run. (A block
    freed on the current stream may still be in use by kernels queued there.)"""
    if stream is None:
        return _CURRENT
    if not isinstance(stream, torch.cuda.Stream):   # anything with a cuda_stream is a stream here
        stream = torch.cuda.ExternalStream(stream.cuda_stream)
    return torch.cuda.stream(stream)


def _hand_over(stream, *tensors) -> None:
    """Outputs that were allocated with `stream` current and go to a caller who works on the
    current stream: their blocks are not given away while that one still uses them."""
    if stream is not None:
        for t in tensors:
            t.record_stream(torch.cuda.current_stream(t.device))


def abi_version() -> int:
    return _lib.load().tg_abi_version()


def gate_score(x: torch.Tensor, w1: torch.Tensor, b1: torch.Tensor, w2: torch.Tensor, b2: float,
               out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """s = b2 + w2 . GELU(W1 x + b1) per token. x [N, d], w1 [h, d] (same dtype)."""
    n, d = x.shape
    h = w1.shape[0]
    if w1.shape != (h, d) or w1.dtype != x.dtype or x.dtype not in _DT:
        raise TokenGateError("gate_score: x [N,d] and w1 [h,d] must share a dtype (f32/bf16)")
    _numel(b1, h, "b1")
    _numel(w2, h, "w2")
    new = ()
    if out is None:
        with _on(stream):
            out = torch.empty(n, dtype=torch.float32, device=x.device)
        new = (out,)
    _numel(out, n, "scores")
    st = _lib.load().tg_gate_score(_cuda(x, "x"), _DT[x.dtype], n, d, _cuda(w1, "w1"),
                                   _cuda(b1, "b1", torch.float32), _cuda(w2, "w2", torch.float32),
                                   float(b2), h, _cuda(out, "scores", torch.float32), _stream(stream))
    check(st, "tg_gate_score")
    _hand_over(stream, *new)
    return out


def select_topk(scores: torch.Tensor, cu_seqlens: torch.Tensor, doc_begin: torch.Tensor,
                doc_end: torch.Tensor, k_doc: torch.Tensor, total_kept: int, max_seqlen: int,
                kept_idx: Optional[torch.Tensor] = None, kept_scores: Optional[torch.Tensor] = None,
                cu_kept: Optional[torch.Tensor] = None, want_scores: bool = True,
                kept_pos: Optional[torch.Tensor] = None, want_pos: bool = False, stream=None):
    """Returns (kept_idx int32 [total_kept], kept_scores f32 [total_kept] or None,
    cu_kept int32 [B+1]); with want_pos (or kept_pos given) also kept_pos int32
    [total_kept], the kept rows' positions within their sequences, as a 4th item."""
    B = doc_begin.numel()
    dev = scores.device
    total_kept = int(total_kept)
    _numel(cu_seqlens, B + 1, "cu_seqlens")
    _numel(doc_end, B, "doc_end")
    _numel(k_doc, B, "k_doc")
    new = []

    def empty(n, dtype):
        with _on(stream):
            new.append(torch.empty(n, dtype=dtype, device=dev))
        return new[-1]
    if kept_idx is None:
        kept_idx = empty(total_kept, torch.int32)
    if kept_scores is None and want_scores:
        kept_scores = empty(total_kept, torch.float32)
    if kept_pos is None and want_pos:
        kept_pos = empty(total_kept, torch.int32)
    if cu_kept is None:
        cu_kept = empty(B + 1, torch.int32)
    _numel(kept_idx, total_kept, "kept_idx")
    if kept_scores is not None:
        _numel(kept_scores, total_kept, "kept_scores")
    if kept_pos is not None:
        _numel(kept_pos, total_kept, "kept_pos")
    _numel(cu_kept, B + 1, "cu_kept")
    st = _lib.load().tg_select_topk(
        _cuda(scores, "scores", torch.float32), _cuda(cu_seqlens, "cu_seqlens", torch.int32),
        _cuda(doc_begin, "doc_begin", torch.int32), _cuda(doc_end, "doc_end", torch.int32),
        _cuda(k_doc, "k_doc", torch.int32), B, scores.numel(), total_kept, int(max_seqlen),
        _cuda(kept_idx, "kept_idx", torch.int32),
        _cuda(kept_scores, "kept_scores", torch.float32) if kept_scores is not None else None,
        _cuda(kept_pos, "kept_pos", torch.int32) if kept_pos is not None else None,
        _cuda(cu_kept, "cu_kept", torch.int32), _stream(stream))
    check(st, "tg_select_topk")
    _hand_over(stream, *new)
    if kept_pos is not None:
        return kept_idx, kept_scores, cu_kept, kept_pos
    return kept_idx, kept_scores, cu_kept


def compact_rows(srcs: Sequence[torch.Tensor], kept_idx: torch.Tensor,
                 outs: Optional[Sequence[torch.Tensor]] = None, stream=None):
    """dst[t][r] = src[t][kept_idx[r]] for every tensor (rows = first dim)."""
    n = kept_idx.numel()
    if not srcs:
        raise TokenGateError("compact_rows: at least one source tensor")
    new = ()
    if outs is None:
        with _on(stream):
            outs = new = [torch.empty((n,) + tuple(s.shape[1:]), dtype=s.dtype, device=s.device) for s in srcs]
    k = len(srcs)
    if len(outs) != k:
        raise TokenGateError("compact_rows: one output per source")
    for s, o in zip(srcs, outs):
        if o.shape[1:] != s.shape[1:] or o.dtype != s.dtype or o.shape[0] != n:
            raise TokenGateError("compact_rows: output shape/dtype mismatch")
    src_arr = (ctypes.c_void_p * k)(*[_cuda(s, "src") for s in srcs])
    dst_arr = (ctypes.c_void_p * k)(*[_cuda(o, "dst") for o in outs])
    rb = (ctypes.c_int64 * k)(*[math.prod(s.shape[1:]) * s.element_size() for s in srcs])
    n_src = min(s.shape[0] for s in srcs)
    st = _lib.load().tg_compact_kv(src_arr, dst_arr, rb, k, _cuda(kept_idx, "kept_idx", torch.int32),
                                   n, n_src, _stream(stream))
    check(st, "tg_compact_kv")
    _hand_over(stream, *new)
    return list(outs)


def gated_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, s_kept: torch.Tensor,
                    gain: torch.Tensor, tau: torch.Tensor, cu_kept: torch.Tensor, max_kept: int,
                    out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """Token-gated causal GQA attention. q [K,Hq,dh], k/v [K,Hkv,dh] (same dtype).
    If `lse` ([Hq, K] f32) is given, each row's log-sum-exp is written there."""
    K, hq, dh = q.shape
    hkv = k.shape[1]
    if k.shape != (K, hkv, dh) or v.shape != k.shape or not (q.dtype == k.dtype == v.dtype):
        raise TokenGateError("gated_attention: q [K,Hq,dh], k/v [K,Hkv,dh] with one dtype")
    if q.dtype not in _DT:
        raise TokenGateError(f"gated_attention: unsupported dtype {q.dtype}")
    _numel(s_kept, K, "s_kept")
    _numel(gain, hq, "gain")
    _numel(tau, hq, "tau")
    if cu_kept.numel() < 1:
        raise TokenGateError("cu_kept must have batch+1 >= 1 elements")
    new = ()
    if out is None:
        with _on(stream):
            out = torch.empty_like(q)
        new = (out,)
    _shape(out, q.shape, "out", q.dtype)
    if lse is not None:
        _shape(lse, (hq, K), "lse", torch.float32)
    B = cu_kept.numel() - 1
    st = _lib.load().tg_gated_attention(
        _cuda(q, "q"), _cuda(k, "k"), _cuda(v, "v"), _DT[q.dtype],
        _cuda(s_kept, "s_kept", torch.float32), _cuda(gain, "gain", torch.float32),
        _cuda(tau, "tau", torch.float32), _cuda(cu_kept, "cu_kept", torch.int32), B, K,
        int(max_kept), hq, hkv, dh, _cuda(out, "out"),
        _cuda(lse, "lse") if lse is not None else None, _stream(stream))
    check(st, "tg_gated_attention")
    _hand_over(stream, *new)
    return out


def gated_attention_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                        dout: torch.Tensor, lse: torch.Tensor, s_kept: torch.Tensor,
                        gain: torch.Tensor, tau: torch.Tensor, cu_kept: torch.Tensor,
                        max_kept: int, grads=None, workspace: Optional[torch.Tensor] = None,
                        stream=None):
    """Gradients of gated_attention: returns (dq, dk, dv, ds, dgain, dtau) for upstream
    dout, from the forward's out and lse ([Hq, K] f32)."""
    K, hq, dh = q.shape
    hkv = k.shape[1]
    if k.shape != (K, hkv, dh) or v.shape != k.shape or not (q.dtype == k.dtype == v.dtype):
        raise TokenGateError("gated_attention_bwd: q [K,Hq,dh], k/v [K,Hkv,dh] with one dtype")
    if q.dtype not in _DT:
        raise TokenGateError(f"gated_attention_bwd: unsupported dtype {q.dtype}")
    _shape(out, q.shape, "out", q.dtype)
    _shape(dout, q.shape, "dout", q.dtype)
    _shape(lse, (hq, K), "lse", torch.float32)
    _numel(s_kept, K, "s_kept")
    _numel(gain, hq, "gain")
    _numel(tau, hq, "tau")
    B = cu_kept.numel() - 1
    new = ()
    if grads is None:
        f32 = dict(dtype=torch.float32, device=q.device)
        with _on(stream):
            grads = new = (torch.empty_like(q), torch.empty_like(k), torch.empty_like(v),
                           torch.empty(K, **f32), torch.empty(hq, **f32), torch.empty(hq, **f32))
    dq, dk, dv, ds, dg, dt = grads
    _shape(dq, q.shape, "dq", q.dtype)
    _shape(dk, k.shape, "dk", q.dtype)
    _shape(dv, k.shape, "dv", q.dtype)
    _shape(ds, (K,), "ds", torch.float32)
    _shape(dg, (hq,), "dgain", torch.float32)
    _shape(dt, (hq,), "dtau", torch.float32)
    lib = _lib.load()
    need = int(lib.tg_gated_attention_bwd_workspace_size(_DT[q.dtype], B, K, int(max_kept), hq,
                                                           hkv, dh))
    if workspace is None:
        with _on(stream):
            workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    nb = workspace.numel() * workspace.element_size()
    st = lib.tg_gated_attention_bwd(
        _cuda(q, "q"), _cuda(k, "k"), _cuda(v, "v"), _cuda(out, "out"), _cuda(dout, "dout"),
        _DT[q.dtype], _cuda(lse, "lse"), _cuda(s_kept, "s_kept", torch.float32),
        _cuda(gain, "gain", torch.float32), _cuda(tau, "tau", torch.float32),
        _cuda(cu_kept, "cu_kept", torch.int32), B, K, int(max_kept), hq, hkv, dh, _cuda(dq, "dq"),
        _cuda(dk, "dk"), _cuda(dv, "dv"), _cuda(ds, "ds"), _cuda(dg, "dgain"), _cuda(dt, "dtau"),
        _cuda(workspace, "workspace"), nb, _stream(stream))
    check(st, "tg_gated_attention_bwd")
    _hand_over(stream, *new)
    return dq, dk, dv, ds, dg, dt


def gated_delta_rule_workspace_size(batch: int, total: int, n_heads: int, head_dim_v: int) -> int:
    return int(_lib.load().tg_gated_delta_rule_workspace_size(batch, total, n_heads, head_dim_v))


def gated_delta_rule(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, alpha: torch.Tensor,
                     beta: torch.Tensor, cu_seqlens: torch.Tensor, max_seqlen: Optional[int] = None,
                     out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                     stream=None) -> torch.Tensor:
    """Gated delta rule per sequence and head over packed rows: q, k [T,H,dk], v [T,H,dv]
    bf16, alpha/beta [T,H] f32 -> out [T,H,dv] bf16 (state reset per sequence).
    max_seqlen bounds every sequence's length; when None it is read from cu_seqlens
    (a device-to-host copy). workspace: uint8 of at least gated_delta_rule_workspace_size
    bytes, allocated here when None."""
    T, H, dk = q.shape
    dv = v.shape[2]
    _shape(k, q.shape, "k", q.dtype)
    _shape(v, (T, H, dv), "v", q.dtype)
    _shape(alpha, (T, H), "alpha", torch.float32)
    _shape(beta, (T, H), "beta", torch.float32)
    if cu_seqlens.numel() < 1:
        raise TokenGateError("cu_seqlens must have batch+1 >= 1 elements")
    if q.dtype not in _DT:
        raise TokenGateError(f"gated_delta_rule: unsupported dtype {q.dtype}")
    B = cu_seqlens.numel() - 1
    if max_seqlen is None:
        cu_h = cu_seqlens.detach().to("cpu", torch.int64)
        max_seqlen = int((cu_h[1:] - cu_h[:-1]).max()) if B > 0 else 0
    new = ()
    if out is None:
        with _on(stream):
            out = torch.empty_like(v)
        new = (out,)
    _shape(out, v.shape, "out", v.dtype)
    need = gated_delta_rule_workspace_size(B, T, H, dv)
    if workspace is None:
        with _on(stream):
            workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    if workspace.dtype != torch.uint8 or workspace.numel() < need:
        raise TokenGateError(f"gated_delta_rule: workspace needs {need} bytes (uint8)")
    st = _lib.load().tg_gated_delta_rule(
        _cuda(q, "q"), _cuda(k, "k"), _cuda(v, "v"), _DT[q.dtype], _cuda(alpha, "alpha"),
        _cuda(beta, "beta"), _cuda(cu_seqlens, "cu_seqlens", torch.int32),
        B, T, int(max_seqlen), H, dk, dv, _cuda(out, "out"), _cuda(workspace, "workspace"),
        workspace.numel(), _stream(stream))
    check(st, "tg_gated_delta_rule")
    _hand_over(stream, *new)
    return out


def qkv_rope(xc: torch.Tensor, w_qkv: torch.Tensor, n_hq: int, n_hkv: int, pos: torch.Tensor,
             rope_base: float = 1e6, out=None, stream=None):
    """The kept rows' projections: (q [K,Hq,dh], k [K,Hkv,dh], v [K,Hkv,dh]) bf16 from
    xc [K,d] bf16 and w_qkv [(Hq+2Hkv)*dh, d] bf16, q/k rotated at pos [K] int32."""
    K, d = xc.shape
    n_out = w_qkv.shape[0]
    if (n_out % (n_hq + 2 * n_hkv)) or w_qkv.shape[1] != d or xc.dtype != w_qkv.dtype:
        raise TokenGateError("qkv_rope: w_qkv [(Hq+2Hkv)*dh, d] with the dtype of xc")
    dh = n_out // (n_hq + 2 * n_hkv)
    _numel(pos, K, "pos")
    new = ()
    if out is None:
        with _on(stream):
            out = new = (torch.empty(K, n_hq, dh, dtype=xc.dtype, device=xc.device),
                         torch.empty(K, n_hkv, dh, dtype=xc.dtype, device=xc.device),
                         torch.empty(K, n_hkv, dh, dtype=xc.dtype, device=xc.device))
    q, k, v = out
    _shape(q, (K, n_hq, dh), "q", xc.dtype)
    _shape(k, (K, n_hkv, dh), "k", xc.dtype)
    _shape(v, (K, n_hkv, dh), "v", xc.dtype)
    st = _lib.load().tg_qkv_rope(_cuda(xc, "xc", torch.bfloat16), K, d,
                                 _cuda(w_qkv, "w_qkv", torch.bfloat16), n_hq, n_hkv, dh,
                                 float(rope_base), _cuda(pos, "pos", torch.int32), _cuda(q, "q"),
                                 _cuda(k, "k"), _cuda(v, "v"), _stream(stream))
    check(st, "tg_qkv_rope")
    _hand_over(stream, *new)
    return q, k, v


def compact_qkv_rope(x: torch.Tensor, kept_idx: torch.Tensor, w_qkv: torch.Tensor, n_hq: int,
                     n_hkv: int, pos: torch.Tensor, rope_base: float = 1e6, xc=None, out=None,
                     write_xc: bool = True, stream=None):
    """The compaction fused into the projections: xc = x[kept_idx] (written when
    write_xc, into `xc` if given) and (q, k, v) of those rows, as qkv_rope(xc, ...)
    would give them, in one kernel that gathers the rows from x itself. x [N,d] bf16,
    kept_idx [K] int32. Returns (xc or None, q, k, v)."""
    N, d = x.shape
    K = kept_idx.numel()
    n_out = w_qkv.shape[0]
    if (n_out % (n_hq + 2 * n_hkv)) or w_qkv.shape[1] != d or x.dtype != w_qkv.dtype:
        raise TokenGateError("compact_qkv_rope: w_qkv [(Hq+2Hkv)*dh, d] with the dtype of x")
    dh = n_out // (n_hq + 2 * n_hkv)
    _numel(pos, K, "pos")
    new = []
    if write_xc:
        if xc is None:
            with _on(stream):
                xc = torch.empty(K, d, dtype=x.dtype, device=x.device)
            new.append(xc)
        _shape(xc, (K, d), "xc", x.dtype)
    elif xc is not None:
        raise TokenGateError("compact_qkv_rope: xc given with write_xc=False")
    if out is None:
        with _on(stream):
            out = (torch.empty(K, n_hq, dh, dtype=x.dtype, device=x.device),
                   torch.empty(K, n_hkv, dh, dtype=x.dtype, device=x.device),
                   torch.empty(K, n_hkv, dh, dtype=x.dtype, device=x.device))
        new += out
    q, k, v = out
    _shape(q, (K, n_hq, dh), "q", x.dtype)
    _shape(k, (K, n_hkv, dh), "k", x.dtype)
    _shape(v, (K, n_hkv, dh), "v", x.dtype)
    st = _lib.load().tg_compact_qkv_rope(
        _cuda(x, "x", torch.bfloat16), N, d, _cuda(kept_idx, "kept_idx", torch.int32), K,
        _cuda(xc, "xc") if xc is not None else None, _cuda(w_qkv, "w_qkv", torch.bfloat16),
        n_hq, n_hkv, dh, float(rope_base), _cuda(pos, "pos", torch.int32), _cuda(q, "q"),
        _cuda(k, "k"), _cuda(v, "v"), _stream(stream))
    check(st, "tg_compact_qkv_rope")
    _hand_over(stream, *new)
    return xc, q, k, v


def cache_append(k_new: torch.Tensor, v_new: torch.Tensor, s_new: torch.Tensor,
                 k_cache: torch.Tensor, v_cache: torch.Tensor, s_cache: torch.Tensor,
                 cache_len: torch.Tensor, stream=None) -> None:
    """Row cache_len[b] of sequence b's cache gets k_new[b], v_new[b], s_new[b];
    cache_len[b] += 1. Caches [B, cap, Hkv, dh] bf16 and [B, cap] f32."""
    B, cap, hkv, dh = k_cache.shape
    _shape(v_cache, k_cache.shape, "v_cache", k_cache.dtype)
    _shape(k_new, (B, hkv, dh), "k_new", k_cache.dtype)
    _shape(v_new, (B, hkv, dh), "v_new", k_cache.dtype)
    _shape(s_new, (B,), "s_new", torch.float32)
    _shape(s_cache, (B, cap), "s_cache", torch.float32)
    _shape(cache_len, (B,), "cache_len", torch.int32)
    st = _lib.load().tg_cache_append(
        _cuda(k_new, "k_new", torch.bfloat16), _cuda(v_new, "v_new", torch.bfloat16),
        _cuda(s_new, "s_new"), B, cap, hkv, dh, _cuda(k_cache, "k_cache", torch.bfloat16),
        _cuda(v_cache, "v_cache", torch.bfloat16), _cuda(s_cache, "s_cache"),
        _cuda(cache_len, "cache_len"), _stream(stream))
    check(st, "tg_cache_append")


def decode_workspace_size(batch: int, n_hq: int, head_dim: int, max_len: int) -> int:
    return int(_lib.load().tg_gated_decode_workspace_size(batch, n_hq, head_dim, max_len))


def gated_decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                 s_cache: torch.Tensor, cache_len: torch.Tensor, gain: torch.Tensor,
                 tau: torch.Tensor, max_len: int, out: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One query row per sequence (q [B, Hq, dh] bf16) over its cache rows
    j < cache_len[b]; returns out [B, Hq, dh] bf16."""
    B, hq, dh = q.shape
    Bc, cap, hkv, dh2 = k_cache.shape
    if Bc != B or dh2 != dh:
        raise TokenGateError("gated_decode: q [B,Hq,dh] and caches [B,cap,Hkv,dh]")
    _shape(v_cache, k_cache.shape, "v_cache", k_cache.dtype)
    _shape(s_cache, (B, cap), "s_cache", torch.float32)
    _shape(cache_len, (B,), "cache_len", torch.int32)
    _numel(gain, hq, "gain")
    _numel(tau, hq, "tau")
    new = ()
    if out is None:
        with _on(stream):
            out = torch.empty_like(q)
        new = (out,)
    _shape(out, q.shape, "out", q.dtype)
    need = decode_workspace_size(B, hq, dh, max(int(max_len), 1))
    if workspace is None:
        with _on(stream):
            workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    if workspace.numel() * workspace.element_size() < need:
        raise TokenGateError(f"gated_decode: workspace needs {need} bytes")
    st = _lib.load().tg_gated_decode(
        _cuda(q, "q", torch.bfloat16), _cuda(k_cache, "k_cache", torch.bfloat16),
        _cuda(v_cache, "v_cache", torch.bfloat16), _cuda(s_cache, "s_cache"),
        _cuda(cache_len, "cache_len"), B, cap, int(max_len), hq, hkv, dh,
        _cuda(gain, "gain", torch.float32), _cuda(tau, "tau", torch.float32), _cuda(out, "out"),
        _cuda(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _stream(stream))
    check(st, "tg_gated_decode")
    _hand_over(stream, *new)
    return out


def _call(fn, what: str, stream, tensors, args) -> None:
    """fn(*args, stream) on the tensors' device, which must be one CUDA device (None entries
    are skipped) and is made current for the call if it is not; the stream is that device's
    current one unless given. Raises on a status other than OK."""
    dev = tensors[0].get_device()   # -1 for a CPU tensor
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise TokenGateError(f"{what}: every tensor must be on the same CUDA device")
    if dev < 0:
        raise TokenGateError(f"{what}: every tensor must be a CUDA tensor")
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(dev)
    elif stream.device.index != dev:
        raise TokenGateError(f"{what}: the stream must be on the tensors' device")
    else:
        handle = stream.cuda_stream
    if torch._C._cuda_getDevice() == dev:
        st = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, handle)
    if st != 0:
        check(st, what)


def _ptr(t: torch.Tensor, name: str) -> int:
    if not t.is_contiguous():
        raise TokenGateError(f"{name} must be contiguous")
    return t.data_ptr()


def _heads(t: torch.Tensor, T: int, H: int, dh: int, name: str, dtype) -> int:
    """Token stride in elements of a [T, H, dh] tensor whose heads are dense."""
    if t.shape != (T, H, dh):
        raise TokenGateError(f"{name} must have shape {(T, H, dh)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TokenGateError(f"{name} must be {dtype}, got {t.dtype}")
    st, sh, sd = t.stride()
    if (dh > 1 and sd != 1) or (H > 1 and sh != dh):
        raise TokenGateError(f"{name} must have dense heads (strides [*, {dh}, 1])")
    return st if T > 1 else H * dh


def _norm_rope_args(what, q, k, q_weight, k_weight, pos, rot_dim):
    if q.dim() != 3 or k.dim() != 3:
        raise TokenGateError(f"{what}: q [T,Hq,dh], k [T,Hkv,dh]")
    T, hq, dh = q.shape
    hkv = k.shape[1]
    if q.dtype not in _DT:
        raise TokenGateError(f"{what}: unsupported dtype {q.dtype}")
    _shape(q_weight, (dh,), "q_weight", torch.float32)
    _shape(k_weight, (dh,), "k_weight", torch.float32)
    _shape(pos, (T,), "pos", torch.int32)
    return T, hq, hkv, dh, (dh if rot_dim is None else int(rot_dim))


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, q_weight: torch.Tensor, k_weight: torch.Tensor,
                 pos: torch.Tensor, eps: float = 1e-6, rope_base: float = 1e6,
                 rot_dim: Optional[int] = None, out=None, stream=None):
    """RMS norm of every head of q [T,Hq,dh] and k [T,Hkv,dh] (weights [dh] f32), then the
    rotary embedding of the first rot_dim elements (None: all) at pos [T] int32. q and k
    may be views with any token stride (of a packed projection output); returns (q_out,
    k_out), dense unless `out` is given. `out` may be (q, k) themselves."""
    T, hq, hkv, dh, rot = _norm_rope_args("qk_norm_rope", q, k, q_weight, k_weight, pos, rot_dim)
    dt = q.dtype
    q_st = _heads(q, T, hq, dh, "q", dt)
    k_st = _heads(k, T, hkv, dh, "k", dt)
    if out is None:
        with _on(stream):
            qo, ko = q.new_empty((T, hq, dh)), q.new_empty((T, hkv, dh))
        qo_st, ko_st = hq * dh, hkv * dh
    else:
        qo, ko = out
        qo_st = _heads(qo, T, hq, dh, "q_out", dt)
        ko_st = _heads(ko, T, hkv, dh, "k_out", dt)
    _call(_lib.load().tg_qk_norm_rope, "tg_qk_norm_rope", stream,
          (q, k, q_weight, k_weight, pos, qo, ko),
          (q.data_ptr(), q_st, k.data_ptr(), k_st, _DT[dt], T, hq, hkv, dh, rot,
           _ptr(q_weight, "q_weight"), _ptr(k_weight, "k_weight"), float(eps), float(rope_base), _ptr(pos, "pos"),
           qo.data_ptr(), qo_st, ko.data_ptr(), ko_st))
    if out is None:
        _hand_over(stream, qo, ko)
    return qo, ko


def qk_norm_rope_bwd_workspace_size(n_tokens: int, n_hq: int, n_hkv: int, head_dim: int) -> int:
    return int(_lib.load().tg_qk_norm_rope_bwd_workspace_size(n_tokens, n_hq, n_hkv, head_dim))


def qk_norm_rope_bwd(q: torch.Tensor, k: torch.Tensor, q_weight: torch.Tensor,
                     k_weight: torch.Tensor, pos: torch.Tensor, dq_out: torch.Tensor,
                     dk_out: torch.Tensor, eps: float = 1e-6, rope_base: float = 1e6,
                     rot_dim: Optional[int] = None, grads=None,
                     workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradients of qk_norm_rope for upstream dq_out, dk_out, from the forward's inputs:
    returns (dq, dk, dq_weight, dk_weight), the latter two [dh] f32. Every [T,H,dh]
    tensor may have any token stride."""
    T, hq, hkv, dh, rot = _norm_rope_args("qk_norm_rope_bwd", q, k, q_weight, k_weight, pos, rot_dim)
    dt = q.dtype
    q_st = _heads(q, T, hq, dh, "q", dt)
    k_st = _heads(k, T, hkv, dh, "k", dt)
    gq_st = _heads(dq_out, T, hq, dh, "dq_out", dt)
    gk_st = _heads(dk_out, T, hkv, dh, "dk_out", dt)
    new = ()
    if grads is None:
        with _on(stream):
            grads = new = (q.new_empty((T, hq, dh)), q.new_empty((T, hkv, dh)),
                           torch.empty_like(q_weight), torch.empty_like(k_weight))
    dq, dk, dwq, dwk = grads
    dq_st = _heads(dq, T, hq, dh, "dq", dt)
    dk_st = _heads(dk, T, hkv, dh, "dk", dt)
    _shape(dwq, (dh,), "dq_weight", torch.float32)
    _shape(dwk, (dh,), "dk_weight", torch.float32)
    lib = _lib.load()
    if workspace is None:
        need = lib.tg_qk_norm_rope_bwd_workspace_size(T, hq, hkv, dh)
        with _on(stream):
            workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _call(lib.tg_qk_norm_rope_bwd, "tg_qk_norm_rope_bwd", stream,
          (q, k, q_weight, k_weight, pos, dq_out, dk_out, dq, dk, dwq, dwk, workspace),
          (q.data_ptr(), q_st, k.data_ptr(), k_st, dq_out.data_ptr(), gq_st, dk_out.data_ptr(), gk_st,
           _DT[dt], T, hq, hkv, dh, rot, _ptr(q_weight, "q_weight"), _ptr(k_weight, "k_weight"), float(eps),
           float(rope_base), _ptr(pos, "pos"), dq.data_ptr(), dq_st, dk.data_ptr(), dk_st,
           _ptr(dwq, "dq_weight"), _ptr(dwk, "dk_weight"), _ptr(workspace, "workspace"),
           workspace.numel() * workspace.element_size()))
    _hand_over(stream, *new)
    return dq, dk, dwq, dwk


def _quant_cache(what, k_cache, v_cache, k_scale, v_scale, s_cache, cache_len):
    if k_cache.dim() != 4:
        raise TokenGateError(f"{what}: caches [B,cap,Hkv,dh]")
    B, cap, hkv, dh = k_cache.shape
    if k_cache.dtype not in _CODE_DT:
        raise TokenGateError(f"{what}: a quantised cache is int8 or float8_e4m3fn, got {k_cache.dtype}")
    _shape(v_cache, k_cache.shape, "v_cache", k_cache.dtype)
    _shape(k_scale, (B, cap, hkv), "k_scale", torch.float32)
    _shape(v_scale, (B, cap, hkv), "v_scale", torch.float32)
    _shape(s_cache, (B, cap), "s_cache", torch.float32)
    _shape(cache_len, (B,), "cache_len", torch.int32)
    return B, cap, hkv, dh


def quant_cache_append(k_new: torch.Tensor, v_new: torch.Tensor, s_new: torch.Tensor,
                       cu_new: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                       k_scale: torch.Tensor, v_scale: torch.Tensor, s_cache: torch.Tensor,
                       cache_len: torch.Tensor, start: Optional[torch.Tensor] = None,
                       src_idx: Optional[torch.Tensor] = None, stream=None) -> None:
    """Quantise rows into a cache: sequence b's packed rows [cu_new[b], cu_new[b+1]) go to
    its cache rows from start[b] (None: from cache_len[b]) on, and cache_len[b] becomes
    the row behind them. k_new, v_new [R,Hkv,dh] bf16, s_new [R] f32; packed row r is row
    src_idx[r] of them (int32), or row r when src_idx is None. Caches [B,cap,Hkv,dh] int8
    or float8_e4m3fn with scales [B,cap,Hkv] f32, s_cache [B,cap] f32."""
    B, cap, hkv, dh = _quant_cache("quant_cache_append", k_cache, v_cache, k_scale, v_scale, s_cache,
                                   cache_len)
    R = s_new.numel()
    _shape(s_new, (R,), "s_new", torch.float32)
    _shape(k_new, (R, hkv, dh), "k_new", torch.bfloat16)
    _shape(v_new, (R, hkv, dh), "v_new", torch.bfloat16)
    _shape(cu_new, (B + 1,), "cu_new", torch.int32)
    n_new = R
    if src_idx is not None:
        n_new = src_idx.numel()
        _shape(src_idx, (n_new,), "src_idx", torch.int32)
    if start is not None:
        _shape(start, (B,), "start", torch.int32)
    _call(_lib.load().tg_quant_cache_append, "tg_quant_cache_append", stream,
          (k_cache, v_cache, k_scale, v_scale, s_cache, cache_len, k_new, v_new, s_new, src_idx, cu_new,
           start),
          (_ptr(k_new, "k_new"), _ptr(v_new, "v_new"), _ptr(s_new, "s_new"), R,
           None if src_idx is None else _ptr(src_idx, "src_idx"), n_new, _ptr(cu_new, "cu_new"),
           None if start is None else _ptr(start, "start"), B, cap, hkv, dh, _CODE_DT[k_cache.dtype],
           _ptr(k_cache, "k_cache"), _ptr(v_cache, "v_cache"), _ptr(k_scale, "k_scale"),
           _ptr(v_scale, "v_scale"), _ptr(s_cache, "s_cache"), _ptr(cache_len, "cache_len")))


def quant_cache_read(k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
                     v_scale: torch.Tensor, s_cache: torch.Tensor, cache_len: torch.Tensor,
                     cu_rows: torch.Tensor, total: int, start: Optional[torch.Tensor] = None,
                     dtype: torch.dtype = torch.bfloat16, out=None, stream=None):
    """Rows of a quantised cache as packed (k [total,Hkv,dh], v, s [total] f32), k and v in
    `dtype` (bf16 or f32): sequence b's cache rows from start[b] (None: 0) on fill rows
    [cu_rows[b], cu_rows[b+1]). Rows that no sequence fills are not written: without `out`
    they hold anything."""
    B, cap, hkv, dh = _quant_cache("quant_cache_read", k_cache, v_cache, k_scale, v_scale, s_cache,
                                   cache_len)
    total = int(total)
    _shape(cu_rows, (B + 1,), "cu_rows", torch.int32)
    if start is not None:
        _shape(start, (B,), "start", torch.int32)
    if dtype not in _DT:
        raise TokenGateError(f"quant_cache_read: unsupported dtype {dtype}")
    if out is None:
        with _on(stream):
            k = k_cache.new_empty((total, hkv, dh), dtype=dtype)
            v, s_out = torch.empty_like(k), s_cache.new_empty(total)
    else:
        k, v, s_out = out
        if k.dtype not in _DT:
            raise TokenGateError(f"quant_cache_read: unsupported dtype {k.dtype}")
        _shape(k, (total, hkv, dh), "k", k.dtype)
        _shape(v, (total, hkv, dh), "v", k.dtype)
        _shape(s_out, (total,), "s", torch.float32)
    _call(_lib.load().tg_quant_cache_read, "tg_quant_cache_read", stream,
          (k_cache, v_cache, k_scale, v_scale, s_cache, cache_len, start, cu_rows, k, v, s_out),
          (_ptr(k_cache, "k_cache"), _ptr(v_cache, "v_cache"), _ptr(k_scale, "k_scale"),
           _ptr(v_scale, "v_scale"), _ptr(s_cache, "s_cache"), _ptr(cache_len, "cache_len"),
           None if start is None else _ptr(start, "start"), _ptr(cu_rows, "cu_rows"), total, B, cap, hkv,
           dh, _CODE_DT[k_cache.dtype], _DT[k.dtype], _ptr(k, "k"), _ptr(v, "v"), _ptr(s_out, "s")))
    if out is None:
        _hand_over(stream, k, v, s_out)
    return k, v, s_out


def tree_mask(parents: Sequence[Sequence[int]]) -> torch.Tensor:
    """tree_attention's mask ([B, T] int64, on the CPU) of a tree per sequence: parents[b][t]
    is the drafted token that t continues, or -1 where it continues the cache itself. A
    parent comes before its children; shorter trees are filled up with 0."""
    T = max((len(p) for p in parents), default=0)
    if T > 64:
        raise TokenGateError(f"tree_mask: at most 64 drafted tokens, got {T}")
    rows = []
    for b, par in enumerate(parents):
        bits = []
        for t, p in enumerate(par):
            if not -1 <= p < t:
                raise TokenGateError(f"tree_mask: parents[{b}][{t}] = {p} must be in [-1, {t})")
            bits.append((bits[p] if p >= 0 else 0) | 1 << t)
        rows.append([x - (1 << 64) if x >> 63 else x for x in bits] + [0] * (T - len(bits)))
    return torch.tensor(rows, dtype=torch.int64).reshape(len(rows), T)


def tree_attention_workspace_size(batch: int, n_draft: int, n_hq: int, n_hkv: int, head_dim: int,
                                  max_len: int) -> int:
    return int(_lib.load().tg_tree_attention_workspace_size(batch, n_draft, max_len, n_hq, n_hkv,
                                                            head_dim))


def tree_attention(q: torch.Tensor, k_draft: torch.Tensor, v_draft: torch.Tensor,
                   s_draft: torch.Tensor, tree_mask: torch.Tensor, k_cache: torch.Tensor,
                   v_cache: torch.Tensor, s_cache: torch.Tensor, cache_len: torch.Tensor,
                   gain: torch.Tensor, tau: torch.Tensor, max_len: int,
                   draft_len: Optional[torch.Tensor] = None, k_scale: Optional[torch.Tensor] = None,
                   v_scale: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of T drafted tokens per sequence (q [B,T,Hq,dh], k_draft/v_draft
    [B,T,Hkv,dh] bf16, s_draft [B,T] f32) over the cache rows j < cache_len[b] and the
    drafted tokens in their tree_mask ([B,T] int64, bit i: token i). The cache is bf16
    (cache_append's) or, with k_scale and v_scale, quantised (quant_cache_append's).
    draft_len [B] int32: drafted tokens of each sequence (None: T); rows of out behind
    them are left as they were (zeros where out is allocated here). Returns out
    [B,T,Hq,dh] bf16."""
    if q.dim() != 4 or k_cache.dim() != 4:
        raise TokenGateError("tree_attention: q [B,T,Hq,dh], caches [B,cap,Hkv,dh]")
    B, T, hq, dh = q.shape
    cap, hkv = k_cache.shape[1], k_cache.shape[2]
    _shape(k_cache, (B, cap, hkv, dh), "k_cache")
    _shape(v_cache, k_cache.shape, "v_cache", k_cache.dtype)
    _shape(k_draft, (B, T, hkv, dh), "k_draft", torch.bfloat16)
    _shape(v_draft, (B, T, hkv, dh), "v_draft", torch.bfloat16)
    _shape(s_draft, (B, T), "s_draft", torch.float32)
    _shape(tree_mask, (B, T), "tree_mask", torch.int64)
    _shape(s_cache, (B, cap), "s_cache", torch.float32)
    _shape(cache_len, (B,), "cache_len", torch.int32)
    _shape(gain, (hq,), "gain", torch.float32)
    _shape(tau, (hq,), "tau", torch.float32)
    if draft_len is not None:
        _shape(draft_len, (B,), "draft_len", torch.int32)
    if k_cache.dtype in _CODE_DT:
        if k_scale is None or v_scale is None:
            raise TokenGateError("tree_attention: a quantised cache needs k_scale and v_scale")
        cdt = _CODE_DT[k_cache.dtype]
        _shape(k_scale, (B, cap, hkv), "k_scale", torch.float32)
        _shape(v_scale, (B, cap, hkv), "v_scale", torch.float32)
        ks, vs = _ptr(k_scale, "k_scale"), _ptr(v_scale, "v_scale")
    else:
        if k_cache.dtype != torch.bfloat16 or k_scale is not None or v_scale is not None:
            raise TokenGateError("tree_attention: a cache is bf16 without scales, or int8 or "
                                 "float8_e4m3fn with them")
        cdt, ks, vs = TG_BF16, None, None
    if q.dtype != torch.bfloat16:
        raise TokenGateError(f"q must be {torch.bfloat16}, got {q.dtype}")
    max_len = int(max_len)
    new = ()
    if out is None:
        with _on(stream):
            make = torch.empty_like if draft_len is None else torch.zeros_like
            out = make(q, memory_format=torch.contiguous_format)
        new = (out,)
    else:
        _shape(out, q.shape, "out", torch.bfloat16)
    lib = _lib.load()
    if workspace is None:
        need = lib.tg_tree_attention_workspace_size(B, T, max_len, hq, hkv, dh)
        with _on(stream):
            workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _call(lib.tg_tree_attention, "tg_tree_attention", stream,
          (q, k_draft, v_draft, s_draft, tree_mask, draft_len, k_cache, v_cache, k_scale, v_scale, s_cache,
           cache_len, gain, tau, out, workspace),
          (_ptr(q, "q"), _ptr(k_draft, "k_draft"), _ptr(v_draft, "v_draft"), _ptr(s_draft, "s_draft"),
           _ptr(tree_mask, "tree_mask"), None if draft_len is None else _ptr(draft_len, "draft_len"), B, T,
           _ptr(k_cache, "k_cache"), _ptr(v_cache, "v_cache"), cdt, ks, vs, _ptr(s_cache, "s_cache"),
           _ptr(cache_len, "cache_len"), cap, max_len, hq, hkv, dh, _ptr(gain, "gain"), _ptr(tau, "tau"),
           _ptr(out, "out"), _ptr(workspace, "workspace"), workspace.numel() * workspace.element_size()))
    _hand_over(stream, *new)
    return out


def device_status(reset: bool = True, stream=None) -> int:
    """Synchronise the stream and return (then clear) the device status word."""
    return _lib.load().tg_device_status(_stream(stream), 1 if reset else 0)


def selftest_bounded_wait(timeout_ns: int, stream=None) -> None:
    check(_lib.load().tg_selftest_bounded_wait(int(timeout_ns), _stream(stream)),
          "tg_selftest_bounded_wait")
