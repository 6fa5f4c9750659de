"""GB300-native sequence-parallel attention core (Python binding).

The functions named usp_* mirror the C ABI of include/usp.h one to one and
only marshal arguments (tensors -> device pointers, the current CUDA stream).
Every step of the computation runs in the CUDA library libusp.so; there is
no Python or CPU fallback, and a missing library raises.

The helpers below them (attn_forward, attn_backward, permute,
merge_partials, the kv4_* calls of the 4-bit KV cache) allocate outputs and
workspaces with PyTorch and call the same entry points.
"""
from __future__ import annotations

import ctypes
import struct
from typing import NamedTuple, Optional, Tuple

import torch

from . import _lib

LAYOUT = {"contiguous": 0, "zigzag": 1, "stripe": 2}
DTYPE = {torch.bfloat16: 0, torch.float32: 1}
PERMUTE = {"extract": 0, "restore": 1, "seq2head": 2, "head2seq": 3}
FLAG_FORCE_SIMT = 1
FLAG_SAVED_EXCHANGE = 2
FLAG_NATURAL_ORDER = 4


class UspError(RuntimeError):
    pass


def _p(x) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, torch.Tensor):
        return x.data_ptr() if x.numel() else None
    return int(x)


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream or None
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream or None
    return int(stream) or None


def _check(status: int) -> None:
    if status != 0:
        lib = _lib.load()
        name = lib.usp_status_string(status).decode()
        if name == "USP_ERR_CUDA":
            name += ": " + lib.usp_last_error_detail().decode()
        raise UspError(name)


def _enum(table, x) -> int:
    return table[x] if not isinstance(x, int) else x


# --- the C ABI, one to one ---------------------------------------------------

def usp_attn_fwd(q, k, v, out, lse, B, S, Hq, Hkv, D, softmax_scale, causal,
                 window, sink_tokens, cu_seqlens, cp_size, ulysses_degree,
                 layout, dtype, flags=0, workspace=None, workspace_bytes=0,
                 stream=None) -> None:
    _check(_lib.load().usp_attn_fwd(
        _p(q), _p(k), _p(v), _p(out), _p(lse), B, S, Hq, Hkv, D,
        float(softmax_scale), int(causal), int(window), int(sink_tokens),
        _p(cu_seqlens), cp_size, ulysses_degree, _enum(LAYOUT, layout),
        _enum(DTYPE, dtype), flags, _p(workspace), int(workspace_bytes),
        _stream(stream)))


def usp_attn_fwd_fp8(q, k, v, q_descale, k_descale, v_descale, out, lse, B, S, Hq, Hkv,
                     D, softmax_scale, causal, window, sink_tokens, cu_seqlens, cp_size,
                     ulysses_degree, layout, flags=0, workspace=None, workspace_bytes=0,
                     stream=None) -> None:
    _check(_lib.load().usp_attn_fwd_fp8(
        _p(q), _p(k), _p(v), float(q_descale), float(k_descale), float(v_descale), _p(out),
        _p(lse), B, S, Hq, Hkv, D, float(softmax_scale), int(causal), int(window),
        int(sink_tokens), _p(cu_seqlens), cp_size, ulysses_degree, _enum(LAYOUT, layout),
        flags, _p(workspace), int(workspace_bytes), _stream(stream)))


def usp_attn_fwd_fp8_workspace_size(B, S, Hq, Hkv, D, cp_size, ulysses_degree) -> int:
    return int(_lib.load().usp_attn_fwd_fp8_workspace_size(B, S, Hq, Hkv, D, cp_size,
                                                           ulysses_degree))


def usp_quantize_e4m3(x, out, n, inv_scale, stream=None) -> None:
    _check(_lib.load().usp_quantize_e4m3(_p(x), _p(out), int(n), float(inv_scale),
                                         _stream(stream)))


def usp_attn_fwd_workspace_size(B, S, Hq, Hkv, D, cp_size, ulysses_degree,
                                dtype, flags=0) -> int:
    return int(_lib.load().usp_attn_fwd_workspace_size(
        B, S, Hq, Hkv, D, cp_size, ulysses_degree, _enum(DTYPE, dtype), flags))


def usp_attn_bwd(q, k, v, out, lse, dout, dq, dk, dv, B, S, Hq, Hkv, D,
                 softmax_scale, causal, window, sink_tokens, cu_seqlens,
                 cp_size, ulysses_degree, layout, dtype, flags=0,
                 workspace=None, workspace_bytes=0, stream=None) -> None:
    _check(_lib.load().usp_attn_bwd(
        _p(q), _p(k), _p(v), _p(out), _p(lse), _p(dout), _p(dq), _p(dk),
        _p(dv), B, S, Hq, Hkv, D, float(softmax_scale), int(causal),
        int(window), int(sink_tokens), _p(cu_seqlens), cp_size,
        ulysses_degree, _enum(LAYOUT, layout), _enum(DTYPE, dtype), flags,
        _p(workspace), int(workspace_bytes), _stream(stream)))


def usp_attn_bwd_workspace_size(B, S, Hq, Hkv, D, cp_size, ulysses_degree,
                                dtype, flags=0) -> int:
    return int(_lib.load().usp_attn_bwd_workspace_size(
        B, S, Hq, Hkv, D, cp_size, ulysses_degree, _enum(DTYPE, dtype), flags))


def usp_attn_bwd_noalloc(q, k, v, out, lse, dout, dq, dk, dv, B, S, Hq, Hkv,
                         D, softmax_scale, causal, window, sink_tokens,
                         cu_seqlens, cp_size, ulysses_degree, layout, dtype,
                         flags=0, stream=None) -> None:
    """usp_attn_bwd without a workspace: scratch comes from the library's
    fixed 64 MiB device array (for callers that cannot allocate; calls that
    overlap on the GPU race on it)."""
    _check(_lib.load().usp_attn_bwd_noalloc(
        _p(q), _p(k), _p(v), _p(out), _p(lse), _p(dout), _p(dq), _p(dk),
        _p(dv), B, S, Hq, Hkv, D, float(softmax_scale), int(causal),
        int(window), int(sink_tokens), _p(cu_seqlens), cp_size,
        ulysses_degree, _enum(LAYOUT, layout), _enum(DTYPE, dtype), flags,
        _stream(stream)))


def usp_merge_partials(o_parts, lse_parts, n, rows, D, tree_order, o_out,
                       out_dtype, lse_out, stream=None) -> None:
    _check(_lib.load().usp_merge_partials(
        _p(o_parts), _p(lse_parts), n, rows, D, int(tree_order), _p(o_out),
        _enum(DTYPE, out_dtype), _p(lse_out), _stream(stream)))


def usp_attn_decode(q, k, v, out, lse, B, Tq, S, Hq, Hkv, D, softmax_scale,
                    causal, cp_size, splits_per_shard, tree_order, dtype,
                    workspace=None, workspace_bytes=0, stream=None) -> None:
    _check(_lib.load().usp_attn_decode(
        _p(q), _p(k), _p(v), _p(out), _p(lse), B, Tq, S, Hq, Hkv, D,
        float(softmax_scale), int(causal), cp_size, splits_per_shard,
        int(tree_order), _enum(DTYPE, dtype), _p(workspace),
        int(workspace_bytes), _stream(stream)))


def usp_attn_decode_workspace_size(B, Tq, S, Hq, Hkv, D, cp_size,
                                   splits_per_shard) -> int:
    return int(_lib.load().usp_attn_decode_workspace_size(
        B, Tq, S, Hq, Hkv, D, cp_size, splits_per_shard))


def usp_kv4_append(cache, k, v, new_weight, cu_seqlens, T, dtype, seq_lens_out,
                   stream=None) -> None:
    """cache: a _lib.Kv4CacheStruct (as in the other usp_kv4 calls)."""
    _check(_lib.load().usp_kv4_append(
        ctypes.addressof(cache), _p(k), _p(v), _p(new_weight), _p(cu_seqlens), int(T),
        _enum(DTYPE, dtype), _p(seq_lens_out), _stream(stream)))


def usp_kv4_read(cache, start, T, k, v, dtype, stream=None) -> None:
    _check(_lib.load().usp_kv4_read(ctypes.addressof(cache), _p(start), int(T), _p(k), _p(v),
                                    _enum(DTYPE, dtype), _stream(stream)))


def usp_attn_decode_kv4(cache, q, out, lse, Tq, Hq, softmax_scale, causal, window,
                        sink_tokens, accumulate, dtype, workspace=None,
                        workspace_bytes=0, stream=None) -> None:
    _check(_lib.load().usp_attn_decode_kv4(
        ctypes.addressof(cache), _p(q), _p(out), _p(lse), Tq, Hq, float(softmax_scale),
        int(causal), int(window), int(sink_tokens), int(accumulate), _enum(DTYPE, dtype),
        _p(workspace), int(workspace_bytes), _stream(stream)))


def usp_attn_decode_kv4_workspace_size(B, Tq, capacity, Hq, Hkv, D, accumulate) -> int:
    return int(_lib.load().usp_attn_decode_kv4_workspace_size(B, Tq, capacity, Hq, Hkv, D,
                                                              int(accumulate)))


def usp_attn_key_weights(q, k, lse, weight, B, S, Hq, Hkv, D, softmax_scale, causal, window,
                         sink_tokens, cu_seqlens, cp_size, layout, observe, dtype, flags=0,
                         workspace=None, workspace_bytes=0, stream=None) -> None:
    _check(_lib.load().usp_attn_key_weights(
        _p(q), _p(k), _p(lse), _p(weight), B, S, Hq, Hkv, D, float(softmax_scale), int(causal),
        int(window), int(sink_tokens), _p(cu_seqlens), cp_size, _enum(LAYOUT, layout),
        int(observe), _enum(DTYPE, dtype), flags, _p(workspace), int(workspace_bytes),
        _stream(stream)))


def usp_attn_key_weights_workspace_size(B, S, Hq, Hkv, observe, dtype, flags=0) -> int:
    return int(_lib.load().usp_attn_key_weights_workspace_size(
        B, S, Hq, Hkv, int(observe), _enum(DTYPE, dtype), flags))


def usp_kv4_evict(src, dst, kept, keep, recent, sink_tokens, stream=None) -> None:
    _check(_lib.load().usp_kv4_evict(ctypes.addressof(src), ctypes.addressof(dst), _p(kept),
                                     int(keep), int(recent), int(sink_tokens), _stream(stream)))


def usp_permute(src, dst, kind, layout, B, S, H, D, cp_size, ulysses_degree,
                elem_bytes, stream=None) -> None:
    _check(_lib.load().usp_permute(
        _p(src), _p(dst), _enum(PERMUTE, kind), _enum(LAYOUT, layout), B, S, H,
        D, cp_size, ulysses_degree, elem_bytes, _stream(stream)))


def usp_check_cu_seqlens(cu_seqlens_host, nseq, total_tokens) -> None:
    """Raise unless cu_seqlens_host (int32, host) starts at 0, never
    decreases and ends at total_tokens (the debug-mode check)."""
    st = _lib.load().usp_check_cu_seqlens(_p(cu_seqlens_host), int(nseq), int(total_tokens))
    if st != 0:
        lib = _lib.load()
        raise UspError(lib.usp_status_string(st).decode() + ": "
                       + lib.usp_last_error_detail().decode())


def usp_launch_count() -> int:
    return int(_lib.load().usp_launch_count())


def usp_device_status() -> None:
    """Raise if a kernel flagged a failed (timed-out) wait since the last call."""
    _check(_lib.load().usp_device_status())


def usp_selftest_wait_timeout(limit_us: int, stream=None) -> None:
    """Launch a kernel whose bounded wait must time out after limit_us
    (diagnostics: the next usp_device_status() reports USP_ERR_TIMEOUT)."""
    _check(_lib.load().usp_selftest_wait_timeout(int(limit_us), _stream(stream)))


def usp_profile_enable(on: bool) -> None:
    _check(_lib.load().usp_profile_enable(int(bool(on))))


def usp_profile_read(max_stats: int = 64) -> dict:
    """{kernel name: (launches, total device ms)} since the last read."""
    arr = (_lib.KernelStat * max_stats)()
    n = _lib.load().usp_profile_read(arr, max_stats)
    if n < 0:
        raise UspError("USP_ERR_CUDA")
    return {arr[i].name.decode(): (int(arr[i].launches), float(arr[i].total_ms))
            for i in range(n)}


# --- allocation helpers -----------------------------------------------------

def _dims(q: torch.Tensor, k: torch.Tensor, cu_seqlens):
    if cu_seqlens is not None:
        T, Hq, D = q.shape
        return int(cu_seqlens.numel() - 1), T, Hq, k.shape[1], D, 1
    B, S, Hq, D = q.shape
    return B, S, Hq, k.shape[2], D, B


def _packed_dims(qkv: torch.Tensor, cu_seqlens):
    if cu_seqlens is not None:
        T, _, H, D = qkv.shape
        return int(cu_seqlens.numel() - 1), T, H, D, 1
    B, S, _, H, D = qkv.shape
    return B, S, H, D, B


def check_cu_seqlens(cu_seqlens: torch.Tensor, total_tokens: int) -> None:
    """Check packed-sequence boundaries on the host before a call (the
    attention calls trust them); copies a device tensor to the host."""
    cu = cu_seqlens.detach().to("cpu", torch.int32).contiguous()
    if cu.dim() != 1 or cu.numel() < 2:
        raise UspError("USP_ERR_INVALID_ARG: cu_seqlens needs at least two entries")
    usp_check_cu_seqlens(cu, cu.numel() - 1, total_tokens)


def attn_forward_qkvpacked(qkv, *, causal=True, window=0, sink_tokens=0,
                           cu_seqlens=None, cp=1, ud=1, layout="contiguous",
                           softmax_scale=0.0, flags=0, workspace=None, stream=None):
    """(out, lse) for a packed rank-major qkv [B,S,3,H,D] (packed sequences:
    [T,3,H,D] with cu_seqlens)."""
    B, S, H, D, Bl = _packed_dims(qkv, cu_seqlens)
    out = torch.empty(qkv.shape[:-3] + (H, D), dtype=qkv.dtype, device=qkv.device)
    lse = torch.empty((Bl, H, S) if cu_seqlens is None else (H, S),
                      dtype=torch.float32, device=qkv.device)
    ws, ws_n = _use_workspace(
        workspace, usp_attn_fwd_workspace_size(Bl, S, H, H, D, cp, ud, qkv.dtype, flags),
        qkv.device)
    _check(_lib.load().usp_attn_fwd_qkvpacked(
        _p(qkv), _p(out), _p(lse), B, S, H, D, float(softmax_scale), int(causal),
        int(window), int(sink_tokens), _p(cu_seqlens), cp, ud, _enum(LAYOUT, layout),
        _enum(DTYPE, qkv.dtype), flags, _p(ws), int(ws_n), _stream(stream)))
    return out, lse


def attn_backward_qkvpacked(qkv, out, lse, dout, *, causal=True, window=0,
                            sink_tokens=0, cu_seqlens=None, cp=1, ud=1,
                            layout="contiguous", softmax_scale=0.0, flags=0,
                            workspace=None, saved_exchange=False,
                            stream=None) -> torch.Tensor:
    """dqkv (qkv's shape) for a packed qkv and the forward's (out, lse);
    saved_exchange as in attn_backward."""
    B, S, H, D, Bl = _packed_dims(qkv, cu_seqlens)
    dqkv = torch.empty_like(qkv)
    if saved_exchange:
        if workspace is None:
            raise ValueError("saved_exchange needs the forward's workspace")
        flags |= FLAG_SAVED_EXCHANGE
    ws, ws_n = _use_workspace(
        workspace, usp_attn_bwd_workspace_size(Bl, S, H, H, D, cp, ud, qkv.dtype, flags),
        qkv.device)
    _check(_lib.load().usp_attn_bwd_qkvpacked(
        _p(qkv), _p(out), _p(lse), _p(dout), _p(dqkv), B, S, H, D,
        float(softmax_scale), int(causal), int(window), int(sink_tokens),
        _p(cu_seqlens), cp, ud, _enum(LAYOUT, layout), _enum(DTYPE, qkv.dtype),
        flags, _p(ws), int(ws_n), _stream(stream)))
    return dqkv


def attn_decode(q, k, v, *, causal=True, cp=1, splits=1, tree_order=True,
                softmax_scale=0.0, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(out [B,Tq,Hq,D], lse [B,Tq,Hq]) of the newest Tq tokens q
    [B,Tq,Hq,D] against a rank-major contiguous KV cache k, v [B,S,Hkv,D]."""
    B, Tq, Hq, D = q.shape
    S, Hkv = k.shape[1], k.shape[2]
    out = torch.empty_like(q)
    lse = torch.empty((B, Tq, Hq), dtype=torch.float32, device=q.device)
    ws_n = usp_attn_decode_workspace_size(B, Tq, S, Hq, Hkv, D, cp, splits)
    ws = torch.empty(ws_n, dtype=torch.uint8, device=q.device)
    usp_attn_decode(q, k, v, out, lse, B, Tq, S, Hq, Hkv, D, softmax_scale,
                    causal, cp, splits, tree_order, q.dtype, ws, ws_n, stream)
    return out, lse


def _use_workspace(workspace, need, device):
    """The caller's uint8 workspace (checked for size), else a fresh one."""
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=device) if need else None, need
    if workspace.dtype != torch.uint8 or workspace.numel() < need:
        raise ValueError(f"workspace must be a uint8 tensor of at least {need} bytes")
    return workspace, workspace.numel()


def attn_workspace(q, k, *, cu_seqlens=None, cp=1, ud=1, flags=0,
                   natural=False) -> torch.Tensor:
    """A workspace that fits both attn_forward and attn_backward of these
    shapes. Passing the same one to both, and saved_exchange=True to the
    backward, lets the backward reuse the forward's Ulysses exchange (or,
    natural=True, its rank-major copies)."""
    if natural:
        flags |= FLAG_NATURAL_ORDER
    B, S, Hq, Hkv, D, Bl = _dims(q, k, cu_seqlens)
    n = usp_attn_bwd_workspace_size(Bl, S, Hq, Hkv, D, cp, ud, q.dtype, flags)
    return torch.empty(n, dtype=torch.uint8, device=q.device)


def attn_forward(q, k, v, *, causal=True, window=0, sink_tokens=0,
                 cu_seqlens=None, cp=1, ud=1, layout="contiguous",
                 softmax_scale=0.0, flags=0, workspace=None, stream=None,
                 natural=False) -> Tuple[torch.Tensor, torch.Tensor]:
    """(out, lse) for rank-major q/k/v ([B,S,H,D] or packed [T,H,D]);
    natural=True: q/k/v and out in natural sequence order (lse rank-major),
    the layout's extract and restore done inside the call
    (FLAG_NATURAL_ORDER)."""
    if natural:
        flags |= FLAG_NATURAL_ORDER
    B, S, Hq, Hkv, D, Bl = _dims(q, k, cu_seqlens)
    out = torch.empty_like(q)
    lse = torch.empty((Bl, Hq, S) if cu_seqlens is None else (Hq, S),
                      dtype=torch.float32, device=q.device)
    ws, ws_n = _use_workspace(
        workspace, usp_attn_fwd_workspace_size(Bl, S, Hq, Hkv, D, cp, ud, q.dtype, flags),
        q.device)
    usp_attn_fwd(q, k, v, out, lse, B, S, Hq, Hkv, D, softmax_scale, causal,
                 window, sink_tokens, cu_seqlens, cp, ud, layout, q.dtype,
                 flags, ws, ws_n, stream)
    return out, lse


def attn_backward(q, k, v, out, lse, dout, *, causal=True, window=0,
                  sink_tokens=0, cu_seqlens=None, cp=1, ud=1,
                  layout="contiguous", softmax_scale=0.0, flags=0,
                  workspace=None, saved_exchange=False, stream=None, natural=False):
    """(dq, dk, dv) for rank-major tensors and the forward's (out, lse).
    saved_exchange: workspace is the one the forward wrote (attn_workspace),
    holding its head-sharded q, k, v, out (FLAG_SAVED_EXCHANGE).
    natural: as in attn_forward (every tensor but lse in natural order)."""
    if natural:
        flags |= FLAG_NATURAL_ORDER
    B, S, Hq, Hkv, D, Bl = _dims(q, k, cu_seqlens)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    if saved_exchange:
        if workspace is None:
            raise ValueError("saved_exchange needs the forward's workspace")
        flags |= FLAG_SAVED_EXCHANGE
    ws, ws_n = _use_workspace(
        workspace, usp_attn_bwd_workspace_size(Bl, S, Hq, Hkv, D, cp, ud, q.dtype, flags),
        q.device)
    usp_attn_bwd(q, k, v, out, lse, dout, dq, dk, dv, B, S, Hq, Hkv, D,
                 softmax_scale, causal, window, sink_tokens, cu_seqlens, cp,
                 ud, layout, q.dtype, flags, ws, ws_n, stream)
    return dq, dk, dv


def quantize_e4m3(x: torch.Tensor, inv_scale: float, stream=None) -> torch.Tensor:
    """E4M3 codes (uint8, x's shape) of a bf16 tensor times inv_scale."""
    if x.dtype != torch.bfloat16 or not x.is_contiguous():
        raise ValueError("quantize_e4m3 takes a contiguous bf16 tensor")
    out = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    usp_quantize_e4m3(x, out, x.numel(), inv_scale, stream)
    return out


def attn_forward_fp8(q8, k8, v8, q_descale, k_descale, v_descale, *, causal=True,
                     window=0, sink_tokens=0, cu_seqlens=None, cp=1, ud=1,
                     layout="contiguous", softmax_scale=0.0, workspace=None, stream=None
                     ) -> Tuple[torch.Tensor, torch.Tensor]:
    """(out bf16, lse) for rank-major e4m3 codes q8/k8/v8 (uint8 or
    float8_e4m3fn tensors, [B,S,H,128] or packed [T,H,128]) with per-tensor
    descales."""
    B, S, Hq, Hkv, D, Bl = _dims(q8, k8, cu_seqlens)
    out = torch.empty(q8.shape, dtype=torch.bfloat16, device=q8.device)
    lse = torch.empty((Bl, Hq, S) if cu_seqlens is None else (Hq, S),
                      dtype=torch.float32, device=q8.device)
    ws, ws_n = _use_workspace(
        workspace, usp_attn_fwd_fp8_workspace_size(Bl, S, Hq, Hkv, D, cp, ud), q8.device)
    usp_attn_fwd_fp8(q8, k8, v8, q_descale, k_descale, v_descale, out, lse, B, S, Hq, Hkv,
                     D, softmax_scale, causal, window, sink_tokens, cu_seqlens, cp, ud,
                     layout, 0, ws, ws_n, stream)
    return out, lse


def permute(x: torch.Tensor, kind: str, layout: str = "contiguous", cp: int = 1,
            ud: int = 1, stream=None) -> torch.Tensor:
    """Layout extract/restore of [B,S,H,D] (packed: [T,H,D]) or the Ulysses
    exchange ([B,S,H,D] <-> [ud,B,S,H/ud,D]). One 4-byte number per token, such as
    the key weights w [B,Hkv,S]: permute(w.view(B * Hkv, S, 1, 1), ...).view_as(w)."""
    if kind in ("extract", "restore"):
        xb = x if x.dim() == 4 else x.unsqueeze(0)
        B, S, H, D = xb.shape
        dst = torch.empty_like(x)
    elif kind == "seq2head":
        B, S, H, D = x.shape
        dst = torch.empty((ud, B, S, H // ud, D), dtype=x.dtype, device=x.device)
    else:
        _, B, S, Hg, D = x.shape
        H = Hg * ud
        dst = torch.empty((B, S, H, D), dtype=x.dtype, device=x.device)
    usp_permute(x, dst, kind, layout, B, S, H, D, cp, ud, x.element_size(),
                stream)
    return dst


def merge_partials(o_parts: torch.Tensor, lse_parts: torch.Tensor,
                   tree_order: bool = False, out_dtype=torch.float32,
                   stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """o_parts [n, rows, D] fp32, lse_parts [n, rows] -> (O [rows, D], LSE)."""
    n, rows, D = o_parts.shape
    o = torch.empty((rows, D), dtype=out_dtype, device=o_parts.device)
    lse = torch.empty((rows,), dtype=torch.float32, device=o_parts.device)
    usp_merge_partials(o_parts, lse_parts, n, rows, D, tree_order, o,
                       out_dtype, lse, stream)
    return o, lse


# --- the 4-bit KV cache --------------------------------------------------------

class KV4Cache(NamedTuple):
    """A KV cache in 4 bits (usp_kv4_cache_t in include/usp.h, which gives the
    number format): codes uint8 [B, Hkv, capacity, D/2], E4M3 scales uint8
    [B, Hkv, capacity, D/32], cached tokens int32 [B], and (or None) the
    attention weight each key has collected, fp32 [B, Hkv, capacity]. All on
    one device and contiguous; capacity a multiple of 16."""
    k: torch.Tensor
    k_scale: torch.Tensor
    v: torch.Tensor
    v_scale: torch.Tensor
    seq_lens: torch.Tensor
    key_weight: Optional[torch.Tensor] = None
    k_descale: float = 1.0
    v_descale: float = 1.0


def kv4_cache(B: int, capacity: int, Hkv: int, D: int, *, device="cuda", key_weight=False,
              k_descale: float = 1.0, v_descale: float = 1.0) -> KV4Cache:
    """An empty cache; the capacity is rounded up to a multiple of 16.
    descales: what a stored value is multiplied with. 1 suits keys and values
    whose blocks of 32 have maxima between 0.1 and 3136 (the scales' range)."""
    C = -(-int(capacity) // 16) * 16
    z = dict(dtype=torch.uint8, device=device)
    return KV4Cache(
        torch.zeros((B, Hkv, C, D // 2), **z), torch.zeros((B, Hkv, C, D // 32), **z),
        torch.zeros((B, Hkv, C, D // 2), **z), torch.zeros((B, Hkv, C, D // 32), **z),
        torch.zeros((B,), dtype=torch.int32, device=device),
        torch.zeros((B, Hkv, C), dtype=torch.float32, device=device) if key_weight else None,
        float(k_descale), float(v_descale))


def _need(x, name, dtype, shape, device) -> None:
    if x.dtype != dtype or tuple(x.shape) != tuple(shape) or x.device != device:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)} on {device}, "
                         f"got {x.dtype} {tuple(x.shape)} on {x.device}")
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _fits(x, dtype, shape, index) -> bool:
    return (x.dtype is dtype and x.shape == shape and x.get_device() == index
            and x.is_contiguous())


def _require(x, name, dtype, shape, index, like) -> None:
    """_need, with the common case (it fits) in as few calls as possible: a
    decoding step's helpers run for a few microseconds on the GPU."""
    if not _fits(x, dtype, shape, index):
        _need(x, name, dtype, shape, like.device)


def _call(fn, index, stream, *args) -> None:
    """fn(*args, stream) on the tensors' device and (default) its current
    stream; raises what it returns."""
    if index < 0:
        raise ValueError("the tensors must be on a CUDA device")
    raw = torch._C._cuda_getCurrentRawStream(index) if stream is None else _stream(stream)
    if torch._C._cuda_getDevice() == index:
        st = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            st = fn(*args, raw)
    if st:
        _check(st)


def _on(stream, device):
    """Context in which `stream` (a Stream or a raw handle) is the current one, so
    that what a call allocates belongs to the stream it runs on: memory of
    another stream may still be written by work queued there, or be handed on
    while this call's kernels run."""
    if device.type != "cuda":
        raise ValueError("the tensors must be on a CUDA device")
    if not isinstance(stream, torch.cuda.Stream):
        raw = int(stream)
        stream = torch.cuda.ExternalStream(raw, device=device) if raw else \
            torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


_U8, _I32, _F32 = torch.uint8, torch.int32, torch.float32
_pack_kv4 = struct.Struct("6Q4i2f").pack  # a _lib.Kv4CacheStruct's bytes (2 us less per call)


def _kv4_struct(cache: KV4Cache):
    """(C struct's bytes, device index, B, Hkv, capacity, D) of a cache whose
    tensors fit together, else ValueError."""
    k, ks, v, vs, lens, w, kd, vd = cache
    shape = k.shape
    if len(shape) != 4:
        raise ValueError("cache.k must be [B, Hkv, capacity, D/2]")
    B, H, C, half = shape
    at = k.get_device()
    sshape = (B, H, C, half // 16)
    if not (_fits(k, _U8, shape, at) and _fits(ks, _U8, sshape, at) and _fits(v, _U8, shape, at)
            and _fits(vs, _U8, sshape, at) and _fits(lens, _I32, (B,), at)
            and (w is None or _fits(w, _F32, (B, H, C), at))):
        _need(k, "cache.k", _U8, shape, k.device)
        _need(v, "cache.v", _U8, shape, k.device)
        _need(ks, "cache.k_scale", _U8, sshape, k.device)
        _need(vs, "cache.v_scale", _U8, sshape, k.device)
        _need(lens, "cache.seq_lens", _I32, (B,), k.device)
        if w is not None:
            _need(w, "cache.key_weight", _F32, (B, H, C), k.device)
    try:
        s = _pack_kv4(k.data_ptr(), ks.data_ptr(), v.data_ptr(), vs.data_ptr(),
                      0 if w is None else w.data_ptr(), lens.data_ptr(), B, C, H, 2 * half, kd, vd)
    except struct.error as e:
        raise ValueError(f"the sizes must fit 32 bits and the descales be numbers, got {kd} and {vd}") from e
    return s, at, B, H, C, 2 * half


def kv4_append(cache: KV4Cache, k: torch.Tensor, v: torch.Tensor, *, key_weight=None,
               cu_seqlens=None, seq_lens_out=None, stream=None) -> torch.Tensor:
    """Store new tokens' keys and values (bf16 or fp32, natural order) behind
    each sequence's cached ones: k, v [B,T,Hkv,D], or packed [T,Hkv,D] with
    cu_seqlens. key_weight: their attention weights so far ([B,Hkv,T], packed
    [Hkv,T], natural order: attn_key_weights, restored by permute if the layout is
    not contiguous), else 0. Returns the new lengths, written to
    seq_lens_out (default: the cache's own seq_lens, in place). Tokens that
    find no room are dropped."""
    s, at, B, H, _, D = _kv4_struct(cache)
    packed = cu_seqlens is not None
    dt = k.dtype
    if dt not in DTYPE:
        raise ValueError("keys and values must be bf16 or fp32")
    if k.dim() != (3 if packed else 4):
        raise ValueError("k must be [B, T, Hkv, D], packed [T, Hkv, D]")
    T = k.shape[0] if packed else k.shape[1]
    shape = (T, H, D) if packed else (B, T, H, D)
    _require(k, "k", dt, shape, at, cache.k)
    _require(v, "v", dt, shape, at, cache.k)
    if packed:
        _require(cu_seqlens, "cu_seqlens", _I32, (B + 1,), at, cache.k)
    if key_weight is not None:
        if cache.key_weight is None:
            raise ValueError("the cache has no key_weight to store the weights in")
        _require(key_weight, "key_weight", _F32, (H, T) if packed else (B, H, T), at,
                 cache.k)
    lens = cache.seq_lens
    if seq_lens_out is not None:
        lens = seq_lens_out
        _require(lens, "seq_lens_out", _I32, (B,), at, cache.k)
    _call(_lib.load().usp_kv4_append, at, stream, s, k.data_ptr(), v.data_ptr(),
          None if key_weight is None else key_weight.data_ptr(),
          cu_seqlens.data_ptr() if packed else None, T, DTYPE[dt], lens.data_ptr())
    return lens


def kv4_read(cache: KV4Cache, tokens: int, *, starts=None, dtype=torch.bfloat16, stream=None
             ) -> Tuple[torch.Tensor, torch.Tensor]:
    """(k, v) [B, tokens, Hkv, D]: the values of rows starts[b] (default 0) ..
    of every sequence; zeros behind its length."""
    if stream is not None:
        with _on(stream, cache.k.device):
            return kv4_read(cache, tokens, starts=starts, dtype=dtype)
    s, at, B, H, _, D = _kv4_struct(cache)
    if dtype not in DTYPE:
        raise ValueError("keys and values are read as bf16 or fp32")
    if starts is not None:
        _require(starts, "starts", _I32, (B,), at, cache.k)
    k = torch.empty((B, tokens, H, D), dtype=dtype, device=cache.k.device)
    v = torch.empty_like(k)
    _call(_lib.load().usp_kv4_read, at, None, s,
          None if starts is None else starts.data_ptr(), tokens, k.data_ptr(), v.data_ptr(),
          DTYPE[dtype])
    return k, v


def attn_decode_kv4(q: torch.Tensor, cache: KV4Cache, *, causal=True, window=0, sink_tokens=0,
                    accumulate=False, softmax_scale=0.0, workspace=None, stream=None
                    ) -> Tuple[torch.Tensor, torch.Tensor]:
    """(out [B,Tq,Hq,D], lse [B,Tq,Hq]) of the newest Tq tokens q [B,Tq,Hq,D]
    (already in the cache) against the cached keys; accumulate adds each key's
    attention weight of this step, among this cache's keys, to cache.key_weight."""
    if stream is not None:
        with _on(stream, q.device):
            return attn_decode_kv4(q, cache, causal=causal, window=window,
                                   sink_tokens=sink_tokens, accumulate=accumulate,
                                   softmax_scale=softmax_scale, workspace=workspace)
    s, at, B, Hkv, C, D = _kv4_struct(cache)
    _, Tq, Hq, _ = q.shape
    _require(q, "q", torch.bfloat16, (B, Tq, Hq, D), at, cache.k)
    if accumulate and cache.key_weight is None:
        raise ValueError("accumulate needs a cache with key_weight")
    lib = _lib.load()
    dev = q.device
    out = torch.empty_like(q)
    lse = torch.empty((B, Tq, Hq), dtype=_F32, device=dev)
    need = lib.usp_attn_decode_kv4_workspace_size(B, Tq, C, Hq, Hkv, D,
                                                  1 if accumulate else 0)
    ws = torch.empty(need, dtype=_U8, device=dev) if workspace is None else \
        _use_workspace(workspace, need, dev)[0]
    _call(lib.usp_attn_decode_kv4, at, None, s, q.data_ptr(), out.data_ptr(),
          lse.data_ptr(), Tq, Hq, softmax_scale, 1 if causal else 0, window, sink_tokens,
          1 if accumulate else 0, 0, ws.data_ptr(), ws.numel())
    return out, lse


def attn_key_weights(q, k, lse, *, causal=True, window=0, sink_tokens=0, cu_seqlens=None, cp=1,
                     layout="contiguous", observe=0, softmax_scale=0.0, flags=0, workspace=None,
                     stream=None) -> torch.Tensor:
    """[B,Hkv,S] fp32 (packed [Hkv,T]): the attention weight that each key
    collected from the observed queries (observe = n: the last n of each
    sequence; 0: all) and the query heads sharing its KV head, from the
    forward's q, k (rank-major) and lse; rank-major too (permute restores it)."""
    if stream is not None:
        with _on(stream, q.device):
            return attn_key_weights(q, k, lse, causal=causal, window=window,
                                    sink_tokens=sink_tokens, cu_seqlens=cu_seqlens, cp=cp,
                                    layout=layout, observe=observe, softmax_scale=softmax_scale,
                                    flags=flags, workspace=workspace)
    B, S, Hq, Hkv, D, Bl = _dims(q, k, cu_seqlens)
    at = q.get_device()
    dt = q.dtype
    if dt not in DTYPE:
        raise ValueError("q and k must be bf16 or fp32")
    lead = (Bl,) if cu_seqlens is None else ()
    _require(q, "q", dt, lead + (S, Hq, D), at, q)
    _require(k, "k", dt, lead + (S, Hkv, D), at, q)
    _require(lse, "lse", _F32, lead + (Hq, S), at, q)
    if cu_seqlens is not None:
        _require(cu_seqlens, "cu_seqlens", _I32, (B + 1,), at, q)
    lib = _lib.load()
    weight = torch.empty(lead + (Hkv, S), dtype=_F32, device=q.device)
    need = lib.usp_attn_key_weights_workspace_size(Bl, S, Hq, Hkv, observe, DTYPE[dt], flags)
    ws = workspace
    if ws is not None:
        ws = _use_workspace(ws, need, q.device)[0]
    elif need:
        ws = torch.empty(need, dtype=_U8, device=q.device)
    _call(lib.usp_attn_key_weights, at, None, q.data_ptr(), k.data_ptr(), lse.data_ptr(),
          weight.data_ptr(), B, S, Hq, Hkv, D, softmax_scale, 1 if causal else 0, window,
          sink_tokens, None if cu_seqlens is None else cu_seqlens.data_ptr(), cp,
          _enum(LAYOUT, layout), observe, DTYPE[dt], flags,
          None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel())
    return weight


def kv4_evict(cache: KV4Cache, keep: int, *, recent=0, sink_tokens=0, out=None, stream=None
              ) -> Tuple[KV4Cache, torch.Tensor]:
    """(cache, kept [B,Hkv,keep] int32): every sequence longer than `keep`
    keeps, in each KV head, its first sink_tokens, its last `recent` and the
    keys with the largest key_weight, in order; kept gives their old rows (-1
    behind the last). out: another cache that takes them (default: in place)."""
    if stream is not None:
        with _on(stream, cache.k.device):
            return kv4_evict(cache, keep, recent=recent, sink_tokens=sink_tokens, out=out)
    if cache.key_weight is None:
        raise ValueError("eviction needs a cache with key_weight")
    if keep < 1:
        raise ValueError("keep must be at least 1")
    s, at, B, H = _kv4_struct(cache)[:4]
    d, dst = s, cache
    if out is not None:
        dst = out
        d, at2 = _kv4_struct(out)[:2]
        if at2 != at:
            raise ValueError("both caches must be on one device")
        if (cache.k_descale, cache.v_descale) != (out.k_descale, out.v_descale):
            raise ValueError("both caches must have the same descales")
    kept = torch.empty((B, H, keep), dtype=_I32, device=cache.k.device)
    _call(_lib.load().usp_kv4_evict, at, None, s, d,
          kept.data_ptr(), keep, recent, sink_tokens)
    return dst, kept
