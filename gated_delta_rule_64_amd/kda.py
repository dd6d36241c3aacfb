"""Python binding of libkda: the same entry points, torch tensors in.

Argument marshalling only: shapes are read from the tensors, outputs that the
caller does not pass are allocated with torch (device memory is torch's
plumbing), and each call goes straight to the C ABI on torch's current HIP
stream.  Every step of the computation runs in libkda's kernels.
"""

from __future__ import annotations

import ctypes

import torch

from ._lib import KDA_BF16, KDA_F32, check, lib


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return KDA_F32
    if t.dtype == torch.bfloat16:
        return KDA_BF16
    raise TypeError(f"unsupported dtype {t.dtype}; libkda takes float32 or bfloat16")


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libkda takes device tensors")
    if not t.is_contiguous():
        raise ValueError("libkda takes contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream(device=None):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _n_seqs(cu_seqlens):
    if cu_seqlens is None:
        return 1
    if cu_seqlens.dtype != torch.int32:
        raise TypeError("cu_seqlens must be int32")
    return cu_seqlens.numel() - 1


def kda_preprocess(q_in, k_in, v_in, w_q, w_k, w_v, g_alpha, b_beta, H, dk, dv,
                   cu_seqlens=None, conv_state=None, out=None):
    """Short conv + L2 norm + gates.  Inputs [T, H*d]; returns
    (q [T,H,dk], k [T,H,dk], v [T,H,dv], log_alpha fp32 [T,H,dk], beta fp32 [T,H]).
    ``conv_state`` (fp32 [N, 3, H*(2dk+dv)]) is read and rewritten in place."""
    T = q_in.shape[0]
    x = _dtype_code(q_in)
    dev = q_in.device
    if out is None:
        out = (torch.empty((T, H, dk), dtype=q_in.dtype, device=dev),
               torch.empty((T, H, dk), dtype=q_in.dtype, device=dev),
               torch.empty((T, H, dv), dtype=q_in.dtype, device=dev),
               torch.empty((T, H, dk), dtype=torch.float32, device=dev),
               torch.empty((T, H), dtype=torch.float32, device=dev))
    q_o, k_o, v_o, la_o, b_o = out
    check(lib().kda_preprocess(T, H, dk, dv, _ptr(cu_seqlens), _n_seqs(cu_seqlens), x,
                               _ptr(q_in), _ptr(k_in), _ptr(v_in), _ptr(w_q), _ptr(w_k), _ptr(w_v),
                               _ptr(g_alpha), _ptr(b_beta), _ptr(conv_state),
                               _ptr(q_o), _ptr(k_o), _ptr(v_o), _ptr(la_o), _ptr(b_o), _stream(dev)))
    return out


def kda_prefill_workspace_bytes(T_tot, N, H, dk, dv, x_dtype):
    if isinstance(x_dtype, torch.dtype):
        x_dtype = KDA_BF16 if x_dtype == torch.bfloat16 else KDA_F32
    return int(lib().kda_prefill_workspace_bytes(T_tot, N, H, dk, dv, x_dtype))


def _snap_buffers(snap_interval, T, N, H, dk, dv, dev, snapshots, snap_offsets):
    cap = T // snap_interval
    if snapshots is None:
        snapshots = torch.empty((max(cap, 1), H, dk, dv), dtype=torch.float32, device=dev)
    if snap_offsets is None:
        snap_offsets = torch.empty(N + 1, dtype=torch.int32, device=dev)
    return snapshots, snap_offsets


def kda_prefill_chunked(q, k, v, log_alpha, beta, out_gate=None, initial_state=None,
                        final_state=None, cu_seqlens=None, workspace=None, out=None,
                        want_final_state=True, snap_interval=None, snapshots=None, snap_offsets=None):
    """Chunked recurrence over preprocessed tokens q,k [T,H,dk], v [T,H,dv].
    Returns (out [T,H,dv], final_state fp32 [N,H,dk,dv] or None); with
    ``snap_interval`` (a multiple of 64) also (snapshots [C,H,dk,dv],
    snap_offsets int32 [N+1]): the state after every ``snap_interval`` tokens
    of each sequence, sequence n's m-th at row snap_offsets[n] + m - 1."""
    T, H, dk = q.shape
    dv = v.shape[2]
    N = _n_seqs(cu_seqlens)
    x = _dtype_code(q)
    g = _dtype_code(log_alpha)
    dev = q.device
    if out is None:
        out = torch.empty((T, H, dv), dtype=q.dtype, device=dev)
    if final_state is None and want_final_state:
        final_state = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev)
    need = kda_prefill_workspace_bytes(T, N, H, dk, dv, x)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    if snap_interval is None:
        check(lib().kda_prefill_chunked(T, H, dk, dv, _ptr(cu_seqlens), N, x, g,
                                        _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                                        _ptr(out_gate), _ptr(initial_state), _ptr(final_state), _ptr(out),
                                        _ptr(workspace), workspace.numel(), _stream(dev)))
        return out, final_state
    snapshots, snap_offsets = _snap_buffers(snap_interval, T, N, H, dk, dv, dev, snapshots, snap_offsets)
    check(lib().kda_prefill_chunked_snap(T, H, dk, dv, _ptr(cu_seqlens), N, x, g,
                                         _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                                         _ptr(out_gate), _ptr(initial_state), _ptr(final_state), _ptr(out),
                                         _ptr(workspace), workspace.numel(), snap_interval, _ptr(snapshots),
                                         snapshots.shape[0], _ptr(snap_offsets), _stream(dev)))
    return out, final_state, snapshots, snap_offsets


def kda_decode_step(q, k, v, log_alpha, beta, state, out_gate=None, out=None):
    """One token per sequence; ``state`` fp32 [B,H,dk,dv] is updated in place.
    Returns out [B,H,dv]."""
    B, H, dk = q.shape
    dv = v.shape[2]
    if out is None:
        out = torch.empty((B, H, dv), dtype=q.dtype, device=q.device)
    check(lib().kda_decode_step(B, H, dk, dv, _dtype_code(q), _dtype_code(log_alpha),
                                _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(out_gate),
                                _ptr(state), _ptr(out), _stream(q.device)))
    return out


def kda_prefill_layer(q_in, k_in, v_in, w_q, w_k, w_v, g_alpha, b_beta, H, dk, dv, out_gate=None,
                      initial_state=None, final_state=None, cu_seqlens=None, conv_state=None, workspace=None,
                      out=None, want_final_state=True, snap_interval=None, snapshots=None, snap_offsets=None):
    """kda_preprocess + kda_prefill_chunked in one call (bf16, dk = dv = 128):
    raw inputs [T, H*d] as for kda_preprocess, the rest as for
    kda_prefill_chunked.  Returns (out [T,H,dv], final_state fp32 [N,H,dk,dv] or None).
    ``conv_state`` (fp32 [N, 3, H*(2dk+dv)]) is read and rewritten in place."""
    T = q_in.shape[0]
    N = _n_seqs(cu_seqlens)
    x = _dtype_code(q_in)
    dev = q_in.device
    if out is None:
        out = torch.empty((T, H, dv), dtype=q_in.dtype, device=dev)
    if final_state is None and want_final_state:
        final_state = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev)
    need = kda_prefill_workspace_bytes(T, N, H, dk, dv, x)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    if snap_interval is None:
        check(lib().kda_prefill_layer(T, H, dk, dv, _ptr(cu_seqlens), N, x,
                                      _ptr(q_in), _ptr(k_in), _ptr(v_in), _ptr(w_q), _ptr(w_k), _ptr(w_v),
                                      _ptr(g_alpha), _ptr(b_beta), _ptr(conv_state), _ptr(out_gate),
                                      _ptr(initial_state), _ptr(final_state), _ptr(out),
                                      _ptr(workspace), workspace.numel(), _stream(dev)))
        return out, final_state
    snapshots, snap_offsets = _snap_buffers(snap_interval, T, N, H, dk, dv, dev, snapshots, snap_offsets)
    check(lib().kda_prefill_layer_snap(T, H, dk, dv, _ptr(cu_seqlens), N, x,
                                       _ptr(q_in), _ptr(k_in), _ptr(v_in), _ptr(w_q), _ptr(w_k), _ptr(w_v),
                                       _ptr(g_alpha), _ptr(b_beta), _ptr(conv_state), _ptr(out_gate),
                                       _ptr(initial_state), _ptr(final_state), _ptr(out),
                                       _ptr(workspace), workspace.numel(), snap_interval, _ptr(snapshots),
                                       snapshots.shape[0], _ptr(snap_offsets), _stream(dev)))
    return out, final_state, snapshots, snap_offsets


def kda_prefill_layer_noalloc(q_in, k_in, v_in, w_q, w_k, w_v, g_alpha, b_beta, H, dk, dv, out_gate=None,
                              initial_state=None, final_state=None, cu_seqlens=None, conv_state=None, out=None,
                              want_final_state=True):
    """kda_prefill_layer without a workspace: the library's fixed scratch
    (KDA_NOALLOC_SCRATCH_BYTES per GPU) holds it.  Returns (out, final_state)."""
    T = q_in.shape[0]
    N = _n_seqs(cu_seqlens)
    x = _dtype_code(q_in)
    dev = q_in.device
    if out is None:
        out = torch.empty((T, H, dv), dtype=q_in.dtype, device=dev)
    if final_state is None and want_final_state:
        final_state = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev)
    check(lib().kda_prefill_layer_noalloc(T, H, dk, dv, _ptr(cu_seqlens), N, x,
                                          _ptr(q_in), _ptr(k_in), _ptr(v_in), _ptr(w_q), _ptr(w_k), _ptr(w_v),
                                          _ptr(g_alpha), _ptr(b_beta), _ptr(conv_state), _ptr(out_gate),
                                          _ptr(initial_state), _ptr(final_state), _ptr(out), _stream(dev)))
    return out, final_state


def kda_decode_layer(q_in, k_in, v_in, w_q, w_k, w_v, g_alpha, b_beta, H, dk, dv, conv_state, state,
                     out_gate=None, state_indices=None, out=None):
    """One raw token per sequence through preprocess + decode step in one call.
    Inputs [B, H*d] (or [B, H, d]) as for kda_preprocess; ``conv_state`` fp32
    [S, 3, H*(2dk+dv)] and ``state`` fp32 [S, H, dk, dv] are pools updated in
    place, sequence b using row ``state_indices[b]`` (int32 [B]; row b when
    None, then S must be B; an index outside [0, S) marks a padding row whose
    output is zero).  Returns out [B, H, dv]."""
    B = q_in.shape[0]
    slots = state.shape[0]
    if state_indices is not None and state_indices.dtype != torch.int32:
        raise TypeError("state_indices must be int32")
    if out is None:
        out = torch.empty((B, H, dv), dtype=q_in.dtype, device=q_in.device)
    check(lib().kda_decode_layer(B, H, dk, dv, _dtype_code(q_in),
                                 _ptr(q_in), _ptr(k_in), _ptr(v_in), _ptr(w_q), _ptr(w_k), _ptr(w_v),
                                 _ptr(g_alpha), _ptr(b_beta), _ptr(conv_state), _ptr(out_gate),
                                 _ptr(state), slots, _ptr(state_indices), _ptr(out), _stream(q_in.device)))
    return out


def kda_spec_draft_bytes(H, dk, dv, x_dtype):
    """Bytes of draft buffer per pool slot for kda_spec_verify."""
    if isinstance(x_dtype, torch.dtype):
        x_dtype = KDA_BF16 if x_dtype == torch.bfloat16 else KDA_F32
    return int(lib().kda_spec_draft_bytes(H, dk, dv, x_dtype))


def kda_spec_verify(q_in, k_in, v_in, w_q, w_k, w_v, g_alpha, b_beta, H, dk, dv, conv_state, state, drafts,
                    accepted=None, out_gate=None, state_indices=None, out=None):
    """Commit ``accepted[b]`` tokens of the previous call, then run the T new
    raw tokens (inputs [B, T, H*d] or [B, T, H, d]) from that state without
    advancing it.  ``drafts`` is a device buffer of S * kda_spec_draft_bytes
    bytes (S = pool rows).  Returns out [B, T, H, dv]."""
    B, T = q_in.shape[0], q_in.shape[1]
    for t in (accepted, state_indices):
        if t is not None and t.dtype != torch.int32:
            raise TypeError("accepted and state_indices must be int32")
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=q_in.dtype, device=q_in.device)
    check(lib().kda_spec_verify(B, T, H, dk, dv, _dtype_code(q_in),
                                _ptr(q_in), _ptr(k_in), _ptr(v_in), _ptr(w_q), _ptr(w_k), _ptr(w_v),
                                _ptr(g_alpha), _ptr(b_beta), _ptr(conv_state), _ptr(out_gate),
                                _ptr(state), state.shape[0], _ptr(state_indices), _ptr(accepted),
                                _ptr(drafts), _ptr(out), _stream(q_in.device)))
    return out


def kda_backward_workspace_bytes(T_tot, N, H, dk, dv):
    return int(lib().kda_backward_workspace_bytes(T_tot, N, H, dk, dv))


def kda_prefill_backward(q, k, v, log_alpha, beta, dy, out_gate=None, initial_state=None, dS_final=None,
                         cu_seqlens=None, workspace=None, want_dS0=True):
    """Gradients of kda_prefill_chunked for output gradients dy [T,H,dv] (and
    dS_final on the final states).  Returns a dict of fp32 tensors dq, dk,
    dlog_alpha [T,H,dk], dv [T,H,dv], dbeta [T,H], dz (None without a gate)
    and dS0 [N,H,dk,dv] (None if not wanted)."""
    T, H, dk = q.shape
    dv = v.shape[2]
    N = _n_seqs(cu_seqlens)
    dev = q.device
    f32 = dict(dtype=torch.float32, device=dev)
    g = {"dq": torch.empty((T, H, dk), **f32), "dk": torch.empty((T, H, dk), **f32),
         "dv": torch.empty((T, H, dv), **f32), "dlog_alpha": torch.empty((T, H, dk), **f32),
         "dbeta": torch.empty((T, H), **f32),
         "dz": torch.empty((T, H, dv), **f32) if out_gate is not None else None,
         "dS0": torch.empty((N, H, dk, dv), **f32) if want_dS0 else None}
    need = kda_backward_workspace_bytes(T, N, H, dk, dv)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    check(lib().kda_prefill_backward(T, H, dk, dv, _ptr(cu_seqlens), N, _dtype_code(q), _dtype_code(log_alpha),
                                     _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(out_gate),
                                     _ptr(initial_state), _ptr(dy), _ptr(dS_final),
                                     _ptr(g["dq"]), _ptr(g["dk"]), _ptr(g["dv"]), _ptr(g["dlog_alpha"]),
                                     _ptr(g["dbeta"]), _ptr(g["dz"]), _ptr(g["dS0"]),
                                     _ptr(workspace), workspace.numel(), _stream(dev)))
    return g


def _device(*tensors):
    """The one device of a call's tensors (None entries are skipped)."""
    dev = tensors[0].device
    for t in tensors:
        if t is not None and t.device != dev:
            raise ValueError(f"tensors on {dev} and {t.device} in one call")
    if dev.type != "cuda":
        raise ValueError("libkda takes device tensors")
    return dev


def _shape(name, t, shape, dtype):
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} is {t.dtype}, expected {dtype}")


# the current stream's handle without the wrapper object that
# torch.cuda.current_stream makes (3 of the 12 us of a small call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _addr(t):
    """A tensor's device address as a plain number (None stays None), for
    arguments that ctypes already takes as pointers.  _device has seen that it
    is a device tensor."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("libkda takes contiguous tensors")
    return t.data_ptr()


def _call(dev, name, *args):
    """One call of the library on the device's current stream."""
    fn, index = getattr(lib(), name), dev.index
    if index == torch.cuda.current_device():
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(index))
    if status != 0:
        check(status)


def _workspace(workspace, need, dev):
    if workspace is None:
        return torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    if workspace.dtype != torch.uint8:
        raise TypeError("workspace must be uint8")
    return workspace


def _attn_shapes(q, k, v, out_gate, cu_seqlens):
    """Sizes of a packed attention batch, every tensor checked against them."""
    T, H, dk = q.shape
    Hkv, dv = k.shape[1], v.shape[2]
    _shape("k", k, (T, Hkv, dk), q.dtype)
    _shape("v", v, (T, Hkv, dv), q.dtype)
    if out_gate is not None:
        _shape("out_gate", out_gate, (T, H, dv), q.dtype)
    return T, H, Hkv, dk, dv, _n_seqs(cu_seqlens)


def kda_attn_prefill(q, k, v, out_gate=None, cu_seqlens=None, scale=None, out=None, lse=None):
    """Causal attention over packed prompts: q [T,H,dk], k [T,Hkv,dk], v
    [T,Hkv,dv]; ``scale`` defaults to dk^-0.5.  Returns (out [T,H,dv], lse
    fp32 [T,H]).  Rows behind cu_seqlens[-1] are left as they were."""
    T, H, Hkv, dk, dv, N = _attn_shapes(q, k, v, out_gate, cu_seqlens)
    dev = _device(q, k, v, out_gate, cu_seqlens, out, lse)
    if out is None:
        out = torch.empty((T, H, dv), dtype=q.dtype, device=dev)
    else:
        _shape("out", out, (T, H, dv), q.dtype)
    if lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=dev)
    else:
        _shape("lse", lse, (T, H), torch.float32)
    _call(dev, "kda_attn_prefill", T, H, Hkv, dk, dv, _addr(cu_seqlens), N, _dtype_code(q),
          dk ** -0.5 if scale is None else scale, _addr(q), _addr(k), _addr(v), _addr(out_gate), _addr(out), _addr(lse))
    return out, lse


def kda_attn_backward_workspace_bytes(T_tot, N, H, Hkv, dk, dv, x_dtype, with_gate):
    if isinstance(x_dtype, torch.dtype):
        x_dtype = KDA_BF16 if x_dtype == torch.bfloat16 else KDA_F32
    return int(lib().kda_attn_backward_workspace_bytes(T_tot, N, H, Hkv, dk, dv, x_dtype, int(bool(with_gate))))


def kda_attn_backward_max_workspace_bytes(max_T_tot, H, Hkv, dk, dv, x_dtype, with_gate):
    """What every call of up to ``max_T_tot`` tokens needs at most (a call of
    fewer tokens can need more than a larger one)."""
    if isinstance(x_dtype, torch.dtype):
        x_dtype = KDA_BF16 if x_dtype == torch.bfloat16 else KDA_F32
    return int(lib().kda_attn_backward_max_workspace_bytes(max_T_tot, H, Hkv, dk, dv, x_dtype, int(bool(with_gate))))


def kda_attn_prefill_backward(q, k, v, out, lse, dy, out_gate=None, cu_seqlens=None, scale=None, workspace=None):
    """Gradients of kda_attn_prefill for output gradients dy [T,H,dv]; ``out``
    and ``lse`` are what it returned.  Returns a dict of dq [T,H,dk], dk
    [T,Hkv,dk], dv [T,Hkv,dv] and dz [T,H,dv] (None without a gate) in q's
    type.  Rows behind cu_seqlens[-1] are not written."""
    T, H, Hkv, dk, dv, N = _attn_shapes(q, k, v, out_gate, cu_seqlens)
    dev = _device(q, k, v, out, lse, dy, out_gate, cu_seqlens, workspace)
    for name, t in (("out", out), ("dy", dy)):
        _shape(name, t, (T, H, dv), q.dtype)
    _shape("lse", lse, (T, H), torch.float32)
    x = _dtype_code(q)
    g = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v),
         "dz": torch.empty_like(out_gate) if out_gate is not None else None}
    need = kda_attn_backward_workspace_bytes(T, N, H, Hkv, dk, dv, x, out_gate is not None)
    workspace = _workspace(workspace, need, dev)
    _call(dev, "kda_attn_prefill_backward", T, H, Hkv, dk, dv, _addr(cu_seqlens), N, x,
          dk ** -0.5 if scale is None else scale, _addr(q), _addr(k), _addr(v), _addr(out_gate), _addr(out), _addr(lse),
          _addr(dy), _addr(g["dq"]), _addr(g["dk"]), _addr(g["dv"]), _addr(g["dz"]), _addr(workspace), workspace.numel())
    return g


def _cache_shapes(k_cache, v_cache, page_table):
    """(num_pages, Hkv, page_size, dk, dv, slots, max_pages) of a cache."""
    pages, Hkv, page, dk = k_cache.shape
    dv = v_cache.shape[3]
    _shape("v_cache", v_cache, (pages, Hkv, page, dv), k_cache.dtype)
    slots, width = page_table.shape
    _shape("page_table", page_table, (slots, width), torch.int32)
    return pages, Hkv, page, dk, dv, slots, width


def kda_attn_tree_workspace_bytes(B, T, H, Hkv, dk, dv, x_dtype, max_context):
    """``max_context``: tokens that a page-table row can hold."""
    if isinstance(x_dtype, torch.dtype):
        x_dtype = KDA_BF16 if x_dtype == torch.bfloat16 else KDA_F32
    return int(lib().kda_attn_tree_workspace_bytes(B, T, H, Hkv, dk, dv, x_dtype, max_context))


def kda_attn_tree_max_workspace_bytes(max_B, max_T, H, Hkv, dk, dv, x_dtype, max_context):
    """What every call of up to ``max_B`` sequences of up to ``max_T`` tokens
    needs at most (a call of fewer sequences can need more than a larger one)."""
    if isinstance(x_dtype, torch.dtype):
        x_dtype = KDA_BF16 if x_dtype == torch.bfloat16 else KDA_F32
    return int(lib().kda_attn_tree_max_workspace_bytes(max_B, max_T, H, Hkv, dk, dv, x_dtype, max_context))


def kda_attn_tree(q, k_new, v_new, k_cache, v_cache, page_table, lens, tree_mask=None, out_gate=None,
                  slot_indices=None, scale=None, workspace=None, out=None, lse=None):
    """Drafted tokens q [B,T,H,dk] (T <= 64; T = 1 is plain decode) over the
    paged cache and over each other: ``tree_mask`` int64 [B,T], bit j of word
    t set where token t attends draft j (None: a chain).  k_new [B,T,Hkv,dk]
    and v_new [B,T,Hkv,dv] are the drafts' own keys and values, not yet in the
    cache.  Sequence b uses slot ``slot_indices[b]`` (None: b) of page_table
    int32 [S,max_pages] and lens int32 [S]; an index outside [0, S) marks a
    padding row, whose output is zero.  Returns (out [B,T,H,dv], lse fp32
    [B,T,H])."""
    B, T, H, dk = q.shape
    pages, Hkv, page, _, dv, slots, width = _cache_shapes(k_cache, v_cache, page_table)
    _shape("k_cache", k_cache, (pages, Hkv, page, dk), q.dtype)
    _shape("k_new", k_new, (B, T, Hkv, dk), q.dtype)
    _shape("v_new", v_new, (B, T, Hkv, dv), q.dtype)
    _shape("lens", lens, (slots,), torch.int32)
    if tree_mask is not None:
        _shape("tree_mask", tree_mask, (B, T), torch.int64)
    if out_gate is not None:
        _shape("out_gate", out_gate, (B, T, H, dv), q.dtype)
    if slot_indices is not None:
        _shape("slot_indices", slot_indices, (B,), torch.int32)
    dev = _device(q, k_new, v_new, k_cache, v_cache, page_table, lens, tree_mask, out_gate, slot_indices, workspace,
                  out, lse)
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=q.dtype, device=dev)
    else:
        _shape("out", out, (B, T, H, dv), q.dtype)
    if lse is None:
        lse = torch.empty((B, T, H), dtype=torch.float32, device=dev)
    else:
        _shape("lse", lse, (B, T, H), torch.float32)
    x = _dtype_code(q)
    workspace = _workspace(workspace, kda_attn_tree_workspace_bytes(B, T, H, Hkv, dk, dv, x, width * page), dev)
    _call(dev, "kda_attn_tree", B, T, H, Hkv, dk, dv, x, dk ** -0.5 if scale is None else scale,
          _addr(q), _addr(k_new), _addr(v_new), _addr(tree_mask), _addr(out_gate), _addr(k_cache), _addr(v_cache), pages, page,
          _addr(page_table), slots, width, _addr(lens), _addr(slot_indices), _addr(out), _addr(lse),
          _addr(workspace), workspace.numel())
    return out, lse


def kda_cache_append(k_new, v_new, k_cache, v_cache, page_table, lens, cu_seqlens=None, rows=None, slot_indices=None):
    """Writes new tokens' keys and values k_new [R,Hkv,dk], v_new [R,Hkv,dv]
    into the cache: sequence n's tokens cu_seqlens[n] .. cu_seqlens[n+1] - 1
    go behind the lens[slot] tokens that its slot (``slot_indices[n]``, or n)
    holds; token t comes from row ``rows[t]`` (int32; None: row t).  lens is
    not advanced."""
    pages, Hkv, page, dk, dv, slots, width = _cache_shapes(k_cache, v_cache, page_table)
    R, N = k_new.shape[0], _n_seqs(cu_seqlens)
    _shape("k_new", k_new, (R, Hkv, dk), k_cache.dtype)
    _shape("v_new", v_new, (R, Hkv, dv), k_cache.dtype)
    _shape("lens", lens, (slots,), torch.int32)
    T = R
    if rows is not None:
        T = rows.numel()
        _shape("rows", rows, (T,), torch.int32)
    if slot_indices is not None:
        _shape("slot_indices", slot_indices, (N,), torch.int32)
    dev = _device(k_new, v_new, k_cache, v_cache, page_table, lens, cu_seqlens, rows, slot_indices)
    _call(dev, "kda_cache_append", T, N, _addr(cu_seqlens), R, _addr(rows), Hkv, dk, dv, _dtype_code(k_cache),
          _addr(k_new), _addr(v_new), _addr(k_cache), _addr(v_cache), pages, page, _addr(page_table), slots, width,
          _addr(lens), _addr(slot_indices))


def kda_cache_workspace_bytes(num_pages, slots, n):
    return int(lib().kda_cache_workspace_bytes(num_pages, slots, n))


def _slot_list(name, t):
    _shape(name, t, (t.numel(),), torch.int32)
    return t.numel()


def _status(status, n, dev):
    if status is None:
        return torch.empty(n, dtype=torch.int32, device=dev)
    _shape("status", status, (n,), torch.int32)
    return status


def kda_cache_free(slot_list, page_table, lens, refs):
    """Empties the slots of ``slot_list`` (int32 [n]); pages that no other
    slot names become free."""
    n = _slot_list("slot_list", slot_list)
    slots, width = page_table.shape
    _shape("page_table", page_table, (slots, width), torch.int32)
    _shape("lens", lens, (slots,), torch.int32)
    _shape("refs", refs, (refs.numel(),), torch.int32)
    dev = _device(slot_list, page_table, lens, refs)
    _call(dev, "kda_cache_free", n, _addr(slot_list), refs.numel(), _addr(page_table), slots, width, _addr(lens), _addr(refs))


def kda_cache_fork(src, dst, k_cache, v_cache, page_table, lens, refs, status=None, workspace=None):
    """Slot dst[i] (empty) becomes a copy of slot src[i]: full pages shared,
    the rows of a partly filled last page copied.  Returns status int32 [n]:
    0 done, 1 too few free pages, 2 refused."""
    pages, Hkv, page, dk, dv, slots, width = _cache_shapes(k_cache, v_cache, page_table)
    n = _slot_list("src", src)
    _shape("dst", dst, (n,), torch.int32)
    _shape("lens", lens, (slots,), torch.int32)
    _shape("refs", refs, (pages,), torch.int32)
    dev = _device(src, dst, k_cache, v_cache, page_table, lens, refs, status, workspace)
    status = _status(status, n, dev)
    workspace = _workspace(workspace, kda_cache_workspace_bytes(pages, slots, n), dev)
    _call(dev, "kda_cache_fork", n, _addr(src), _addr(dst), Hkv, dk, dv, _dtype_code(k_cache), _addr(k_cache), _addr(v_cache),
          pages, page, _addr(page_table), slots, width, _addr(lens), _addr(refs), _addr(status), _addr(workspace),
          workspace.numel())
    return status


def kda_cache_reserve(slot_list, new_lens, page_size, page_table, lens, refs, status=None, workspace=None):
    """Gives every listed slot the pages that it lacks behind its length for
    new_lens[i] tokens.  Returns status int32 [n]: 0 done, 1 too few free
    pages, 2 refused."""
    n = _slot_list("slot_list", slot_list)
    _shape("new_lens", new_lens, (n,), torch.int32)
    slots, width = page_table.shape
    _shape("page_table", page_table, (slots, width), torch.int32)
    _shape("lens", lens, (slots,), torch.int32)
    _shape("refs", refs, (refs.numel(),), torch.int32)
    dev = _device(slot_list, new_lens, page_table, lens, refs, status, workspace)
    status = _status(status, n, dev)
    workspace = _workspace(workspace, kda_cache_workspace_bytes(refs.numel(), slots, n), dev)
    _call(dev, "kda_cache_reserve", n, _addr(slot_list), _addr(new_lens), refs.numel(), page_size, _addr(page_table), slots,
          width, _addr(lens), _addr(refs), _addr(status), _addr(workspace), workspace.numel())
    return status


def kda_cache_compact(k_cache, v_cache, page_table, refs, live=None, workspace=None):
    """Moves the pages in use to the front of the pool.  Returns ``live``
    int32 [1], how many there are (pages from there on are free)."""
    pages, Hkv, page, dk, dv, slots, width = _cache_shapes(k_cache, v_cache, page_table)
    _shape("refs", refs, (pages,), torch.int32)
    dev = _device(k_cache, v_cache, page_table, refs, live, workspace)
    if live is None:
        live = torch.empty(1, dtype=torch.int32, device=dev)
    else:
        _shape("live", live, (1,), torch.int32)
    workspace = _workspace(workspace, kda_cache_workspace_bytes(pages, slots, 0), dev)
    _call(dev, "kda_cache_compact", Hkv, dk, dv, _dtype_code(k_cache), _addr(k_cache), _addr(v_cache), pages, page,
          _addr(page_table), slots, width, _addr(refs), _addr(live), _addr(workspace), workspace.numel())
    return live


def kda_cache_copy(pool, src, dst):
    """Row dst[i] of ``pool`` (any type, [rows, ...]) becomes a copy of row
    src[i] (int32 lists): pages of a cache, or rows of the KDA state and
    conv-history pools of a sequence that is forked."""
    n = _slot_list("src", src)
    _shape("dst", dst, (n,), torch.int32)
    rows = pool.shape[0]
    row_bytes = pool.numel() // max(rows, 1) * pool.element_size()
    dev = _device(pool, src, dst)
    _call(dev, "kda_cache_copy", _addr(pool), row_bytes, rows, _addr(src), _addr(dst), n)


def kda_probe_peak(kind, blocks, iters=0, src=None, out=None):
    """Peak-rate probe (see kda.h): kind 0 bf16 matrix-core loop, 1 fp32
    matrix-core loop, 2 streaming read of ``src``.  Returns ``out``."""
    dev = src.device if src is not None else torch.device("cuda")
    if out is None:
        out = torch.empty(blocks * 256, dtype=torch.float32, device=dev)
    nbytes = src.numel() * src.element_size() if src is not None else 0
    check(lib().kda_probe_peak(kind, blocks, iters, _ptr(src), nbytes, _ptr(out), _stream(dev)))
    return out
