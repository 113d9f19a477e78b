"""Convenience calls over the binding: allocate outputs and workspace with torch, then call
the C entry point.  Shapes and semantics are those of include/dspark.h."""
from __future__ import annotations

import torch

from . import binding as b


def _wdt(W1):
    return b.F32 if W1 is None else b.dtype_code(W1.dtype)


def make_params(base: torch.Tensor, W1, T: float, seed: int, softcap: float = 0.0) -> b.SampleParams:
    B, gamma, V = base.shape
    r = 0 if W1 is None else W1.shape[1]
    return b.params(B, gamma, V, r, T, seed, b.dtype_code(base.dtype), _wdt(W1), softcap)


def markov_sample_block(base, W1, W2, anchor, T, seed, ws=None, out=None, stream=None, softcap=0.0):
    """Returns (tokens [B,gamma] int32, draft_lse [B,gamma] f32, z_at_tok [B,gamma] f32, workspace)."""
    p = make_params(base, W1, T, seed, softcap)
    B, gamma, _ = base.shape
    dev = base.device
    if out is None:
        out = (torch.empty((B, gamma), dtype=torch.int32, device=dev), torch.empty((B, gamma), device=dev),
               torch.empty((B, gamma), device=dev))
    if ws is None:
        ws = b.workspace(b.dspark_sample_workspace_size(p), dev)
    b.dspark_markov_sample_block(p, base, W1, W2, anchor, out[0], out[1], out[2], ws, stream)
    return out[0], out[1], out[2], ws


def verify(base, W1, W2, anchor, tokens, draft_lse, z_at_tok, target, T, seed, verify_len=None,
           target_row_offsets=None, ws=None, out=None, stream=None, softcap=0.0):
    """Returns (n_accepted [B] int32, correction_token [B] int32, workspace)."""
    p = make_params(base, W1, T, seed, softcap)
    B = base.shape[0]
    gamma_t = 0 if target_row_offsets is not None else target.shape[1]
    dev = base.device
    if out is None:
        out = (torch.empty(B, dtype=torch.int32, device=dev), torch.empty(B, dtype=torch.int32, device=dev))
    if ws is None:
        ws = b.workspace(b.dspark_verify_workspace_size(p, gamma_t), dev)
    b.dspark_verify(p, base, W1, W2, anchor, tokens, draft_lse, z_at_tok, target, gamma_t, verify_len,
                    target_row_offsets, out[0], out[1], ws, stream)
    return out[0], out[1], ws


def markov_sample_block_head(base, W1, W2, anchor, T, seed, kind, hidden, Wg, Wc=None, Wo=None, ws=None,
                             out=None, stream=None, softcap=0.0):
    """Gated / RNN head sampling.  Returns (tokens, draft_lse, z_at_tok, head_vec [B,gamma,r] f32, workspace)."""
    p = make_params(base, W1, T, seed, softcap)
    B, gamma, _ = base.shape
    dev = base.device
    h = b.head(kind, hidden, Wg, Wc, Wo)
    if out is None:
        out = (torch.empty((B, gamma), dtype=torch.int32, device=dev), torch.empty((B, gamma), device=dev),
               torch.empty((B, gamma), device=dev), torch.empty((B, gamma, W1.shape[1]), device=dev))
    if ws is None:
        ws = b.workspace(b.dspark_sample_head_workspace_size(p, h), dev)
    b.dspark_markov_sample_block_head(p, h, base, W1, W2, anchor, out[0], out[1], out[2], out[3], ws, stream)
    return out[0], out[1], out[2], out[3], ws


def verify_head(base, head_vec, W2, anchor, tokens, draft_lse, z_at_tok, target, T, seed, verify_len=None,
                target_row_offsets=None, ws=None, out=None, stream=None, softcap=0.0):
    """dspark_verify for Gated / RNN drafts: q is rebuilt from head_vec [B,gamma,r] f32.
    Returns (n_accepted, correction_token, workspace)."""
    B, gamma, V = base.shape
    r = head_vec.shape[-1]
    p = b.params(B, gamma, V, r, T, seed, b.dtype_code(base.dtype), b.dtype_code(W2.dtype), softcap)
    gamma_t = 0 if target_row_offsets is not None else target.shape[1]
    dev = base.device
    if out is None:
        out = (torch.empty(B, dtype=torch.int32, device=dev), torch.empty(B, dtype=torch.int32, device=dev))
    if ws is None:
        ws = b.workspace(b.dspark_verify_workspace_size(p, gamma_t), dev)
    b.dspark_verify_head(p, base, head_vec, W2, anchor, tokens, draft_lse, z_at_tok, target, gamma_t, verify_len,
                         target_row_offsets, out[0], out[1], ws, stream)
    return out[0], out[1], ws


def accept_rate_tv(d, t, keep, pos_valid=None, want_tau=True, ws=None, out=None, stream=None):
    """d, t [S,A,gamma,V]; keep [S,A] uint8.  Returns (accept_rate, eval_mask, tau or None, workspace)."""
    S, A, gamma, V = d.shape
    dt = b.dtype_code(d.dtype)
    dev = d.device
    if out is None:
        out = (torch.empty((S, A, gamma), device=dev), torch.empty((S, A, gamma), device=dev),
               torch.empty((S, A), device=dev) if want_tau else None)
    if ws is None:
        ws = b.workspace(b.dspark_accept_rate_tv_workspace_size(S, A, gamma, V, dt), dev)
    b.dspark_accept_rate_tv(S, A, gamma, V, dt, d, t, keep, pos_valid, out[0], out[1], out[2], ws, stream)
    return out[0], out[1], out[2], ws


def markov_block_logits(base, W1, W2, anchor, tokens, stream=None, softcap=0.0):
    """Teacher-forced z = base + W2 W1[prev] at every position.  base [B,gamma,V]; returns z [B,gamma,V] f32."""
    p = make_params(base, W1, 1.0, 0, softcap)
    B, gamma, V = base.shape
    z = torch.empty((B, gamma, V), dtype=torch.float32, device=base.device)
    ws = b.workspace(b.dspark_markov_block_logits_workspace_size(p), base.device)
    b.dspark_markov_block_logits(p, base, W1, W2, anchor, tokens, z, ws, stream)
    return z, ws


def tv_l1_loss(accept_rate, eval_mask, decay_gamma=4.0, stream=None):
    """accept_rate, eval_mask [S,A,gamma] f32.  Returns (l1 [S,A,gamma] f32, sums [2] f64: weighted numerator, denominator)."""
    S, A, gamma = accept_rate.shape
    l1 = torch.empty_like(accept_rate)
    sums = torch.empty(2, dtype=torch.float64, device=accept_rate.device)
    b.dspark_tv_l1_loss(S, A, gamma, accept_rate, eval_mask, decay_gamma, l1, sums, stream)
    return l1, sums


def theta_schedule(conf, sps, with_theta=False, stream=None):
    """conf [B,gamma] f32, sps [gamma+1] f32 (device).  Returns (ell [B] int32, theta [B,gamma+1] f32 or None)."""
    B, gamma = conf.shape
    dev = conf.device
    ell = torch.empty(B, dtype=torch.int32, device=dev)
    theta = torch.empty((B, gamma + 1), dtype=torch.float32, device=dev) if with_theta else None
    b.dspark_theta_schedule(B, gamma, conf, sps, ell, theta, stream)
    return ell, theta


def schedule_verify_len(conf, budget, ws=None, out=None, stream=None):
    """conf [B,gamma] f32.  Returns (verify_len [B], offsets [B+1], objective [1], workspace)."""
    B, gamma = conf.shape
    dev = conf.device
    if out is None:
        out = (torch.empty(B, dtype=torch.int32, device=dev), torch.empty(B + 1, dtype=torch.int32, device=dev),
               torch.empty(1, device=dev))
    if ws is None:
        ws = b.workspace(b.dspark_schedule_workspace_size(B, gamma), dev)
    b.dspark_schedule_verify_len(B, gamma, conf, budget, out[0], out[1], out[2], ws, stream)
    return out[0], out[1], out[2], ws


# ------------------------------------------------------------------ the paged key-value cache
# The tensors are checked in csrc/native.cpp, on their way into the library.
_WS = b.CacheParams(1, 1, 1, 1, 0, 0)  # cache_plan's and cache_commit's workspace does not depend on the sizes


def _raw(stream, *made):
    """The stream's address.  Tensors made here for a call on a stream of its own stay reserved for it."""
    if stream is None:
        return None
    kept = [t for t in made if t is not None]
    if kept:
        on = b.torch_stream(stream)
        for t in kept:
            t.record_stream(on)
    return b._stream(stream)


def _cache_ws(ws, like):
    return b.workspace(b.dspark_cache_workspace_size(_WS), like.device) if ws is None else ws


def cache_plan(cache_len, new_len, block_table, n_blocks, free_pages, n_free, page_size, max_tokens, extra=0,
               positions=True, out=None, ws=None, stream=None, error=None):
    """A step's pages, slots and offsets from the requests' lengths (dspark_cache_plan): cache_len, new_len (or
    None), n_blocks [B], free_pages [pages], n_free [1], all int32; block_table [B, max_blocks] int32 gains the new
    pages.  Returns (seq_len [B], offsets [B+1], slots [max_tokens] int64, positions [max_tokens] or None,
    n_blocks [B], n_free [1], workspace); n_blocks and n_free are new tensors.  error [1] int32, or None: the
    caller's, in which the first device error of its calls stays until it is cleared."""
    made = ()
    if out is None:
        B, i32 = cache_len.numel(), {"dtype": torch.int32, "device": cache_len.device}
        made = out = (torch.empty(B, **i32), torch.empty(B + 1, **i32), torch.empty(max_tokens, dtype=torch.int64, device=i32["device"]),
                      torch.empty(max_tokens, **i32) if positions else None, torch.empty(B, **i32), torch.empty(1, **i32))
    ws = _cache_ws(ws, cache_len)
    st = b.native().cache_plan(cache_len, new_len, block_table, n_blocks, free_pages, n_free, page_size, max_tokens, extra, *out,
                               ws, _raw(stream, ws, *made), error)
    b._check(st, "dspark_cache_plan")
    return (*out, ws)


def cache_commit(cache_len, add_len, block_table, n_blocks, free_pages, n_free, page_size, extra=0, done=None, out=None,
                 ws=None, stream=None, error=None, settled=None):
    """The requests' lengths after the verification, and the pages past them back on the stack
    (dspark_cache_commit): add_len [B] int32 (n_accepted) or None, done [B] uint8 or bool, or None; free_pages is
    written in place.  Returns (cache_len [B], n_blocks [B], n_free [1], workspace), new tensors.  error as for
    cache_plan.  settled [2 B + 1] int32, or None: gets the three once more, and may hold the inputs cache_len, n_blocks
    and n_free themselves."""
    made = ()
    if out is None:
        B, i32 = cache_len.numel(), {"dtype": torch.int32, "device": cache_len.device}
        made = out = (torch.empty(B, **i32), torch.empty(B, **i32), torch.empty(1, **i32))
    ws = _cache_ws(ws, cache_len)
    st = b.native().cache_commit(cache_len, add_len, done, block_table, n_blocks, free_pages, n_free, page_size, extra, *out, ws,
                                 _raw(stream, ws, *made), error, settled)
    b._check(st, "dspark_cache_commit")
    return (*out, ws)


def cache_append(k, v, k_pages, v_pages, slots, k_scale=None, v_scale=None, stream=None):
    """Writes k, v [T, Hk, D] (bf16 or fp16; any strides with a dense last dimension) to their slots [T] int64 of
    k_pages, v_pages [pages, page_size, Hk, D] (their type, or e4m3 with k_scale, v_scale [Hk] fp32)."""
    b._check(b.native().cache_append(k, v, k_pages, v_pages, slots, k_scale, v_scale, _raw(stream)), "dspark_cache_append")


def _attention_sizes(q, k_pages, seq_len, max_new):
    """The parameters that decide the workspace's size."""
    T, Hq, D = q.shape
    return b.AttentionParams(T, seq_len.numel(), Hq, k_pages.shape[2], D, 1, 1, 1, max_new, b.cache_dtype_code(q.dtype),
                             b.cache_dtype_code(k_pages.dtype), 1, 0, 1.0, 0.0, 0, 0, 0, 0, 0)


def paged_attention(q, k_pages, v_pages, block_table, seq_len, offsets=None, scale=None, causal=True, window=0,
                    softcap=0.0, k_scale=None, v_scale=None, max_new=0, out=None, lse=None, ws=None, stream=None, error=None):
    """Attention of the new tokens q [T, Hq, D] over the paged cache, which holds their keys and values already
    (dspark_paged_attention): block_table [B, max_blocks], seq_len [B], offsets [B+1] int32 (None: one token a
    request).  scale defaults to D ** -0.5.  lse: None, True, or a [T, Hq] fp32 tensor to write.  error as for
    cache_plan.
    Returns (out [T, Hq, D], lse or None, workspace)."""
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if lse is True:
        lse = torch.empty(q.shape[:2], device=q.device)
    if ws is None and stream is not None:  # (else it is made in the native call, on the current stream)
        ws = b.workspace(b.dspark_paged_attention_workspace_size(_attention_sizes(q, k_pages, seq_len, max_new)), q.device)
    st, ws = b.native().paged_attention(q, k_pages, v_pages, block_table, seq_len, offsets, k_scale, v_scale,
                                        q.shape[-1] ** -0.5 if scale is None else scale, softcap, causal, window, max_new, out,
                                        lse, ws, _raw(stream, ws, out, lse), error)
    b._check(st, "dspark_paged_attention")
    return out, lse, ws
