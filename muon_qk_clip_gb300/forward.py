"""Untimed setup: query/key features of an attention layer from its weights.

This is the model forward that produces Q and K (Q^h = X W_q^h, K^h = X W_k^h
for MHA; the MLA latent projections with RMSNorm and RoPE, [K2-internals]
"MLA 的特殊处理"), run on the library's own kernels (mc_matmul on the tcgen05
GEMM core for bf16, mc_rms_norm, mc_rope) to build inputs for qk_max_logit
and to re-measure S_max after a clip.  It is not part of the MuonClip step: in
training, S_max comes from the forward pass.  project_gqa makes the features of
packed sequences with grouped heads, normalised and rotated (mc_head_norm_rope),
for qk_attention_packed_forward.  Device tensors only.
"""
from __future__ import annotations

import torch

from . import binding as mc


def _on_device(*ts):
    """The context of the one device that the tensors are on, which need not be the
    current one."""
    for t in ts:
        if t.device.type != "cuda":
            raise ValueError("the projection runs on the library's CUDA kernels: pass device tensors")
        if t.device != ts[0].device:
            raise ValueError(f"every tensor must be on one device; these are on {ts[0].device} and {t.device}")
    return torch.cuda.device(ts[0].device)


def project_mha(X, Wq, Wk, H: int):
    """Q = X Wq^T, K = X Wk^T as [B, S, H, d] views (fp32 accumulate, X dtype out)."""
    with _on_device(X, Wq, Wk):
        return _mha(X, Wq, Wk, H)


def _mha(X, Wq, Wk, H):
    B, S, D = X.shape
    x2 = X.reshape(B * S, D)
    q = mc.matmul(x2, Wq.contiguous())
    k = mc.matmul(x2, Wk.contiguous())
    return q.reshape(B, S, H, -1), k.reshape(B, S, H, -1)


def project_mla(X, W, H: int, d_nope=128, d_rope=64, d_v=128, with_v=False):
    """MLA features: Q [B,S,H,d_nope+d_rope] = [q^C || RoPE(q^R)], K^C a
    [B,S,H,d_nope] strided view into the [B,S,H,d_nope+d_v] key/value
    projection, and the shared rotary key K^R = RoPE(X W_KR^T) [B,S,d_rope];
    with_v adds the values V, the other strided view [B,S,H,d_v] of that
    projection.  The latents c_Q = RMSNorm(X W_DQ^T) and c_KV =
    RMSNorm(X W_DKV^T) are rounded to X's dtype before their up-projections."""
    with _on_device(X, *W.values()):
        return _mla(X, W, H, d_nope, d_rope, d_v, with_v)


def _mla(X, W, H, d_nope, d_rope, d_v, with_v):
    B, S, D = X.shape
    x2 = X.reshape(B * S, D)
    cq = mc.rms_norm(mc.matmul(x2, W["W_DQ"].contiguous()))
    q = mc.matmul(cq, W["W_UQ"].contiguous()).reshape(B, S, H, d_nope + d_rope)
    mc.rope_(q[..., d_nope:])
    ckv = mc.rms_norm(mc.matmul(x2, W["W_DKV"].contiguous()))
    kv = mc.matmul(ckv, W["W_UKV"].contiguous()).reshape(B, S, H, d_nope + d_v)
    kr = mc.matmul(x2, W["W_KR"].contiguous()).reshape(B, S, d_rope)
    mc.rope_(kr)
    if with_v:
        return q, kv[..., :d_nope], kr, kv[..., d_nope:]
    return q, kv[..., :d_nope], kr


def packed_positions(offsets, T: int):
    """Place of each of T packed tokens in its sequence, int32 on offsets' device: the
    tokens from offsets[s] to offsets[s + 1] count from 0."""
    t = torch.arange(T, dtype=torch.int32, device=offsets.device)
    s = torch.searchsorted(offsets, t, right=True, out_int32=True) - 1
    return (t - offsets[s.clamp_(min=0)]).clamp_(min=0)


def _gains(W, dtype):
    """The norm weights of queries and keys, if any, in the features' type.  (AdamW's in fp32: a bf16
    weight near 1 has steps of 2^-8 and 2^-7 and stays where it is under updates of 1e-4.)"""
    return [None if w is None else w.to(dtype) for w in (W.get("q_norm"), W.get("k_norm"))]


def _padded(X, T, n, d):
    """New [T, n, d] of X's type whose rows are padded to whole 8 features, as the packed attention's are."""
    return X.new_empty((T, n, (d + 7) // 8 * 8))[..., :d]


def _heads(X, w, n):
    """X w^T as [T, n, width], in rows of 16-byte pitch (mc_matmul's)."""
    N, per = w.shape[0], 16 // X.element_size()
    out = X.new_empty((X.shape[0], (N + per - 1) // per * per))[:, :N]
    return mc.matmul(X, w.contiguous(), out=out).unflatten(1, (n, -1))


def project_gqa(X, W, H: int, H_kv: int, positions=None, rot=None, theta: float = 10000.0, eps: float = 1e-6, norm=True):
    """Features of packed tokens X [T, D] with grouped heads: Q = X W_Q^T [T,H,d] and
    K = X W_K^T [T,H_kv,d], each head normalised, times W["q_norm"] and W["k_norm"]
    [d] where given (fp32 or X's type: rounded to that for the call), its last `rot`
    features (all by default) rotated at `positions`; V = X W_V^T [T,H_kv,d_v].  Returns (q, k, v, saved), saved for
    backward.project_gqa_backward.  Heads of a width that is no multiple of eight lie in
    rows padded to one.  norm=False: heads without a norm, whose logits may grow (QK-Clip's
    layers: gqa_segments)."""
    with _on_device(X, *W.values(), *(() if positions is None else (positions,))):
        T = X.shape[0]
        q, k, v = _heads(X, W["W_Q"], H), _heads(X, W["W_K"], H_kv), _heads(X, W["W_V"], H_kv)
        d, dv = q.shape[2], v.shape[2]
        yq, yk, rstd = mc.qk_norm_rope(q, k, *_gains(W, X.dtype), positions, theta, rot, eps,
                                       out_q=_padded(X, T, H, d), out_k=_padded(X, T, H_kv, d), norm=norm)
        if dv % 8:
            v = _padded(X, T, H_kv, dv).copy_(v)
        return yq, yk, v, (q, k, rstd)
