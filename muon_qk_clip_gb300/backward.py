"""Gradients of the query/key/value projections (forward.py), from the gradients
of the features that qk_attention_backward returns to the weight gradients that
muonclip_step takes:

    q, kc, kr, v = forward.project_mla(X, W, H, with_v=True)
    o, lse, smax = mc.qk_attention_forward(q, kc, v, kr, lse=True)
    dq, dk, dv, dkr = mc.qk_attention_backward(q, kc, v, o, lse, do, k_shared=kr)
    dW, dX = backward.project_mla_backward(X, W, H, dq, dk, dkr, dv)
    mc.muonclip_step(W_list, [dW[n] for n in names], M_list, hp, layers=[...])

Products run on mc_matmul, norms and rotations on mc_rms_norm_backward and
mc_rope_backward; torch only lays out operands (transposes, concatenations).
Weight gradients and dX have X's dtype (bf16: fp32 sums rounded once).  Device
tensors only.
"""
from __future__ import annotations

import torch

from . import binding as mc
from .forward import _on_device


def _turned(t):
    """Transpose of a 2-D tensor as rows of 16-byte pitch (mc_matmul's operands)."""
    per = 16 // t.element_size()
    out = t.new_empty((t.shape[1], (t.shape[0] + per - 1) // per * per))[:, :t.shape[0]]
    return out.copy_(t.t())


def _pitched(t):
    """t with rows of 16-byte pitch: t itself if it has them, or a copy (of
    broadcast rows too)."""
    per = 16 // t.element_size()
    if t.stride(1) == 1 and t.stride(0) % per == 0 and t.stride(0) >= t.shape[1] and t.data_ptr() % 16 == 0:
        return t
    out = t.new_empty((t.shape[0], (t.shape[1] + per - 1) // per * per))[:, :t.shape[1]]
    return out.copy_(t)


def _product(a, b, status):
    """A B^T with operands laid out for mc_matmul."""
    per = 16 // a.element_size()
    M, N = a.shape[0], b.shape[0]
    out = a.new_empty((M, (N + per - 1) // per * per))[:, :N]
    return mc.matmul(_pitched(a), _pitched(b), out=out, status=status)


def _weight(dy, x, status):
    """dW = dY^T X of Y = X W^T, sums over the tokens."""
    return _product(_turned(dy), _turned(x), status).contiguous()


def project_mha_backward(X, Wq, Wk, dq, dk, status=None):
    """Of project_mha: dq, dk [B, S, H, d] to (dWq, dWk, dX)."""
    with _on_device(X, Wq, Wk, dq, dk):
        return _mha(X, Wq, Wk, dq, dk, status)


def _mha(X, Wq, Wk, dq, dk, status):
    B, S, D = X.shape
    x2 = X.reshape(B * S, D)
    dq2, dk2 = dq.reshape(B * S, -1), dk.reshape(B * S, -1)
    # one product over the concatenated features, so dX is rounded once
    dX = _product(torch.cat([dq2, dk2], 1), _turned(torch.cat([Wq, Wk], 0)), status)
    return _weight(dq2, x2, status), _weight(dk2, x2, status), dX.reshape(B, S, D)


def project_mla_backward(X, W, H: int, dq, dk, dkr, dv=None, d_nope=128, d_rope=64, d_v=128, eps: float = 1e-6,
                         theta: float = 10000.0, status=None):
    """Of project_mla: dq [B,S,H,d_nope+d_rope], dk [B,S,H,d_nope] (of k^C), dkr
    [B,S,d_rope] (of the shared rotary key, summed over the heads as
    qk_attention_backward gives it) and dv [B,S,H,d_v] (None: zero) to
    ({name: dW}, dX) for W_DQ, W_UQ, W_DKV, W_UKV and W_KR.  The latents are
    recomputed from X; their norm's sums run in another order than project_mla's,
    so a value next to a rounding border may differ from the forward's in its last
    bit.  No gradient is overwritten."""
    with _on_device(X, dq, dk, dkr, *W.values(), *(() if dv is None else (dv,))):
        return _mla(X, W, H, dq, dk, dkr, dv, d_nope, d_rope, d_v, eps, theta, status)


def _mla(X, W, H, dq, dk, dkr, dv, d_nope, d_rope, d_v, eps, theta, status):
    B, S, D = X.shape
    T = B * S
    x2 = X.reshape(T, D)
    kv = dk.new_zeros((B, S, H, d_nope + d_v)) if dv is None else dk.new_empty((B, S, H, d_nope + d_v))
    kv[..., :d_nope] = dk
    if dv is not None:
        kv[..., d_nope:] = dv
    q = dq.clone(memory_format=torch.contiguous_format)
    mc.rope_backward(q[..., d_nope:], theta, out=q[..., d_nope:])
    dkr2 = mc.rope_backward(dkr, theta).reshape(T, d_rope)
    dW, down = {"W_KR": _weight(dkr2, x2, status)}, [dkr2]
    for d2, w_down, w_up in ((kv.reshape(T, -1), "W_DKV", "W_UKV"), (q.reshape(T, -1), "W_DQ", "W_UQ")):
        latent = _product(x2, W[w_down], status)
        c, _, _, rstd = mc.add_rms_norm(latent, eps=eps)
        dW[w_up] = _weight(d2, c, status)
        dc = _product(d2, _turned(W[w_up]), status)
        dl, _ = mc.rms_norm_backward(dc, latent, rstd)
        dW[w_down] = _weight(dl, x2, status)
        down.append(dl)
    # one product over the concatenated down-projections, so dX is rounded once
    dX = _product(torch.cat(down, 1), _turned(torch.cat([W["W_KR"], W["W_DKV"], W["W_DQ"]], 0)), status)
    return dW, dX.reshape(B, S, D)
