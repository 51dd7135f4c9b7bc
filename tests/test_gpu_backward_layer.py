"""The gradient calls composed as a training step uses them (backward.py): the
projections' weight gradients from the features' gradients, an attention
layer's from the output's, and the MuonClip step on them.

fp32 projections against fp64 autograd of the same definitions: each value
passes through at most four fp32 products and two row sums, n <= 512 terms
each: relative to the largest entry, 8 * 512 * 2^-24 = 2.5e-4 bounds the sums'
rounding with every term of one sign; the compensated sums of the products stay
far inside.  bf16: at most 12 roundings of intermediates on any path from the
inputs to a weight gradient, each at most 2^-8 of its tensor's 2-norm, so
12 * 2^-8 in the 2-norm of the result (random signs: a few 2^-8).
"""
import numpy as np
import pytest
import torch

import oracle as O
from muon_qk_clip_gb300 import abi, backward, build, forward, synth
from muon_qk_clip_gb300 import binding as mc
from tests.gpu_helpers import f64

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
BOUND = {F32: 2.5e-4, BF16: 12 * 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    abi.load()


def mk(shape, std, key, dtype):
    return synth.normal(shape, std, key, 11).to(dtype).cuda()


def double(t):
    return t.detach().double().cpu().requires_grad_(True)


def rope64(x, theta=10000.0):
    S, d = x.shape[1], x.shape[-1]
    ang = torch.arange(S, dtype=torch.float64)[:, None] * theta ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
    shape = [1, S] + [1] * (x.dim() - 3) + [d // 2]
    c, s = ang.cos().view(shape), ang.sin().view(shape)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)


def mla64(X, W, H, dn, dr, dv):
    norm = lambda t: t / torch.sqrt(t.pow(2).mean(-1, keepdim=True) + 1e-6)  # noqa: E731
    B, S, _ = X.shape
    q = (norm(X @ W["W_DQ"].T) @ W["W_UQ"].T).view(B, S, H, dn + dr)
    q = torch.cat([q[..., :dn], rope64(q[..., dn:])], -1)
    kv = (norm(X @ W["W_DKV"].T) @ W["W_UKV"].T).view(B, S, H, dn + dv)
    return q, kv[..., :dn], rope64(X @ W["W_KR"].T), kv[..., dn:]


def close(got, ref, bound, what):
    ref = ref.numpy()
    err = np.linalg.norm(f64(got) - ref) / np.linalg.norm(ref)
    assert got.shape == ref.shape and err <= bound, (what, err)


def mla_weights(D, H, ql, kl, dn, dr, dv, dtype):
    return {"W_DQ": mk((ql, D), 0.1, "dq", dtype), "W_UQ": mk((H * (dn + dr), ql), 0.2, "uq", dtype),
            "W_DKV": mk((kl, D), 0.1, "dkv", dtype), "W_UKV": mk((H * (dn + dv), kl), 0.2, "ukv", dtype),
            "W_KR": mk((dr, D), 0.1, "kr", dtype)}


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,S", [(1, 1), (2, 37), (1, 300)])
def test_project_mha_backward(B, S, dtype):
    D, H, d = 256, 4, 64
    X, Wq, Wk = mk((B, S, D), 1.0, "x", dtype), mk((H * d, D), 0.1, "wq", dtype), mk((H * d, D), 0.1, "wk", dtype)
    dq, dk = mk((B, S, H, d), 0.1, "gq", dtype), mk((B, S, H, d), 0.1, "gk", dtype)
    got = backward.project_mha_backward(X, Wq, Wk, dq, dk)
    x, wq, wk = double(X), double(Wq), double(Wk)
    ((x @ wq.T).view(B, S, H, d) * dq.double().cpu()).sum().add(
        ((x @ wk.T).view(B, S, H, d) * dk.double().cpu()).sum()).backward()
    for g, r, n in zip(got, (wq.grad, wk.grad, x.grad), ("dWq", "dWk", "dX")):
        close(g, r, BOUND[dtype], n)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_project_backward_of_broadcast_tensors(dtype):
    """Rows that share memory (one token's X, or one gradient for all tokens) are
    read as the rows that they stand for."""
    B, D, H, d = 5, 64, 2, 32
    Wq, Wk = mk((H * d, D), 0.1, "wq", dtype), mk((H * d, D), 0.1, "wk", dtype)
    X, dq, dk = (mk((1, 1, *s), 1.0, n, dtype).expand(B, 1, *s) for n, s in (("x", (D,)), ("gq", (H, d)), ("gk", (H, d))))
    got = backward.project_mha_backward(X, Wq, Wk, dq, dk)
    want = backward.project_mha_backward(X.contiguous(), Wq, Wk, dq.contiguous(), dk.contiguous())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("with_v", [True, False])
def test_project_mla_backward(dtype, with_v):
    B, S, D, H, ql, kl, dn, dr, dv = 2, 75, 192, 3, 96, 64, 16, 8, 24
    W = mla_weights(D, H, ql, kl, dn, dr, dv, dtype)
    X = mk((B, S, D), 1.0, "mx", dtype)
    grads = [mk((B, S, H, dn + dr), 0.1, "g0", dtype), mk((B, S, H, dn), 0.1, "g1", dtype), mk((B, S, dr), 0.1, "g2", dtype),
             mk((B, S, H, dv), 0.1, "g3", dtype) if with_v else None]
    keep = [None if g is None else g.clone() for g in grads]
    dW, dX = backward.project_mla_backward(X, W, H, *grads, d_nope=dn, d_rope=dr, d_v=dv)
    assert all(g is None or torch.equal(g, k) for g, k in zip(grads, keep))
    x, w = double(X), {n: double(t) for n, t in W.items()}
    outs = mla64(x, w, H, dn, dr, dv)
    sum((o * g.double().cpu()).sum() for o, g in zip(outs, grads) if g is not None).backward()
    close(dX, x.grad, BOUND[dtype], "dX")
    for n in W:
        close(dW[n], w[n].grad, BOUND[dtype], n)


def attention64(q, kc, kr, v):
    k = torch.cat([kc, kr[:, :, None, :].expand(*kc.shape[:3], -1)], -1)
    S = q.shape[1]
    s = torch.einsum("bihd,bjhd->bhij", q, k) / np.sqrt(q.shape[-1])
    s = s.masked_fill(torch.ones(S, S).triu(1).bool(), -np.inf)
    return torch.einsum("bhij,bjhd->bihd", s.softmax(-1), v)


def test_mla_layer_gradients_and_muonclip_step():
    """X through the MLA projections, attention and back to every projection's
    gradient, then one MuonClip step on those gradients with the forward's S_max:
    the step equals the oracle's on the same (stored) gradients."""
    B, S, D, H, ql, kl, dn, dr, dv = 1, 200, 256, 3, 96, 64, 64, 16, 32
    W = mla_weights(D, H, ql, kl, dn, dr, dv, BF16)
    X, do = mk((B, S, D), 1.0, "lx", BF16), mk((B, S, H, dv), 0.05, "ldo", BF16)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, kc, kr, v = forward.project_mla(X, W, H, dn, dr, dv, with_v=True)
    o, lse, smax = mc.qk_attention_forward(q, kc, v, kr, lse=True, status=st)
    dq, dk, dvv, dkr = mc.qk_attention_backward(q, kc, v, o, lse, do, k_shared=kr, status=st)
    dW, dX = backward.project_mla_backward(X, W, H, dq, dk, dkr, dvv, d_nope=dn, d_rope=dr, d_v=dv, status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    x, w = double(X), {n: double(t) for n, t in W.items()}
    (attention64(*[mla64(x, w, H, dn, dr, dv)[i] for i in (0, 1, 2, 3)]) * do.double().cpu()).sum().backward()
    close(dX, x.grad, BOUND[BF16], "dX")
    for n in W:
        close(dW[n], w[n].grad, BOUND[BF16], n)
    # the step: fp32 masters, the gradients as stored
    names = list(W)
    Wf, M = [W[n].float() for n in names], [torch.zeros_like(W[n], dtype=F32) for n in names]
    before = {n: f64(t) for n, t in zip(names, Wf)}
    hp = mc.Hparams(tau=float(smax.max()) / 2)
    by = dict(zip(names, Wf))
    mc.muonclip_step(Wf, [dW[n] for n in names], M, hp, status=st,
                     layers=[mc.ClipLayer(smax, mc.mla_segments(by["W_UQ"], by["W_UKV"], H, dn, dr, dv))])
    torch.cuda.synchronize()
    assert st.item() == 0
    f32 = lambda a: float(np.float32(a))  # noqa: E731
    ohp = O.Hparams(mu=f32(hp.mu), lr=f32(hp.lr), weight_decay=f32(hp.weight_decay), rms_scale=f32(hp.rms_scale),
                    ns_coeffs=tuple(f32(c) for c in hp.ns_coeffs), ns_eps=f32(hp.ns_eps), tau=f32(hp.tau))
    ref, _, _ = O.muonclip_step(before, {n: f64(dW[n]) for n in names}, {n: 0 * before[n] for n in names}, ohp,
                                layers=[(f64(smax), O.mla_segments(H, dn, dr, dv))])
    for n, t in zip(names, Wf):
        # 1e-5 of the update (fp32 Newton-Schulz) and the fp32 weight's rounding
        assert np.max(np.abs(f64(t) - ref[n])) <= 1e-5 * np.max(np.abs(ref[n] - before[n])) + 4e-7 * np.max(np.abs(ref[n])), n


def test_prenorm_residual_block_gradients():
    """A pre-norm block's ends: h = x + r, y = norm(h) w feeds the MHA projections;
    their dX comes back through the norm and joins the residual's gradient."""
    B, S, D, H, d = 1, 120, 256, 4, 64
    x, r = mk((B * S, D), 1.0, "px", F32), mk((B * S, D), 2.0, "pr", F32)
    w = 1 + mk((D,), 0.2, "pw", F32)
    Wq, Wk = mk((H * d, D), 0.1, "pq", F32), mk((H * d, D), 0.1, "pk", F32)
    dq, dk = mk((B, S, H, d), 0.1, "pgq", F32), mk((B, S, H, d), 0.1, "pgk", F32)
    dh = mk((B * S, D), 0.1, "pdh", F32)                       # what arrives along the residual stream
    y, _, h, rstd = mc.add_rms_norm(x, r, w)
    dWq, dWk, dy = backward.project_mha_backward(y.view(B, S, D), Wq, Wk, dq, dk)
    dx, dw = mc.rms_norm_backward(dy.reshape(B * S, D), h, rstd, weight=w, dres=dh)
    X, Rr, ww, a, b = double(x), double(r), double(w), double(Wq), double(Wk)
    hh = X + Rr
    yy = hh / torch.sqrt(hh.pow(2).mean(-1, keepdim=True) + 1e-6) * ww
    loss = ((yy @ a.T).view(B, S, H, d) * dq.double().cpu()).sum() + ((yy @ b.T).view(B, S, H, d) * dk.double().cpu()).sum()
    (loss + (hh * dh.double().cpu()).sum()).backward()
    for g, ref, n in ((dx, X.grad, "dx"), (dx, Rr.grad, "dresidual"), (dw, ww.grad, "dw"), (dWq, a.grad, "dWq"), (dWk, b.grad, "dWk")):
        close(g, ref, BOUND[F32], n)


def test_projection_backward_rejects_host_tensors():
    X, W = torch.zeros(1, 4, 8), torch.zeros(8, 8)
    with pytest.raises(ValueError, match="device tensors"):
        backward.project_mha_backward(X, W, W, X.view(1, 4, 1, 8), X.view(1, 4, 1, 8))


def test_chained_layer_calls_match_calls_one_by_one():
    """Forward, attention's gradient (long and short sequences), rotary gradient:
    queued behind each other, eagerly and captured, with the bits of calls that each
    wait for the one before."""
    for B, S in ((2, 300), (40, 12)):
        q, k, v, do = (mk((B, S, 4, d), 1.0, n, BF16) for n, d in (("cq", 192), ("ck", 128), ("cv", 128), ("cd", 128)))
        ks, big = mk((B, S, 64), 1.0, "cks", BF16), torch.empty(64 << 20, device="cuda")

        def chain(wait):
            done = torch.cuda.synchronize if wait else (lambda: None)
            big.fill_(1.0)
            done()
            o, lse, _ = mc.qk_attention_forward(q, k, v, ks, lse=True)
            done()
            dq, dk, dv, dks = mc.qk_attention_backward(q, k, v, o, lse, do, k_shared=ks)
            done()
            mc.rope_backward(dq[..., 128:], out=dq[..., 128:])
            done()
            dks = mc.rope_backward(dks)
            done()
            return dq, dk, dv, dks

        want = chain(True)
        runs = [chain(False) for _ in range(4)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for got in runs for a, b in zip(want, got))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = [chain(False), chain(False)]
        for _ in range(2):
            for t in (*got[0], *got[1]):
                t.fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for g in got for a, b in zip(want, g))
