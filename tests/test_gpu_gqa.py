"""The packed layer as a training step uses it: projections, norms of the heads with
their rotation, attention over packed sequences, and back to every weight's
gradient; then the MuonClip step of the matrices and AdamW of the norm weights.

Gradients against fp64 autograd of the same definitions: at most 12 roundings of
intermediates on any path from the inputs to a gradient, each at most 2^-8 of its
tensor's 2-norm: 12 * 2^-8 in the 2-norm of the result (logits of heads of unit
weight are of order one, so an error of a logit is one of its probability)."""
import numpy as np
import pytest
import torch

import oracle as O
from muon_qk_clip_gb300 import abi, backward, build, forward, synth
from muon_qk_clip_gb300 import binding as mc
from tests.gpu_helpers import f64

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
BOUND = 12 * 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    abi.load()


def mk(shape, std, key, dtype=BF16):
    return synth.normal(shape, std, key, 17).to(dtype).cuda()


def layer(D, H, G, d, dv, norm=True):
    W = {"W_Q": mk((H * d, D), 0.1, "wq"), "W_K": mk((G * d, D), 0.1, "wk"), "W_V": mk((G * dv, D), 0.1, "wv")}
    if norm:
        W["q_norm"], W["k_norm"] = (1 + mk((d,), 0.2, "nq", F32)).to(BF16), (1 + mk((d,), 0.2, "nk", F32)).to(BF16)
    return W


def offsets_of(lens):
    return torch.tensor([0, *np.cumsum(lens)], dtype=torch.int32, device="cuda")


def run(X, W, H, G, offsets, do, rot=None, status=None):
    """(o, smax, dW, dX) of the framework's calls."""
    pos = forward.packed_positions(offsets, X.shape[0])
    q, k, v, saved = forward.project_gqa(X, W, H, G, pos, rot)
    o, lse, smax = mc.qk_attention_packed_forward(q, k, v, offsets, lse=True, status=status)
    dq, dk, dv = mc.qk_attention_packed_backward(q, k, v, o, lse, do, offsets, status=status)
    dW, dX = backward.project_gqa_backward(X, W, dq, dk, dv, saved, pos, rot, status=status)
    return o, smax, dW, dX


def layer64(x, w, H, G, lens, rot, theta=10000.0, eps=1e-6):
    """Output [T, H, dv] and S_max [H] in 64 bits."""
    T = x.shape[0]
    def heads(weight, n, gain):
        z = (x @ weight.T).view(T, n, -1)
        z = z / torch.sqrt(z.pow(2).mean(-1, keepdim=True) + eps)
        z = z if gain is None else z * gain
        pos = torch.cat([torch.arange(n_) for n_ in lens]).double()
        ang = pos[:, None, None] * theta ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
        a, b = z[..., z.shape[-1] - rot::2], z[..., z.shape[-1] - rot + 1::2]
        turned = torch.stack([a * ang.cos() - b * ang.sin(), a * ang.sin() + b * ang.cos()], -1).flatten(-2)
        return torch.cat([z[..., :z.shape[-1] - rot], turned], -1)
    q, k = heads(w["W_Q"], H, w.get("q_norm")), heads(w["W_K"], G, w.get("k_norm"))
    v = (x @ w["W_V"].T).view(T, G, -1)
    k, v = (t.repeat_interleave(H // G, 1) for t in (k, v))
    outs, best, at = [], [], 0
    for n in lens:
        if n == 0:
            continue
        s = torch.einsum("ihd,jhd->hij", q[at:at + n], k[at:at + n]) / np.sqrt(q.shape[-1])
        s = s.masked_fill(torch.ones(n, n).triu(1).bool(), -np.inf)
        outs.append(torch.einsum("hij,jhd->ihd", s.softmax(-1), v[at:at + n]))
        best.append(s.amax((1, 2)))
        at += n
    return torch.cat(outs), torch.stack(best).amax(0)


def close(got, ref, what):
    ref = ref.detach().numpy()
    err = np.linalg.norm(f64(got) - ref) / np.linalg.norm(ref)
    assert got.shape == ref.shape and err <= BOUND, (what, err)


@pytest.mark.parametrize("lens,H,G,d,dv,rot,norm", [
    ([37, 100, 0, 1, 62], 4, 2, 64, 64, 64, True),
    ([129, 15], 6, 2, 80, 48, 40, True),
    ([70], 3, 1, 32, 32, 0, False),
    ([1, 1, 1], 8, 8, 128, 128, 128, True)])
def test_layer_gradients(lens, H, G, d, dv, rot, norm):
    D, T = 192, sum(lens)
    W = layer(D, H, G, d, dv, norm)
    X, do = mk((T, D), 1.0, "x"), mk((T, H, dv), 0.05, "do")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, smax, dW, dX = run(X, W, H, G, offsets_of(lens), do, rot, st)
    torch.cuda.synchronize()
    assert st.item() == 0 and set(dW) == set(W)
    x, w = X.double().cpu().requires_grad_(True), {n: t.double().cpu().requires_grad_(True) for n, t in W.items()}
    ref, best = layer64(x, w, H, G, lens, rot)
    (ref * do.double().cpu()).sum().backward()
    close(o, ref, "o")
    # a logit: four roundings, of q and k before and behind their norm, each at most 2^-8 of a norm
    most = 4 * 2.0 ** -8 * 1.1 * np.sqrt(d) * float((W["q_norm"].abs().max() * W["k_norm"].abs().max()) if norm else 1.0)
    assert np.max(np.abs(f64(smax) - best.detach().numpy())) <= most
    if max(lens) == 1:                      # a token that sees only itself: nothing reaches its scores
        assert all(torch.all(dW[n] == 0) for n in W if n != "W_V")
    else:
        for n in W:
            if n != "W_V":
                close(dW[n], w[n].grad, n)
    close(dW["W_V"], w["W_V"].grad, "W_V")
    close(dX, x.grad, "dX")


def test_training_step_of_a_packed_layer():
    """The gradients through muonclip_step, clipped by the forward's S_max on the query heads alone,
    and adamw_step: the matrices as the oracle's step on the same gradients, the norm weights as
    AdamW's formula in 64 bits."""
    lens, H, G, d, dv, D = [90, 61, 130], 4, 2, 64, 64, 256
    W = layer(D, H, G, d, dv)
    X, do = mk((sum(lens), D), 1.0, "x"), mk((sum(lens), H, dv), 0.05, "do")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    _, smax, dW, _ = run(X, W, H, G, offsets_of(lens), do, status=st)
    names, gains = ["W_Q", "W_K", "W_V"], ["q_norm", "k_norm"]
    Wf = {n: t.float() for n, t in W.items()}
    before = {n: f64(t) for n, t in Wf.items()}
    M, s = [torch.zeros_like(Wf[n]) for n in names], mc.adamw_state([Wf[n] for n in gains])
    hp, ahp = mc.Hparams(tau=float(smax.max()) * 0.9), mc.AdamHparams()
    mc.muonclip_step([Wf[n] for n in names], [dW[n] for n in names], M, hp, status=st,
                     layers=[mc.ClipLayer(smax, mc.gqa_segments(Wf["W_Q"], H))])
    mc.adamw_step([Wf[n] for n in gains], [dW[n] for n in gains], hp=ahp, step=1, status=st, **s)
    torch.cuda.synchronize()
    assert st.item() == 0
    f32 = lambda a: float(np.float32(a))  # noqa: E731
    ohp = O.Hparams(mu=f32(hp.mu), lr=f32(hp.lr), weight_decay=f32(hp.weight_decay), rms_scale=f32(hp.rms_scale),
                    ns_coeffs=tuple(f32(c) for c in hp.ns_coeffs), ns_eps=f32(hp.ns_eps), tau=f32(hp.tau))
    ref, _, _ = O.muonclip_step({n: before[n] for n in names}, {n: f64(dW[n]) for n in names}, {n: 0 * before[n] for n in names}, ohp)
    gamma = np.minimum(1.0, f32(hp.tau) / f64(smax))
    assert gamma.min() < 1
    ref["W_Q"] = (ref["W_Q"].reshape(H, d, D) * gamma[:, None, None]).reshape(H * d, D)
    for n in names:                          # 1e-5 of the update (fp32 Newton-Schulz) and the fp32 weight's rounding
        assert np.max(np.abs(f64(Wf[n]) - ref[n])) <= 1e-5 * np.max(np.abs(ref[n] - before[n])) + 4e-7 * np.max(np.abs(ref[n])), n
    for n in gains:                          # the first step's m and v are g and g^2 of the bias-corrected update
        g, p = f64(dW[n]), before[n]
        want = p - ahp.lr * (g / (np.abs(g) + ahp.eps) + ahp.weight_decay * p)
        # m and v of three roundings and a half of three, two factors, the root, fma and quotient: within 16 of 2^-24
        assert np.all(np.abs(f64(Wf[n]) - want) <= 2.0 ** -24 * (16 * ahp.lr * (1 + np.abs(p)) + np.abs(p))), n


def test_layer_captured_with_new_sequences_and_steps():
    """Forward, gradients and both optimizer steps in one graph, replayed on other offsets and a
    counted step: the bits of eager calls."""
    H, G, d, D, T = 4, 2, 64, 256, 200
    W = layer(D, H, G, d, d)
    X, do = mk((T, D), 1.0, "x"), mk((T, H, d), 0.05, "do")
    names, gains = ["W_Q", "W_K", "W_V"], ["q_norm", "k_norm"]
    packs = [offsets_of(x) for x in ([100, 60, 40], [1, 0, 199], [30, 140, 30])]

    def state():
        w = {n: t.clone() for n, t in W.items()}
        return w, [torch.zeros_like(w[n], dtype=F32) for n in names], mc.adamw_state([w[n] for n in gains])

    def step(w, M, s, offsets, t):
        _, smax, dW, _ = run(X, w, H, G, offsets, do)
        mc.muonclip_step([w[n] for n in names], [dW[n] for n in names], M, mc.Hparams(tau=2.0),
                         layers=[mc.ClipLayer(smax, mc.gqa_segments(w["W_Q"], H))])
        mc.adamw_step([w[n] for n in gains], [dW[n] for n in gains], step=t, **s)
        t += 1

    eager, t = state(), torch.ones(1, dtype=torch.int64, device="cuda")
    for offsets in packs:
        step(*eager, offsets, t)
    torch.cuda.synchronize()
    held, offsets, t = state(), packs[0].clone(), torch.ones(1, dtype=torch.int64, device="cuda")
    spare = state()
    step(*spare, offsets, t.clone())           # first use outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*held, offsets, t)
    for other in packs:
        offsets.copy_(other)
        graph.replay()
    torch.cuda.synchronize()
    assert t.item() == 4
    for n in W:
        assert torch.equal(held[0][n], eager[0][n]), n
    for a, b in zip((*held[1], *held[2]["M"], *held[2]["V"]), (*eager[1], *eager[2]["M"], *eager[2]["V"])):
        assert torch.equal(a, b)


def test_projections_refuse():
    X, W = torch.zeros(4, 8), {"W_Q": torch.zeros(8, 8), "W_K": torch.zeros(8, 8), "W_V": torch.zeros(8, 8)}
    with pytest.raises(ValueError, match="device tensors"):
        forward.project_gqa(X, W, 1, 1)
    with pytest.raises(ValueError, match="device tensors"):
        backward.project_gqa_backward(X, W, X[:, None], X[:, None], X[:, None], (X, X, X))


def test_offsets_past_32_bits():
    """More than 2^31 values per tensor: the last sequence's results have the bits of that sequence
    alone (forward, backward, head norms), the last values' AdamW step those of a small tensor."""
    H, G, d, n, count = 32, 1, 128, 37, 15000
    T = n * count                            # 555,000 tokens, 2.27e9 values of q
    assert T * H * d > 1 << 31
    base = mk((n, H, d), 1.0, "big")
    q = base.repeat(count, 1, 1)
    k, v = (mk((n, G, d), 1.0, s).repeat(count, 1, 1) for s in ("bk", "bv"))
    offsets = torch.arange(0, T + 1, n, dtype=torch.int32, device="cuda")
    one = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    w = mk((d,), 1.0, "bw")
    pos = forward.packed_positions(offsets, T)
    yq, yk, rstd = mc.qk_norm_rope(q, k, w, w, pos)
    sq, sk, srstd = mc.qk_norm_rope(q[:n], k[:n], w, w, pos[:n])
    assert torch.equal(yq[-n:], sq) and torch.equal(yk[-n:], sk) and torch.equal(rstd[-n:], srstd)
    o, lse, smax = mc.qk_attention_packed_forward(yq, yk, v, offsets, lse=True)
    so, slse, ssmax = mc.qk_attention_packed_forward(sq, sk, v[:n], one, lse=True)
    assert torch.equal(o[-n:], so) and torch.equal(lse[:, -n:], slse) and torch.equal(smax, ssmax)
    dq, dk, dv = mc.qk_attention_packed_backward(yq, yk, v, o, lse, q, offsets)
    sdq, sdk, sdv = mc.qk_attention_packed_backward(sq, sk, v[:n], so, slse, q[:n], one)
    # a group's query tiles may be divided otherwise among items: fp32 sums of 32 x 37 terms in another order, then a rounding
    assert torch.equal(dq[-n:], sdq)
    for big, small in ((dk, sdk), (dv, sdv)):
        gap = (f64(big[-n:]) - f64(small)) / np.max(np.abs(f64(small)))
        assert np.max(np.abs(gap)) <= 2.0 ** -7
    del o, lse, yq, dk, dv
    gq, gk, dwq, _ = mc.qk_norm_rope_backward(dq, sdk.repeat(count, 1, 1), q, k, rstd, w, w, pos, dq=dq)
    tq, tk, swq, _ = mc.qk_norm_rope_backward(sdq, sdk, q[:n], k[:n], srstd, w, w, pos[:n])
    assert torch.equal(gq[-n:], tq) and torch.equal(gk[-n:], tk)
    # fp32 sums of T H terms over at least 152 blocks of 8 warps of a row each: chains of at most T H / 1216 terms and the blocks'
    terms = sdq.float().abs().unflatten(-1, (-1, 2)).sum(-1, keepdim=True).expand(-1, -1, -1, 2).flatten(-2) * (q[:n].float() * srstd[:, :H, None]).abs()
    assert np.all(np.abs(f64(dwq) / count - f64(swq)) <= (T * H / 1216 + 400) * 2.0 ** -24 * f64(terms.sum((0, 1))))
    del gq, dq, rstd
    for bits in (32, 8):
        P, Gr = [q.view(-1)], [q.view(-1).clone()]
        small = [P[0][-4096:].clone()], [Gr[0][-4096:].clone()]
        s, t = mc.adamw_state(P, bits), mc.adamw_state(small[0], bits)
        mc.adamw_step(P, Gr, step=1, **s)
        mc.adamw_step(*small, step=1, **t)
        assert torch.equal(P[0][-4096:], small[0][0])
        for name in ("M", "V"):
            a, b = s[name][0][-4096:], t[name][0]
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        del P, Gr, s


def test_layer_with_tokens_of_no_sequence():
    """A fixed T whose offsets leave out the first and the last tokens: they reach no gradient,
    whatever memory the features' gradients are allocated in; and a captured layer replayed on
    offsets that leave out more has the bits of eager calls."""
    lens, lead, tail, H, G, d, D = [90, 0, 61], 20, 85, 4, 2, 64, 192
    n = sum(lens)
    T, own = lead + n + tail, slice(lead, lead + n)
    W = layer(D, H, G, d, d)
    X, do = mk((T, D), 1.0, "x"), mk((T, H, d), 0.05, "do")
    offsets = offsets_of(lens) + lead
    held = [torch.full((T, h, d), float("nan"), dtype=BF16, device="cuda") for h in (H, H, H, G, G, G)]
    torch.cuda.synchronize()
    del held
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, smax, dW, dX = run(X, W, H, G, offsets, do, status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    x, w = X[own].double().cpu().requires_grad_(True), {m: t.double().cpu().requires_grad_(True) for m, t in W.items()}
    ref, _ = layer64(x, w, H, G, lens, d)
    (ref * do[own].double().cpu()).sum().backward()
    close(o[own], ref, "o")
    for name in W:
        close(dW[name], w[name].grad, name)
    close(dX[own], x.grad, "dX")
    other = torch.ones(T, dtype=torch.bool, device="cuda")
    other[own] = False
    assert torch.all(o[other] == 0) and torch.all(dX[other] == 0)
    packs = [offsets_of([T, 0]), torch.stack([offsets[0], offsets[1], offsets[3]]), offsets_of([5, 30]) + 7]
    want = [run(X, W, H, G, p, do) for p in packs]
    cell = packs[0].clone()
    run(X, W, H, G, cell, do)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(X, W, H, G, cell, do)
    for p, (o1, s1, dW1, dX1) in zip(packs, want):
        cell.copy_(p)
        graph.replay()
        torch.cuda.synchronize()
        o2, s2, dW2, dX2 = got
        assert torch.equal(o1, o2) and torch.equal(s1, s2) and torch.equal(dX1, dX2)
        assert all(torch.equal(dW1[m], dW2[m]) for m in W)


def test_norm_weights_move_over_steps():
    """README's loop: fp32 norm weights near 1, the default learning rate.  Over 12 steps they go where
    AdamW's formula in 64 bits takes them from the same gradients, and the layer sees them (bf16
    weights near 1 would stay exactly where they are: half a step of theirs is 2^-9)."""
    lens, H, G, d, D = [70, 33], 4, 2, 64, 128
    W = layer(D, H, G, d, d)
    gains = ["q_norm", "k_norm"]
    for n in gains:
        W[n] = 1 + mk((d,), 1e-3, n, F32)
    X, do, offsets = mk((sum(lens), D), 1.0, "x"), mk((sum(lens), H, d), 0.05, "do"), offsets_of(lens)
    s, hp = mc.adamw_state([W[n] for n in gains]), mc.AdamHparams()
    start = {n: W[n].clone() for n in gains}
    P, M, V = ({n: f for n, f in zip(gains, (f64(W[n]) * k for n in gains))} for k in (1, 0, 0))
    first = None
    for t in range(1, 13):
        o, _, dW, _ = run(X, W, H, G, offsets, do)
        first = o if first is None else first
        mc.adamw_step([W[n] for n in gains], [dW[n] for n in gains], hp=hp, step=t, **s)
        for n in gains:
            g = f64(dW[n])
            M[n] = hp.beta1 * M[n] + (1 - hp.beta1) * g
            V[n] = hp.beta2 * V[n] + (1 - hp.beta2) * g * g
            P[n] = P[n] - hp.lr * (M[n] / (1 - hp.beta1 ** t) / (np.sqrt(V[n] / (1 - hp.beta2 ** t)) + hp.eps) + hp.weight_decay * P[n])
    for n in gains:
        # a step: lr's share of 40 roundings of the update, and one of the weight; m may cancel, v not
        assert np.max(np.abs(f64(W[n]) - P[n])) <= 12 * (hp.lr * 200 * 2.0 ** -24 + 2.0 ** -23)
        assert torch.all(W[n] != start[n]) and float((W[n] - start[n]).abs().mean()) > 2 * hp.lr
    assert not torch.equal(first, run(X, W, H, G, offsets, do)[0])


@pytest.mark.parametrize("lens,H,G,d,dv,rot", [([60, 9], 4, 2, 36, 20, 36), ([131], 3, 1, 90, 33, 30), ([40, 17], 1, 1, 18, 17, 0)])
def test_layer_of_widths_that_are_no_multiple_of_eight(lens, H, G, d, dv, rot):
    """The layer's features come in rows that the packed attention takes, its gradients in rows that
    the projections' take."""
    D, T = 64, sum(lens)
    W, X, do = layer(D, H, G, d, dv), mk((T, D), 1.0, "x"), mk((T, H, dv), 0.05, "do")
    held = torch.zeros((T, H, (dv + 7) // 8 * 8), dtype=BF16, device="cuda")[..., :dv]
    held.copy_(do)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, _, dW, dX = run(X, W, H, G, offsets_of(lens), held, rot, st)
    torch.cuda.synchronize()
    assert st.item() == 0
    x, w = X.double().cpu().requires_grad_(True), {n: t.double().cpu().requires_grad_(True) for n, t in W.items()}
    ref, _ = layer64(x, w, H, G, lens, rot)
    (ref * do.double().cpu()).sum().backward()
    close(o, ref, "o")
    for n in W:
        close(dW[n], w[n].grad, n)
    close(dX, x.grad, "dX")


@pytest.mark.parametrize("lens,H,G,d,dv,rot", [([37, 100, 0, 1, 62], 4, 2, 64, 64, 64), ([129, 15], 3, 1, 80, 48, 40)])
def test_layer_without_head_norms_and_its_clip(lens, H, G, d, dv, rot):
    """Plain rotary heads, whose logits may grow: gradients against fp64 autograd, and QK-Clip by the
    forward's S_max on the query heads' rows brings the layer's S_max to tau."""
    D, T = 192, sum(lens)
    W = {n: t * 0.7 for n, t in layer(D, H, G, d, dv, norm=False).items()}
    X, do, offsets = mk((T, D), 1.0, "x"), mk((T, H, dv), 0.05, "do"), offsets_of(lens)
    pos = forward.packed_positions(offsets, T)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, k, v, saved = forward.project_gqa(X, W, H, G, pos, rot, norm=False)
    o, lse, smax = mc.qk_attention_packed_forward(q, k, v, offsets, lse=True, status=st)
    dq, dk, dvv = mc.qk_attention_packed_backward(q, k, v, o, lse, do, offsets, status=st)
    dW, dX = backward.project_gqa_backward(X, W, dq, dk, dvv, saved, pos, rot, status=st)
    torch.cuda.synchronize()
    assert st.item() == 0 and set(dW) == set(W)
    x, w = X.double().cpu().requires_grad_(True), {n: t.double().cpu().requires_grad_(True) for n, t in W.items()}
    # in 64 bits, x / sqrt(mean + 1e300) * 1e150 is x: a head that is not normalised
    one = {n: torch.full((d,), 1e150, dtype=torch.float64) for n in ("q_norm", "k_norm")}
    ref, best = layer64(x, {**w, **one}, H, G, lens, rot, eps=1e300)
    (ref * do.double().cpu()).sum().backward()
    for got, want, name in [(o, ref, "o"), (dX, x.grad, "dX")] + [(dW[n], w[n].grad, n) for n in W]:
        close(got, want, name)
    # a logit: roundings of q and k behind the products and behind the rotation, 4 of 2^-8 of a norm each
    reach = lambda t: float(t.float().norm(dim=-1).max())  # noqa: E731
    most = 4 * 2.0 ** -8 * reach(q) * reach(k) / np.sqrt(d)
    assert np.max(np.abs(f64(smax) - best.detach().numpy())) <= most
    tau = float(smax.max()) * 0.5
    mc.qk_clip_apply(smax, tau, mc.gqa_segments(W["W_Q"], H))
    q, k, v, _ = forward.project_gqa(X, W, H, G, pos, rot, norm=False)
    _, _, after = mc.qk_attention_packed_forward(q, k, v, offsets)
    torch.cuda.synchronize()
    assert np.all(np.abs(f64(after) - np.minimum(f64(smax), tau)) <= 2 * most)
