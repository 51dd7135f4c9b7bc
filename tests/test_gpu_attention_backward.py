"""GPU parity of qk_attention_backward with the oracle's gradients.

Bounds, from the kernel's arithmetic (u = 2^-8: half a step of bf16, relative;
w = 2^-24: of fp32), with magnitudes summed over absolute values:
  * the exponent of p: the fp32 sum of D products, its scaling and the rounded
    lse give an absolute error of at most
        a_ij = w (D + 4) scale |q_i|.|k_j| + 4 w |lse_i|;
    the hardware's base-2 exponential adds 2^-22 relative: p has relative error
    e = a + 2^-22, and u more as an operand
  * dv: sum (u + e) p |do| + S w sum p |do|, then u |dv| for the rounding
  * ds = p (dp - delta): e |ds| + p w (d_v + 4) (|do|.|v| + |do|.|o|), and u |ds|
    as an operand
  * dq, dk: the sums of ds's error with |k|, |q|, S w of the sum's magnitude,
    u of the result; dk_shared sums those of the heads
"""
import numpy as np
import pytest
import torch

import oracle as O
from muon_qk_clip_gb300 import abi, build
from muon_qk_clip_gb300 import binding as mc
from muon_qk_clip_gb300 import synth
from tests.gpu_helpers import f64

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
U, W = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    abi.load()


def inputs(B, S, H, dh, dr, dv, seed, causal=True, head_scale=None):
    """bf16 q, k, ks, v, do and the oracle's o (bf16) and lse (fp32) for them."""
    q = synth.normal((B, S, H, dh + dr), 1.0, "bq", seed)
    if head_scale is not None:
        q = q * torch.tensor(head_scale)[None, None, :, None]
    q = q.to(BF16)
    k = synth.normal((B, S, H, dh), 1.0, "bk", seed).to(BF16)
    ks = synth.normal((B, S, dr), 1.0, "bks", seed).to(BF16) if dr else None
    v = synth.normal((B, S, H, dv), 1.0, "bv", seed).to(BF16)
    do = synth.normal((B, S, H, dv), 0.01, "bdo", seed).to(BF16)
    o, lse, _ = O.attention_forward(f64(q), f64(k), f64(v), None if ks is None else f64(ks), causal=causal)
    return q, k, ks, v, do, torch.from_numpy(o).to(BF16), torch.from_numpy(lse).float()


def bounds(q, k, ks, v, do, o, lse, causal, scale=None, operand=U):
    """(gradients, error bounds) in float64, as the module's docstring derives them;
    operand: the rounding of p and ds as operands."""
    Q, K, V, dO, Og, L = (f64(t) for t in (q, k, v, do, o, lse))
    Ks = None if ks is None else f64(ks)
    B, S, H, D = Q.shape
    dh, dv = K.shape[3], V.shape[3]
    scale = 1.0 / np.sqrt(D) if scale is None else scale
    ref = O.attention_backward(Q, K, V, Og, L, dO, Ks, causal=causal, scale=scale)
    eq, ek, ev = (np.zeros_like(r) for r in ref[:3])
    es = None if Ks is None else np.zeros_like(ref[3])
    for b in range(B):
        for h in range(H):
            qq, vv, dd, oo = Q[b, :, h], V[b, :, h], dO[b, :, h], Og[b, :, h]
            kk = O.head_keys(K, Ks, b, h)
            p = np.exp(np.minimum(scale * qq @ kk.T - L[b, h][:, None], 700.0))
            if causal:
                p = np.tril(p)
            a = W * (D + 4) * scale * (np.abs(qq) @ np.abs(kk).T) + 4 * W * np.abs(L[b, h])[:, None]
            e = a + 2.0 ** -22
            ds = np.abs(p * (dd @ vv.T - np.sum(dd * oo, 1)[:, None]))
            mags = np.abs(dd) @ np.abs(vv).T + np.sum(np.abs(dd) * np.abs(oo), 1)[:, None]
            err = (e + operand) * ds + p * (1 + e + operand) * W * (dv + 4) * mags
            pd = p.T @ np.abs(dd)
            ev[b, :, h] = ((operand + e) * p).T @ np.abs(dd) + S * W * pd
            eq[b, :, h] = scale * ((err + S * W * ds) @ np.abs(kk))
            full = scale * ((err + S * W * ds).T @ np.abs(qq))
            ek[b, :, h] = full[:, :dh]
            if es is not None:
                es[b] += full[:, dh:]
    errs = [eq, ek, ev, es]
    return ref, [None if r is None else x * 1.01 + U * np.abs(r) + 1e-30 for r, x in zip(ref, errs)]


def check(got, ref, tol):
    for name, g, r, t in zip(("dq", "dk", "dv", "dk_shared"), got, ref, tol):
        if r is None:
            assert g is None
            continue
        err = np.abs(f64(g) - r)
        assert np.all(err <= t), (f"{name}: {int(np.sum(~(err <= t)))} of {err.size} outside, "
                                  f"worst excess {np.nanmax(err - t):.3g}, max err {np.nanmax(err):.3g}")


def dev(*ts):
    return [None if t is None else t.cuda() for t in ts]


CASES = [
    (1, 1, 1, 64, 0, 64, True),           # one token
    (2, 3, 2, 16, 0, 16, True),           # the narrowest widths
    (1, 128, 2, 128, 0, 128, True),       # exactly one block
    (1, 129, 2, 128, 0, 128, True),       # one row into the second
    (2, 300, 3, 128, 0, 128, True),       # ragged last block
    (1, 384, 2, 64, 0, 128, False),       # unmasked, whole blocks, values wider than keys
    (3, 333, 2, 80, 0, 48, False),        # widths off the 64-wide chunks
    (1, 200, 2, 24, 0, 72, True),
    (1, 290, 2, 192, 0, 64, True),        # q.k length 192 without a shared part: 96-query tiles
    (1, 257, 2, 128, 64, 128, True),      # MLA
    (2, 96, 3, 128, 64, 128, True),       # MLA, exactly one query tile
    (1, 193, 3, 128, 64, 128, False),     # MLA, no mask
    (1, 150, 5, 64, 40, 96, True),        # MLA, one chunk each, odd rotary width
    (1, 700, 1, 128, 8, 16, True),        # several tiles of both sizes
]


@pytest.mark.parametrize("B,S,H,dh,dr,dv,causal", CASES)
def test_attention_backward_parity(B, S, H, dh, dr, dv, causal):
    q, k, ks, v, do, o, lse = inputs(B, S, H, dh, dr, dv, 70 + S, causal)
    ref, tol = bounds(q, k, ks, v, do, o, lse, causal)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    dq_, dk_, dks_, dv_, ddo, do_, dl = dev(q, k, ks, v, do, o, lse)
    got = mc.qk_attention_backward(dq_, dk_, dv_, do_, dl, ddo, k_shared=dks_, causal=causal, status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    check(got, ref, tol)
    again = mc.qk_attention_backward(dq_, dk_, dv_, do_, dl, ddo, k_shared=dks_, causal=causal)
    assert all(a is b is None or torch.equal(a, b) for a, b in zip(got, again))     # equal bits


def test_attention_backward_heavy_logits():
    """Heads with logits far over tau: nearly one-hot rows, where ds is a small
    difference of large terms, and an explicit scale."""
    q, k, ks, v, do, o, lse = inputs(1, 400, 3, 128, 0, 128, 91, True, head_scale=[1.0, 12.0, 25.0])
    ref, tol = bounds(q, k, ks, v, do, o, lse, True)
    a = dev(q, k, v, o, lse, do)
    check(mc.qk_attention_backward(*a), ref, tol)
    q, k, ks, v, do, _, _ = inputs(1, 140, 2, 64, 0, 64, 92)
    out, lse, _ = O.attention_forward(f64(q), f64(k), f64(v), scale=0.31)
    o, lse = torch.from_numpy(out).to(BF16), torch.from_numpy(lse).float()
    ref, tol = bounds(q, k, ks, v, do, o, lse, True, scale=0.31)
    check(mc.qk_attention_backward(*dev(q, k, v, o, lse, do), scale=0.31), ref, tol)


def test_attention_backward_strided_outputs_and_inputs():
    """k and v interleaved in one buffer, as the MLA projection gives them, their
    gradients in another; q and its gradient head-major; nothing outside the
    outputs is touched."""
    B, S, H, dh, dr, dv = 2, 200, 3, 64, 16, 48
    q, k, ks, v, do, o, lse = inputs(B, S, H, dh, dr, dv, 93)
    ref, tol = bounds(q, k, ks, v, do, o, lse, True)
    kv = torch.cat([k, v], -1).cuda()
    dkv = torch.full((B, S + 2, H, dh + dv + 8), 7.0, dtype=BF16, device="cuda")
    qh = q.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3)
    dq = torch.full((B, H, S + 1, dh + dr), 7.0, dtype=BF16, device="cuda").permute(0, 2, 1, 3)
    got = mc.qk_attention_backward(qh, kv[..., :dh], kv[..., dh:], o.cuda(), lse.cuda(), do.cuda(), k_shared=ks.cuda(),
                                   dq=dq[:, :S], dk=dkv[:, :S, :, :dh], dv=dkv[:, :S, :, dh:dh + dv])
    torch.cuda.synchronize()
    check(got, ref, tol)
    assert torch.all(dkv[:, S:] == 7.0) and torch.all(dkv[..., dh + dv:] == 7.0) and torch.all(dq[:, S:] == 7.0)


@pytest.mark.parametrize("B,S,H,dh,dr,dv,off", [(2, 131, 3, 20, 0, 50, 0), (1, 150, 2, 64, 12, 33, 0), (1, 140, 3, 128, 61, 127, 8),
                                                (2, 33, 2, 191, 0, 17, 8), (1, 1, 1, 64, 1, 16, 8),
                                                (1, 8, 7, 64, 61, 33, 8), (2, 30, 2, 45, 0, 19, 0)])
def test_attention_backward_odd_widths(B, S, H, dh, dr, dv, off):
    """Widths that are no multiple of eight, in rows padded to one, on 16-byte
    addresses that are and are not 32-byte ones: what lies between the rows is
    neither read (it is NaN in the inputs) nor written."""
    q, k, ks, v, do, o, lse = inputs(B, S, H, dh, dr, dv, 101)
    ref, tol = bounds(q, k, ks, v, do, o, lse, True)

    def padded(shape, fill):
        w = (shape[-1] + 7) // 8 * 8 + off
        return torch.full((*shape[:-1], w + off), fill, dtype=BF16, device="cuda")

    def within(t):
        if t is None:
            return None
        big = padded(t.shape, float("nan"))
        big[..., off:off + t.shape[-1]] = t.cuda()
        return big[..., off:off + t.shape[-1]]

    bigs = [None if t is None else padded(t.shape, 7.0) for t in (q, k, v, ks)]
    outs = [None if b is None else b[..., off:off + t.shape[-1]] for b, t in zip(bigs, (q, k, v, ks))]
    a = [within(t) for t in (q, k, v, o)]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = mc.qk_attention_backward(*a, lse.cuda(), within(do), k_shared=within(ks), dq=outs[0], dk=outs[1], dv=outs[2],
                                   dk_shared=outs[3], status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    check(got, ref, tol)
    for big, t in zip(bigs, (q, k, v, ks)):
        if big is not None:
            assert torch.all(big[..., :off] == 7.0) and torch.all(big[..., off + t.shape[-1]:] == 7.0)


def test_attention_backward_of_broadcast_keys():
    """One key/value head for every query head (stride 0): the gradients come per
    query head, for the caller to sum."""
    B, S, H, d = 1, 150, 4, 64
    q, k, _, v, do, _, _ = inputs(B, S, H, d, 0, d, 94)
    k, v = k[:, :, :1].expand(B, S, H, d), v[:, :, :1].expand(B, S, H, d)
    out, lse, _ = O.attention_forward(f64(q), f64(k), f64(v))
    o, lse = torch.from_numpy(out).to(BF16), torch.from_numpy(lse).float()
    ref, tol = bounds(q, k, None, v, do, o, lse, True)
    kd, vd = k[:, :, :1].cuda().expand(B, S, H, d), v[:, :, :1].cuda().expand(B, S, H, d)
    check(mc.qk_attention_backward(q.cuda(), kd, vd, o.cuda(), lse.cuda(), do.cuda()), ref, tol)


def test_attention_backward_differences():
    """Against central differences of the oracle's forward along random
    directions: the sum over a whole gradient averages the operand roundings, so
    4 u relative to the sum of magnitudes / sqrt(n) holds with room."""
    q, k, ks, v, do, o, lse = inputs(1, 70, 2, 64, 16, 32, 95)
    got = mc.qk_attention_backward(*dev(q, k, v, o, lse, do), k_shared=ks.cuda())
    x = [f64(t) for t in (q, k, v, ks)]
    rng = np.random.default_rng(0)
    for n in range(4):
        step = rng.standard_normal(x[n].shape)
        val = []
        for eps in (1e-4, -1e-4):
            y = list(x)
            y[n] = x[n] + eps * step
            val.append(float(np.sum(O.attention_forward(y[0], y[1], y[2], y[3])[0] * f64(do))))
        diff = (val[0] - val[1]) / 2e-4
        g = f64(got[n])
        assert abs(np.sum(g * step) - diff) <= 4 * U * np.sqrt(np.sum((g * step) ** 2)) + U * abs(diff)


def test_attention_backward_after_the_forward():
    """The forward's own o and lse feed the backward; a second stream, a given
    workspace, and rows of the batch done alone give the same bits."""
    q, k, ks, v, do, _, _ = inputs(3, 260, 2, 128, 64, 128, 96)
    qd, kd, ksd, vd, dod = dev(q, k, ks, v, do)
    out, lse, _ = mc.qk_attention_forward(qd, kd, vd, ksd, lse=True)
    got = mc.qk_attention_backward(qd, kd, vd, out, lse, dod, k_shared=ksd)
    ref, tol = bounds(q, k, ks, v, do, out.cpu(), lse.cpu(), True)
    check(got, ref, tol)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = torch.empty(mc.attention_backward_workspace_size(qd, kd, ksd), dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)                        # NaN: every value that is read was written in the call
    side.wait_stream(torch.cuda.current_stream())
    one = mc.qk_attention_backward(qd, kd, vd, out, lse, dod, k_shared=ksd, workspace=ws, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, one))
    for b in range(3):
        s = slice(b, b + 1)
        alone = mc.qk_attention_backward(qd[s], kd[s], vd[s], out[s], lse[s], dod[s], k_shared=ksd[s])
        assert all(torch.equal(x[s], y) for x, y in zip(got, alone))


def test_attention_backward_in_cuda_graph():
    q, k, ks, v, do, o, lse = inputs(2, 140, 2, 128, 0, 128, 97)
    a = dev(q, k, v, o, lse, do)
    eager = mc.qk_attention_backward(*a)
    torch.cuda.synchronize()
    outs = [torch.full_like(g, 3.0) for g in eager[:3]]
    ws = torch.empty(mc.attention_backward_workspace_size(a[0], a[1]), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mc.qk_attention_backward(*a, dq=outs[0], dk=outs[1], dv=outs[2], workspace=ws)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(eager[:3], outs))
    a[5].mul_(2.0)                        # new inputs in the same buffers
    graph.replay()
    fresh = mc.qk_attention_backward(*a)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(fresh[:3], outs))


def test_attention_backward_flags_nonfinite():
    q, k, ks, v, do, o, lse = inputs(1, 64, 2, 64, 0, 64, 98)
    do[0, 5, 1, 3] = float("nan")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = mc.qk_attention_backward(*dev(q, k, v, o, lse, do), status=st)
    torch.cuda.synchronize()
    assert st.item() & abi.MC_STATUS_NONFINITE_UPDATE
    assert all(torch.isfinite(g[:, :, 0]).all() for g in got[:3])       # the other head


def test_attention_backward_dense_block_full_size():
    """The dense_block layer's launch (B 4, S 4096, H 16, d 128): two heads of one
    batch row against the oracle, every row of them."""
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    mk = lambda std=1.0: (torch.randn(4, 4096, 16, 128, generator=g, device="cuda") * std).to(BF16)  # noqa: E731
    q, k, v, do = mk(), mk(), mk(), mk(0.01)
    q[:, :, 2] *= 8
    out, lse, _ = mc.qk_attention_forward(q, k, v, lse=True)
    got = mc.qk_attention_backward(q, k, v, out, lse, do)
    torch.cuda.synchronize()
    for b, h in ((0, 2), (3, 15)):
        s = (slice(b, b + 1), slice(None), slice(h, h + 1))
        sub = [t[s].cpu() for t in (q, k, v, do, out)]
        ref, tol = bounds(sub[0], sub[1], None, sub[2], sub[3], sub[4], lse[b:b + 1, h:h + 1].cpu(), True)
        check([x[s] for x in got[:3]] + [None], ref, tol)


@pytest.mark.parametrize("raw", [False, True])
def test_attention_backward_on_another_stream_keeps_its_memory(raw):
    """The workspace that a call allocates for itself on a given stream is not
    handed to the current stream's next allocations while the call still runs."""
    q, k, ks, v, do, o, lse = inputs(2, 140, 2, 128, 32, 64, 99)
    a, ksd = dev(q, k, v, o, lse, do), ks.cuda()
    want = mc.qk_attention_backward(*a, k_shared=ksd)
    n = mc.attention_backward_workspace_size(a[0], a[1], ksd)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)      # about 10 ms
    got = mc.qk_attention_backward(*a, k_shared=ksd, stream=side.cuda_stream if raw else side)
    taken = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    taken += [torch.full_like(g, float("nan")) for g in got]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    assert mc.qk_attention_backward(*a, k_shared=ksd, stream=0)[0].shape == q.shape


@pytest.mark.parametrize("B,S,H,dh,dr,dv,causal", [
    (1, 1, 3, 128, 0, 128, True), (2, 2, 2, 64, 0, 64, True), (3, 5, 4, 24, 0, 40, False), (1, 8, 7, 64, 56, 40, True),
    (2, 15, 2, 128, 64, 128, True), (1, 16, 3, 192, 0, 128, False), (40, 16, 9, 64, 8, 128, True),
    (2, 17, 3, 80, 0, 48, True), (2, 31, 2, 128, 64, 128, True)])
def test_attention_backward_of_short_sequences(B, S, H, dh, dr, dv, causal):
    """Up to 16 positions in fp32: p and ds are not rounded, so the bounds hold
    without their operands' rounding; 17 positions take the tensor cores.  Heads
    with heavy logits among them."""
    q, k, ks, v, do, o, lse = inputs(B, S, H, dh, dr, dv, 110 + S, causal, head_scale=[1.0 + 11.0 * (h % 4 == 1) for h in range(H)])
    ref, tol = bounds(q, k, ks, v, do, o, lse, causal, operand=0.0 if S <= 16 else U)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, k, ks, v, do, o, lse = dev(q, k, ks, v, do, o, lse)
    got = mc.qk_attention_backward(q, k, v, o, lse, do, k_shared=ks, causal=causal, status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    check(got, ref, tol)


def test_attention_backward_of_single_positions_is_exact():
    """One key, and o its value: ds = do . (v - o) = 0, so dq, dk and dk_shared are 0, and dv is do."""
    mk = lambda *s: torch.randn(*s, device="cuda").to(BF16)  # noqa: E731
    q, k, ks, v, do = mk(3, 1, 5, 192), mk(3, 1, 5, 128), mk(3, 1, 64), mk(3, 1, 5, 128), mk(3, 1, 5, 128)
    lse = (torch.cat([k, ks[:, :, None].expand(3, 1, 5, 64)], -1).float() * q.float()).sum(-1).permute(0, 2, 1) / 192 ** 0.5
    dq, dk, dv, dks = mc.qk_attention_backward(q, k, v, v, lse.contiguous(), do, k_shared=ks)
    torch.cuda.synchronize()
    assert not dq.any() and not dk.any() and not dks.any()
    assert torch.equal(dv, do)


def test_attention_backward_of_short_sequences_flags_nonfinite():
    q, k, ks, v, do, o, lse = inputs(2, 9, 2, 64, 16, 64, 130)
    do[1, 5, 0, 3] = float("inf")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, k, ks, v, do, o, lse = dev(q, k, ks, v, do, o, lse)
    got = mc.qk_attention_backward(q, k, v, o, lse, do, k_shared=ks, status=st)
    torch.cuda.synchronize()
    assert st.item() & abi.MC_STATUS_NONFINITE_UPDATE
    assert all(torch.isfinite(g[0]).all() for g in got) and all(torch.isfinite(g[1, :, 1]).all() for g in got[:3])


@pytest.mark.parametrize("S,stride", [(3, (1 << 31) + 8), (20, (1 << 28) + 8)])
def test_attention_backward_offsets_past_32_bits(S, stride):
    """Positions so far apart that element offsets pass 2^31 and byte offsets 2^32,
    in inputs and outputs, by the short sequences' kernel and the tensor cores."""
    q, k, ks, v, do, o, lse = inputs(1, S, 2, 64, 16, 48, 140 + S)
    a = dev(q, k, v, o, lse, do)
    ksd = ks.cuda()
    want = mc.qk_attention_backward(*a, k_shared=ksd)
    far = torch.empty((S - 1) * stride + 1024, dtype=BF16, device="cuda")

    def spread(t, at):                     # [1, S, H, w] or [1, S, w] at `at` of each position's place
        st = (0, stride, t.shape[-1], 1) if t.dim() == 4 else (0, stride, 1)
        return far.as_strided(t.shape, st, at)
    places = [spread(t, at) for t, at in ((a[0], 0), (a[1], 160), (a[2], 288), (a[3], 384), (a[5], 480), (ksd, 576))]
    for p, t in zip(places, (a[0], a[1], a[2], a[3], a[5], ksd)):
        p.copy_(t)
    got = mc.qk_attention_backward(*places[:4], a[4], places[4], k_shared=places[5])
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    room = torch.empty_like(far)
    outs = [room.as_strided(g.shape, (0, stride, g.shape[-1], 1) if g.dim() == 4 else (0, stride, 1), at)
            for g, at in zip(want, (0, 160, 288, 384))]
    got = mc.qk_attention_backward(*a, k_shared=ksd, dq=outs[0], dk=outs[1], dv=outs[2], dk_shared=outs[3])
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))


def test_attention_backward_on_two_streams_at_once():
    sets = [dev(*(inputs(2, S, 3, 64, 0, 64, 150 + S)[i] for i in (0, 1, 3, 5, 6, 4))) for S in (16, 200, 520, 330)]
    want = [mc.qk_attention_backward(*a) for a in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = [mc.qk_attention_backward(*a, stream=s) for a, s in zip(sets, streams)]
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(w[:3], g[:3]))


def lone_query(S, q_shared, do, v, lse):
    """[1, S, 2, 64 + 16 / 64] where only query 0 and key 0 meet values: logits are 0,
    p_00 = exp(-lse), ds_00 = p do v, dv_0 = p do and, per head, the shared key's
    gradient (scale 1) is ds_00 q_shared in its first column; the rest is 0."""
    q, do_ = torch.zeros(1, S, 2, 80), torch.zeros(1, S, 2, 64)
    v_, zero = torch.zeros(1, S, 2, 64), torch.zeros(1, S, 2, 64)
    q[0, 0, :, 64] = torch.tensor(q_shared)
    do_[0, 0, :, 3] = do
    v_[0, 0, :, 3] = v
    q, do_, v_, zero = (t.to(BF16).cuda() for t in (q, do_, v_, zero))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ks, lse = torch.zeros(1, S, 16, dtype=BF16, device="cuda"), torch.full((1, 2, S), lse, device="cuda")
    got = mc.qk_attention_backward(q, zero, v_, zero, lse, do_, k_shared=ks, scale=1.0, status=st)
    torch.cuda.synchronize()
    return got, st.item()


BIG = 2.0 ** 64


@pytest.mark.parametrize("S", [1, 3, 40])
@pytest.mark.parametrize("q_shared", [[BIG, BIG], [BIG, BIG * (1 - 2.0 ** -8)]])
def test_attention_backward_flags_a_shared_key_sum_that_overflows(S, q_shared):
    """Heads whose parts are finite (up to 2^127) with a sum beyond fp32, or beyond
    what rounds to a finite bf16: dk_shared is infinite and the status says so."""
    (dq, dk, dv, dks), st = lone_query(S, q_shared, 2.0 ** 33, 2.0 ** 30, 0.0)
    assert torch.isinf(dks[0, 0, 0]) and torch.isfinite(dks[0, :, 1:]).all()
    assert all(torch.isfinite(t).all() for t in (dq, dk, dv))
    assert st & abi.MC_STATUS_NONFINITE_UPDATE
    (_, _, _, dks), st = lone_query(S, [BIG, -BIG], 2.0 ** 33, 2.0 ** 30, 0.0)
    assert st == 0 and not dks.any()                   # parts that cancel


@pytest.mark.parametrize("S", [1, 16])
def test_attention_backward_flags_values_that_round_to_infinity(S):
    """dv_0 = 1.003 times bf16's largest value: finite in fp32, infinite as stored."""
    (dq, dk, dv, dks), st = lone_query(S, [1.0, 1.0], torch.finfo(BF16).max, 0.0, -0.003)
    assert torch.isinf(dv[0, 0, :, 3]).all() and st & abi.MC_STATUS_NONFINITE_UPDATE
    (_, _, dv, _), st = lone_query(S, [1.0, 1.0], torch.finfo(BF16).max, 0.0, 0.01)
    assert torch.isfinite(dv).all() and st == 0


@pytest.mark.parametrize("B,S,H,dh,dr,dv", [(2, 131, 3, 20, 0, 50), (1, 150, 2, 64, 12, 33), (2, 9, 3, 64, 5, 17)])
def test_attention_backward_allocates_odd_widths(B, S, H, dh, dr, dv):
    """Widths that are no multiple of eight, in inputs whose rows are padded to one:
    the outputs that the call allocates itself are as good as given ones."""
    q, k, ks, v, do, o, lse = inputs(B, S, H, dh, dr, dv, 102)
    ref, tol = bounds(q, k, ks, v, do, o, lse, True)

    def wide(t):
        if t is None:
            return None
        big = torch.full((*t.shape[:-1], (t.shape[-1] + 7) // 8 * 8), float("nan"), dtype=BF16, device="cuda")
        big[..., :t.shape[-1]] = t.cuda()
        return big[..., :t.shape[-1]]
    got = mc.qk_attention_backward(*(wide(t) for t in (q, k, v, o)), lse.cuda(), wide(do), k_shared=wide(ks))
    torch.cuda.synchronize()
    assert all(g is None or g.shape == t.shape for g, t in zip(got, (q, k, v, ks)))
    check(got, ref, tol)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("B,S,H,dr", [(1, 129, 257, 0), (3, 140, 100, 0), (3, 600, 35, 8)])
def test_attention_backward_with_a_ragged_last_group_of_items(B, S, H, dr, causal):
    """More (batch, head) pairs than a group of the work order takes (512 / blocks),
    and not a multiple of it: 256 + 1, 256 + 44 and 102 + 3."""
    dh = 64 if dr else 16
    q, k, ks, v, do, o, lse = inputs(B, S, H, dh, dr, 16, 160 + S, causal)
    ref, tol = bounds(q, k, ks, v, do, o, lse, causal)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, k, ks, v, do, o, lse = dev(q, k, ks, v, do, o, lse)
    got = mc.qk_attention_backward(q, k, v, o, lse, do, k_shared=ks, causal=causal, status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    check(got, ref, tol)
