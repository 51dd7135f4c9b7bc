"""GPU parity of the packed attention (qk_attention_packed_forward, _backward) with
64-bit references, sequence by sequence and head group by head group.

Bounds (u = 2^-8: half a step of bf16, relative; w = 2^-24: of fp32), magnitudes
summed over absolute values:
  * a logit: the fp32 sum of d products and its scaling, absolute
        a_ij = w (d + 4) scale |q_i|.|k_j|
  * numerators: e = a + 2^-22 relative (the hardware's base-2 exponential), u more
    as an operand; the row sum e too, and n w for its additions
        o: sum p |v| (u + 2 e + n w), then u |o|
  * lse: the largest a of the row, 2^-21, 4 w |lse|; S_max: the largest a of the head
  * the backward's as in the dense one, with the gradients of a group's heads and their
    bounds added up: the exponent's error a + 4 w |lse|, ds = p (dp - delta): e |ds| +
    p w (d_v + 4) (|do|.|v| + |do|.|o|) and u |ds| as an operand; dq, dk: the sums of
    that with |k|, |q|, n w of the sum's magnitude, u of the result
"""
import numpy as np
import pytest
import torch

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


def features(lens, H, G, d, dv, seed=0, sharp=1.0, tail=0):
    """bf16 q, k, v, do of sum(lens) + tail tokens, and the offsets."""
    T = sum(lens) + tail
    q = synth.normal((T, H, d), 1.0, "pq", seed)
    q[:, 1::4] *= sharp
    k, v = synth.normal((T, G, d), 1.0, "pk", seed), synth.normal((T, G, dv), 1.0, "pv", seed)
    do = synth.normal((T, H, dv), 0.01, "pd", seed)
    offsets = torch.tensor([0, *np.cumsum(lens)], dtype=torch.int32)
    return [t.to(BF16).cuda() for t in (q, k, v, do)] + [offsets.cuda()]


def pieces(offsets):
    o = offsets.cpu().tolist()
    return [(a, b) for a, b in zip(o, o[1:]) if b > a]


def reference_forward(q, k, v, offsets, scale=None):
    """(o, lse, smax) and their bounds, in 64 bits."""
    Q, K, V = f64(q), f64(k), f64(v)
    T, H, d = Q.shape
    g = H // K.shape[1]
    scale = 1 / np.sqrt(d) if scale is None else scale
    o, to = np.zeros((T, H, V.shape[2])), np.zeros((T, H, V.shape[2]))
    lse, tl = np.zeros((H, T)), np.zeros((H, T))
    smax, ts = np.full(H, -np.inf), np.zeros(H)
    for a, b in pieces(offsets):
        n = b - a
        mask = np.tril(np.ones((n, n), bool))
        for h in range(H):
            qq, kk, vv = Q[a:b, h], K[a:b, h // g], V[a:b, h // g]
            s = np.where(mask, scale * qq @ kk.T, -np.inf)
            err = np.where(mask, W * (d + 4) * scale * (np.abs(qq) @ np.abs(kk).T), 0.0)
            top = s.max(1, keepdims=True)
            p = np.exp(s - top)
            total = p.sum(1, keepdims=True)
            p /= total
            o[a:b, h] = p @ vv
            e = err + err.max(1, keepdims=True) + 2 * 2.0 ** -22
            to[a:b, h] = (p * (U + e + n * W)) @ np.abs(vv) * 1.01 + U * np.abs(o[a:b, h]) + 1e-30
            lse[h, a:b] = (top + np.log(total))[:, 0]
            tl[h, a:b] = err.max(1) + 2.0 ** -21 + 4 * W * np.abs(lse[h, a:b])
            smax[h] = max(smax[h], s.max())
            ts[h] = max(ts[h], err.max())
    return (o, lse, smax), (to, tl, ts + 1e-12)


def check_forward(got, q, k, v, offsets, scale=None):
    ref, tol = reference_forward(q, k, v, offsets, scale)
    rows = np.zeros(q.shape[0], bool)
    for a, b in pieces(offsets):
        rows[a:b] = True
    for name, x, r, t, keep in zip(("o", "lse", "smax"), got, ref, tol, (rows, (slice(None), rows), slice(None))):
        err, t = np.abs(f64(x)[keep] - r[keep]), t[keep]
        assert np.all(err <= t), f"{name}: {int(np.sum(~(err <= t)))} of {err.size} outside, max err {np.nanmax(err):.3g}"


# lengths, query heads, key heads, d, d_v
CASES = [
    ([1], 1, 1, 64, 64),
    ([1], 2, 1, 16, 16),
    ([128], 2, 2, 128, 128),
    ([129], 4, 1, 128, 128),
    ([127, 1, 130], 3, 1, 128, 64),
    ([256, 257, 255], 1, 1, 64, 128),
    ([1, 1, 1, 1, 5], 6, 3, 80, 48),
    ([0, 300, 0, 0, 7, 0], 8, 2, 24, 72),
    ([385], 5, 5, 40, 120),
    ([700, 3, 511], 6, 2, 128, 128),
    ([64, 700], 8, 1, 112, 96),
]


@pytest.mark.parametrize("lens,H,G,d,dv", CASES)
def test_forward_parity(lens, H, G, d, dv):
    q, k, v, _, offsets = features(lens, H, G, d, dv, seed=sum(lens), sharp=8.0)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = mc.qk_attention_packed_forward(q, k, v, offsets, lse=True, status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    check_forward(got, q, k, v, offsets)
    again = mc.qk_attention_packed_forward(q, k, v, offsets, lse=True)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_forward_many_sequences_against_one_by_one():
    """More sequences than one step of the plan's scans takes, most of them short: equal bits with
    each sequence alone."""
    rng = np.random.RandomState(3)
    lens = [int(x) for x in rng.randint(0, 9, 2500)]
    lens[7], lens[1400] = 200, 333
    q, k, v, _, offsets = features(lens, 2, 1, 32, 32)
    o, lse, smax = mc.qk_attention_packed_forward(q, k, v, offsets, lse=True)
    torch.cuda.synchronize()
    at = offsets.cpu().tolist()
    best = torch.full((2,), -np.inf, device="cuda")
    for s in [7, 1400, *range(0, 2500, 97)]:
        a, b = at[s], at[s + 1]
        if a == b:
            continue
        one = torch.tensor([0, b - a], dtype=torch.int32, device="cuda")
        x, y, z = mc.qk_attention_packed_forward(q[a:b], k[a:b], v[a:b], one, lse=True)
        assert torch.equal(x, o[a:b]) and torch.equal(y, lse[:, a:b])
        best = torch.maximum(best, z)
    assert torch.all(best <= smax)


def test_forward_equals_the_dense_one():
    """Sequences of one length without groups: the dense call's problem."""
    B, S, H, d = 3, 300, 4, 128
    q, k, v, _, offsets = features([S] * B, H, H, d, d, sharp=8.0)
    o, lse, smax = mc.qk_attention_packed_forward(q, k, v, offsets, lse=True)
    dense = [t.view(B, S, H, d) for t in (q, k, v)]
    od, ld, sd = mc.qk_attention_forward(*dense, lse=True)
    torch.cuda.synchronize()
    assert torch.equal(smax, sd)
    assert torch.all((o.view(B, S, H, d).float() - od.float()).abs() <= 4 * U * od.float().abs() + 1e-2)
    assert torch.all((lse - ld.permute(1, 0, 2).reshape(H, -1)).abs() <= 1e-5)


def test_rows_of_no_sequence_stay(tail=37):
    """Tokens before the first offset and behind the last belong to no sequence: whatever they hold
    (NaN here) reaches nothing, and the outputs' rows stay as they were."""
    lens, H, G, d = [130, 40], 4, 2, 64
    q, k, v, _, offsets = features(lens, H, G, d, d, tail=tail)
    q2, k2, v2 = (torch.cat([t[-tail:], t[:-tail]]) for t in (q, k, v))      # the strangers first
    n = sum(lens)
    want = mc.qk_attention_packed_forward(q[:n], k[:n], v[:n], offsets, lse=True)
    for a, b, c, off, own in ((q, k, v, offsets, slice(0, n)), (q2, k2, v2, offsets + tail, slice(tail, n + tail))):
        for t in (a, b, c):
            keep = t[own].clone()
            t.fill_(float("nan"))
            t[own] = keep
        out = torch.full_like(a, 7.0)
        lse = torch.full((H, n + tail), 7.0, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = mc.qk_attention_packed_forward(a, b, c, off, out=out, lse=lse, status=st)
        torch.cuda.synchronize()
        assert st.item() == 0
        other = torch.ones(n + tail, dtype=torch.bool, device="cuda")
        other[own] = False
        assert torch.all(out[other] == 7.0) and torch.all(lse[:, other] == 7.0)
        assert torch.equal(out[own], want[0]) and torch.equal(lse[:, own], want[1]) and torch.equal(got[2], want[2])


def test_nonfinite_sequences_keep_to_themselves():
    lens, H, G, d = [100, 150, 60, 90], 4, 1, 128
    q, k, v, _, offsets = features(lens, H, G, d, d)
    want = mc.qk_attention_packed_forward(q, k, v, offsets, lse=True)
    k[120, 0, 3], v[200, 0, 5], q[255, 2, 1] = float("inf"), float("nan"), float("nan")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = mc.qk_attention_packed_forward(q, k, v, offsets, lse=True, status=st)
    torch.cuda.synchronize()
    assert st.item() == abi.MC_STATUS_NONFINITE_LOGIT
    keep = torch.ones(400, dtype=torch.bool, device="cuda")
    keep[100:310] = False
    assert torch.equal(got[0][keep], want[0][keep]) and torch.equal(got[1][:, keep], want[1][:, keep])
    assert not torch.isfinite(got[0][240]).all()


def test_bad_offsets_are_clamped():
    """Offsets that decrease or leave [0, T]: the status says so, the sequences are those of the
    offsets made monotone, and nothing lies outside."""
    q, k, v, _, _ = features([300], 2, 1, 64, 64)
    bad = torch.tensor([-5, 100, 60, 900, 900], dtype=torch.int32, device="cuda")
    good = torch.tensor([0, 100, 100, 300, 300], dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = mc.qk_attention_packed_forward(q, k, v, bad, lse=True, status=st)
    want = mc.qk_attention_packed_forward(q, k, v, good, lse=True)
    torch.cuda.synchronize()
    assert st.item() == abi.MC_STATUS_BAD_OFFSETS
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_accumulate_and_no_tokens():
    q, k, v, _, offsets = features([50, 70], 4, 2, 64, 64)
    _, _, s = mc.qk_attention_packed_forward(q, k, v, offsets)
    high = torch.tensor([1e3, -1e3, 1e3, -1e3], device="cuda")
    _, _, t = mc.qk_attention_packed_forward(q, k, v, offsets, smax=high.clone(), accumulate=True)
    empty = torch.zeros(3, dtype=torch.int32, device="cuda")
    _, _, none = mc.qk_attention_packed_forward(q, k, v, empty)
    _, _, gone = mc.qk_attention_packed_forward(q[:0], k[:0], v[:0], empty)
    torch.cuda.synchronize()
    assert torch.equal(t, torch.maximum(high, s))
    assert torch.all(none == -float("inf")) and torch.all(gone == -float("inf"))


def test_views_streams_and_scale():
    """q, k and v as views of one projection, out in a wider buffer, another stream, an explicit scale."""
    T, H, G, d = 260, 4, 2, 64
    both = synth.normal((T, H + 2 * G, d), 1.0, "views", 1).to(BF16).cuda()
    q, k, v = both[:, :H], both[:, H:H + G], both[:, H + G:]
    offsets = torch.tensor([0, 200, 260], dtype=torch.int32, device="cuda")
    wide = torch.full((T, H, d + 24), 7.0, dtype=BF16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mc.qk_attention_packed_forward(q, k, v, offsets, scale=0.3, out=wide[..., 8:8 + d], lse=True, stream=side)
    torch.cuda.synchronize()
    check_forward(got, q, k, v, offsets, 0.3)
    assert torch.all(wide[..., :8] == 7.0) and torch.all(wide[..., 8 + d:] == 7.0)
    # heads outside the tokens
    head_major = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v)]
    again = mc.qk_attention_packed_forward(*head_major, offsets, scale=0.3, lse=True)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_forward_captured_with_new_offsets():
    q, k, v, _, offsets = features([100, 156], 4, 2, 64, 64)
    other = torch.tensor([0, 30, 256], dtype=torch.int32, device="cuda")
    want = [mc.qk_attention_packed_forward(q, k, v, o, lse=True) for o in (offsets, other)]
    torch.cuda.synchronize()
    held = offsets.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = mc.qk_attention_packed_forward(q, k, v, held, lse=True)
    for o, w in zip((offsets, other), want):
        held.copy_(o)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, w))


def test_long_sequence_against_a_plain_form():
    """A length off every tile over many key blocks, by a plain fp64 form on the device: o within u
    of the operands and u of the result, with a tenth for the fp32 errors."""
    n, H, G, d = 5003, 4, 2, 128
    q, k, v, _, offsets = features([n], H, G, d, d, sharp=8.0)
    o, lse, smax = mc.qk_attention_packed_forward(q, k, v, offsets, lse=True)
    mask = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
    for h in range(H):
        s = (q[:, h].double() @ k[:, h // 2].double().t()) / d ** 0.5
        s = s.masked_fill(~mask, -float("inf"))
        p = torch.softmax(s, -1)
        ref, mag = p @ v[:, h // 2].double(), p @ v[:, h // 2].double().abs()
        assert torch.all((o[:, h].double() - ref).abs() <= 1.1 * U * mag + U * ref.abs())
        assert torch.all((lse[h].double() - torch.logsumexp(s, -1)).abs() <= 1e-4)
        assert abs(float(smax[h]) - float(s.max())) <= 1e-4


# --------------------------------------------------------------------------------------- backward
def reference_backward(q, k, v, o, lse, do, offsets, scale=None, of_o=0.0):
    """(dq, dk, dv) and their bounds, in 64 bits; of_o: relative error of o that delta takes on."""
    Q, K, V, OG, L, DO = (f64(t) for t in (q, k, v, o, lse, do))
    T, H, d = Q.shape
    dvw = V.shape[2]
    g = H // K.shape[1]
    scale = 1 / np.sqrt(d) if scale is None else scale
    out = [np.zeros_like(x) for x in (Q, K, V)]
    tol = [np.zeros_like(x) for x in (Q, K, V)]
    for a, b in pieces(offsets):
        n = b - a
        mask = np.tril(np.ones((n, n), bool))
        for h in range(H):
            qq, kk, vv, oo, dd = Q[a:b, h], K[a:b, h // g], V[a:b, h // g], OG[a:b, h], DO[a:b, h]
            p = np.where(mask, np.exp(np.minimum(scale * qq @ kk.T - L[h, a:b][:, None], 700.0)), 0.0)
            e = W * (d + 4) * scale * (np.abs(qq) @ np.abs(kk).T) + 4 * W * np.abs(L[h, a:b])[:, None] + 2.0 ** -22
            ds = p * (dd @ vv.T - np.sum(dd * oo, 1)[:, None])
            mags = np.abs(dd) @ np.abs(vv).T + np.sum(np.abs(dd) * np.abs(oo), 1)[:, None]
            err = (e + U) * np.abs(ds) + p * (1 + e + U) * W * (dvw + 4) * mags
            err += p * of_o * np.sum(np.abs(dd) * np.abs(oo), 1)[:, None]
            ds[0], err[0] = 0.0, 0.0                     # one key
            out[0][a:b, h] = scale * ds @ kk
            out[1][a:b, h // g] += scale * ds.T @ qq
            out[2][a:b, h // g] += p.T @ dd
            tol[0][a:b, h] = scale * (err + n * W * np.abs(ds)) @ np.abs(kk)
            tol[1][a:b, h // g] += scale * (err + g * n * W * np.abs(ds)).T @ np.abs(qq)
            tol[2][a:b, h // g] += ((U + e + g * n * W) * p).T @ np.abs(dd)
    return out, [x * 1.01 + U * np.abs(r) + 1e-30 for r, x in zip(out, tol)]


def check_backward(got, *args):
    ref, tol = reference_backward(*args)
    rows = np.zeros(ref[0].shape[0], bool)
    for a, b in pieces(args[6]):
        rows[a:b] = True
    for name, x, r, t in zip(("dq", "dk", "dv"), got, ref, tol):
        err = np.abs(f64(x) - r)[rows]
        assert np.all(err <= t[rows]), f"{name}: {int(np.sum(~(err <= t[rows])))} of {err.size} outside, max err {np.nanmax(err):.3g}"


def with_forward(lens, H, G, d, dv, **kw):
    q, k, v, do, offsets = features(lens, H, G, d, dv, **kw)
    o, lse, _ = mc.qk_attention_packed_forward(q, k, v, offsets, lse=True)
    return q, k, v, o, lse, do, offsets


@pytest.mark.parametrize("lens,H,G,d,dv", CASES)
def test_backward_parity(lens, H, G, d, dv):
    args = with_forward(lens, H, G, d, dv, seed=sum(lens), sharp=8.0)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = mc.qk_attention_packed_backward(*args, status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    check_backward(got, *args)
    again = mc.qk_attention_packed_backward(*args)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_backward_of_single_tokens_is_zero():
    """Sequences of one token: dq and dk are exactly 0, dv is the group's sum of do."""
    args = with_forward([1] * 70, 6, 2, 64, 64)
    dq, dk, dv = mc.qk_attention_packed_backward(*args)
    torch.cuda.synchronize()
    assert torch.all(dq == 0) and torch.all(dk == 0)
    want = args[5].double().view(70, 2, 3, 64).sum(2)
    assert torch.all((dv.double() - want).abs() <= U * want.abs() + 1e-7)


def test_backward_many_sequences_against_one_by_one():
    rng = np.random.RandomState(4)
    lens = [int(x) for x in rng.randint(0, 9, 1500)]
    lens[3], lens[1100] = 200, 333
    q, k, v, o, lse, do, offsets = with_forward(lens, 4, 2, 32, 32)
    got = mc.qk_attention_packed_backward(q, k, v, o, lse, do, offsets)
    torch.cuda.synchronize()
    at = offsets.cpu().tolist()
    for s in [3, 1100, *range(0, 1500, 131)]:
        a, b = at[s], at[s + 1]
        if a == b:
            continue
        one = torch.tensor([0, b - a], dtype=torch.int32, device="cuda")
        alone = mc.qk_attention_packed_backward(q[a:b], k[a:b], v[a:b], o[a:b], lse[:, a:b].contiguous(), do[a:b], one)
        assert all(torch.equal(x, y[a:b]) for x, y in zip(alone, got))


def test_backward_rows_of_no_sequence_stay_and_outputs_interleave():
    """Strangers' rows hold NaN and reach nothing; the gradients are views of one buffer, as those
    of a joint projection."""
    lens, H, G, d, tail = [130, 40], 4, 2, 64, 50
    q, k, v, do, offsets = features(lens, H, G, d, d, tail=tail)
    n = sum(lens)
    o, lse, _ = mc.qk_attention_packed_forward(q, k, v, offsets, lse=True)
    want = mc.qk_attention_packed_backward(q[:n], k[:n], v[:n], o[:n], lse[:, :n].contiguous(), do[:n], offsets)
    for t in (q, k, v, o, do):
        t[n:] = float("nan")
    lse[:, n:] = float("nan")
    both = torch.full((n + tail, H + 2 * G, d + 8), 7.0, dtype=BF16, device="cuda")
    dq, dk, dv = both[:, :H, :d], both[:, H:H + G, :d], both[:, H + G:, :d]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    mc.qk_attention_packed_backward(q, k, v, o, lse, do, offsets, dq=dq, dk=dk, dv=dv, status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    assert all(torch.equal(x[:n], y) for x, y in zip((dq, dk, dv), want))
    assert torch.all(both[n:] == 7.0) and torch.all(both[..., d:] == 7.0)


def test_backward_nonfinite_sequences_keep_to_themselves():
    lens, H, G, d = [100, 150, 60, 90], 4, 1, 128
    q, k, v, o, lse, do, offsets = with_forward(lens, H, G, d, d)
    want = mc.qk_attention_packed_backward(q, k, v, o, lse, do, offsets)
    k[120, 0, 3], v[200, 0, 5], do[255, 2, 1] = float("inf"), float("nan"), float("nan")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = mc.qk_attention_packed_backward(q, k, v, o, lse, do, offsets, status=st)
    torch.cuda.synchronize()
    assert st.item() == abi.MC_STATUS_NONFINITE_UPDATE
    keep = torch.ones(400, dtype=torch.bool, device="cuda")
    keep[100:310] = False
    assert all(torch.equal(x[keep], y[keep]) for x, y in zip(got, want))


def test_backward_equals_the_dense_one():
    """Sequences of one length without groups: the dense call's problem, tile by tile the same
    products but for the first query, whose ds is zero here and rounding noise there."""
    B, S, H, d = 2, 400, 3, 128
    q, k, v, o, lse, do, offsets = with_forward([S] * B, H, H, d, d)
    got = mc.qk_attention_packed_backward(q, k, v, o, lse, do, offsets)
    D = [t.view(B, S, H, d) for t in (q, k, v, o)]
    ld = lse.view(H, B, S).permute(1, 0, 2).contiguous()
    dense = mc.qk_attention_backward(*D, ld, do.view(B, S, H, d))
    torch.cuda.synchronize()
    for x, y in zip(got, dense):
        y = y.reshape(B * S, H, d).float()
        assert torch.all((x.float() - y).abs() <= 2 * U * y.abs() + 1e-6)


def test_backward_captured_with_new_offsets():
    q, k, v, do, offsets = features([100, 156], 4, 2, 64, 64)
    other = torch.tensor([0, 30, 256], dtype=torch.int32, device="cuda")
    want = []
    for o in (offsets, other):
        out, lse, _ = mc.qk_attention_packed_forward(q, k, v, o, lse=True)
        want.append(mc.qk_attention_packed_backward(q, k, v, out, lse, do, o))
    torch.cuda.synchronize()
    held = offsets.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse, _ = mc.qk_attention_packed_forward(q, k, v, held, lse=True)
        got = mc.qk_attention_packed_backward(q, k, v, out, lse, do, held)
    for o, w in zip((offsets, other), want):
        held.copy_(o)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, w))


def test_gradient_against_differences():
    """sum(do * o) differentiated numerically in 64 bits, at a few elements, within the bounds with
    the rounding of o (u) added; the differences are good to 1e-8."""
    lens, H, G, d = [9, 14], 4, 2, 16
    q, k, v, o, lse, do, offsets = with_forward(lens, H, G, d, d)
    got = mc.qk_attention_packed_backward(q, k, v, o, lse, do, offsets)
    torch.cuda.synchronize()
    _, tol = reference_backward(q, k, v, o, lse, do, offsets, of_o=1.01 * U)
    X = [f64(t) for t in (q, k, v)]
    DO = f64(do)

    def f(Q, K, V):
        total = 0.0
        for a, b in pieces(offsets):
            m = np.tril(np.ones((b - a, b - a), bool))
            for h in range(H):
                s = np.where(m, Q[a:b, h] @ K[a:b, h // 2].T / np.sqrt(d), -np.inf)
                p = np.exp(s - s.max(1, keepdims=True))
                total += ((p / p.sum(1, keepdims=True) @ V[a:b, h // 2]) * DO[a:b, h]).sum()
        return total

    rng = np.random.RandomState(0)
    for n in range(3):
        for _ in range(25):
            i = tuple(rng.randint(0, x) for x in X[n].shape)
            up, down = [x.copy() for x in X], [x.copy() for x in X]
            up[n][i] += 1e-5
            down[n][i] -= 1e-5
            slope = (f(*up) - f(*down)) / 2e-5
            assert abs(slope - f64(got[n])[i]) <= tol[n][i] + 1e-8


def test_backward_long_group_against_a_plain_form():
    """Several tiles of several heads per key head at a long odd length; the sums in fp64 on the
    device, errors in the 2-norm: p and ds as bf16 operands 2^-9 each at random, results 2^-9."""
    n, H, G, d = 3001, 6, 2, 128
    q, k, v, o, lse, do, offsets = with_forward([n], H, G, d, d, sharp=4.0)
    dq, dk, dv = mc.qk_attention_packed_backward(q, k, v, o, lse, do, offsets)
    mask = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
    rk, rv = torch.zeros_like(dk, dtype=torch.float64), torch.zeros_like(dv, dtype=torch.float64)
    for h in range(H):
        Q, K, V, DO = q[:, h].double(), k[:, h // 3].double(), v[:, h // 3].double(), do[:, h].double()
        p = torch.exp((Q @ K.t()) / d ** 0.5 - lse[h].double()[:, None]).masked_fill(~mask, 0.0)
        ds = p * (DO @ V.t() - (DO * o[:, h].double()).sum(-1, keepdim=True))
        rq = ds @ K / d ** 0.5
        assert (dq[:, h].double() - rq).norm() <= 0.004 * rq.norm()
        rk[:, h // 3] += ds.t() @ Q / d ** 0.5
        rv[:, h // 3] += p.t() @ DO
    assert (dk.double() - rk).norm() <= 0.004 * rk.norm() and (dv.double() - rv).norm() <= 0.004 * rv.norm()


def test_plan_in_the_workspace_equals_that_in_shared_memory():
    """9000 sequences' lists stay in the workspace, 3000's in shared memory: equal bits, forward
    and backward."""
    rng = np.random.RandomState(5)
    lens = [int(x) for x in rng.randint(0, 5, 9000)]
    lens[17], lens[8000] = 300, 140
    args = with_forward(lens, 2, 1, 32, 32)
    q, k, v, o, lse, do, offsets = args
    got = mc.qk_attention_packed_backward(*args)
    for i in range(0, 9000, 3000):
        part = offsets[i:i + 3001]
        a, b = int(part[0]), int(part[-1])
        one = (part - a).contiguous()
        x, y, _ = mc.qk_attention_packed_forward(q[a:b], k[a:b], v[a:b], one, lse=True)
        assert torch.equal(x, o[a:b]) and torch.equal(y, lse[:, a:b])
        alone = mc.qk_attention_packed_backward(q[a:b], k[a:b], v[a:b], x, y, do[a:b], one)
        assert all(torch.equal(m, n[a:b]) for m, n in zip(alone, got))


@pytest.mark.parametrize("axis", ["heads", "tokens"])
def test_broadcast_inputs(axis):
    """Inputs whose heads, or tokens, share memory are read as the rows that they stand for."""
    lens, H, G, d = [140, 1, 75], 4, 2, 64
    q, k, v, do, offsets = features(lens, H, G, d, d)
    if axis == "heads":
        views = [t[:, :1].expand_as(t) for t in (q, k, v, do)]
    else:
        views = [t[:1].expand_as(t) for t in (q, k, v, do)]
    whole = [t.contiguous() for t in views]
    out = []
    for a, b, c, g in (views, whole):
        o, lse, smax = mc.qk_attention_packed_forward(a, b, c, offsets, lse=True)
        out.append((o, lse, smax, *mc.qk_attention_packed_backward(a, b, c, o, lse, g, offsets)))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(*out))


def test_calls_of_several_host_threads():
    """Threads on streams of their own, each with other widths and first uses: the bits of calls
    that each wait for the one before."""
    import threading
    shapes = [([300, 40], 4, 2, 64, 64), ([129], 6, 3, 128, 128), ([5] * 20, 3, 1, 80, 48), ([200, 17], 2, 2, 24, 128)]
    data = [with_forward(*s, seed=i) for i, s in enumerate(shapes)]
    want = [mc.qk_attention_packed_backward(*a) for a in data]
    torch.cuda.synchronize()
    got, errors = [None] * len(shapes), []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            for _ in range(20):
                q, k, v, o, lse, do, offsets = data[i]
                o2, lse2, _ = mc.qk_attention_packed_forward(q, k, v, offsets, lse=True, stream=stream)
                got[i] = mc.qk_attention_packed_backward(q, k, v, o2, lse2, do, offsets, stream=stream)
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(shapes))]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors
    assert all(torch.equal(a, b) for x, y in zip(got, want) for a, b in zip(x, y))


def poison(*like):
    """Freed memory of these shapes and types that holds NaN, for the next allocations to find."""
    held = [torch.full_like(t, float("nan")) for t in like for _ in range(2)]
    torch.cuda.synchronize()
    del held


@pytest.mark.parametrize("lead,tail", [(0, 37), (150, 0), (3, 700), (0, 0)])
@pytest.mark.parametrize("H,G,d,dv", [(4, 2, 64, 64), (3, 1, 80, 48), (1, 1, 16, 128)])
def test_new_outputs_hold_nothing_where_there_is_no_sequence(H, G, d, dv, lead, tail):
    """Outputs that a call allocates: zeros (lse: -inf) in the rows of tokens in no sequence, whatever
    the memory held; the other rows as without such tokens.  A given output keeps its rows."""
    lens = [130, 0, 41]
    n = sum(lens)
    q, k, v, do, offsets = features(lens, H, G, d, dv)
    o, lse, smax = mc.qk_attention_packed_forward(q, k, v, offsets, lse=True)
    grads = mc.qk_attention_packed_backward(q, k, v, o, lse, do, offsets)
    wide = lambda t: torch.cat([torch.full_like(t[:1], float("nan")).expand(lead, -1, -1), t,  # noqa: E731
                                torch.full_like(t[:1], float("nan")).expand(tail, -1, -1)])
    Q, K, V, DO, moved = wide(q), wide(k), wide(v), wide(do), offsets + lead
    T, own = lead + n + tail, slice(lead, lead + n)
    other = torch.ones(T, dtype=torch.bool, device="cuda")
    other[own] = False
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    poison(wide(o), torch.empty(H, T, device="cuda"))
    O2, L2, s2 = mc.qk_attention_packed_forward(Q, K, V, moved, lse=True, status=st)
    assert torch.equal(O2[own], o) and torch.equal(L2[:, own], lse) and torch.equal(s2, smax)
    assert torch.all(O2[other] == 0) and torch.all(L2[:, other] == -float("inf"))
    poison(Q, K, V)
    got = mc.qk_attention_packed_backward(Q, K, V, O2, L2, DO, moved, status=st)
    for x, y in zip(got, grads):
        assert torch.equal(x[own], y) and torch.all(x[other] == 0)
    held = torch.full_like(K, 7.0)
    dq, dk, dvv = mc.qk_attention_packed_backward(Q, K, V, O2, L2, DO, moved, dk=held, status=st)
    torch.cuda.synchronize()
    assert st.item() == 0 and dk is held and torch.all(held[other] == 7.0)
    assert torch.all(dq[other] == 0) and torch.all(dvv[other] == 0)


def test_only_strangers():
    """Offsets that leave every token out: outputs of nothing."""
    q, k, v, do, _ = features([50], 4, 2, 64, 64)
    for at in (0, 20, 50):
        offsets = torch.full((4,), at, dtype=torch.int32, device="cuda")
        poison(q, torch.empty(4, 50, device="cuda"))
        o, lse, smax = mc.qk_attention_packed_forward(q, k, v, offsets, lse=True)
        poison(q, k, v)
        grads = mc.qk_attention_packed_backward(q, k, v, o, lse, do, offsets)
        torch.cuda.synchronize()
        assert torch.all(o == 0) and torch.all(lse == -float("inf")) and torch.all(smax == -float("inf"))
        assert all(torch.all(x == 0) for x in grads)


def test_allocation_that_fails_raises_torchs_error():
    """Views of a few values that stand for more rows than memory holds: the outputs cannot be allocated,
    torch says so, and the next call works."""
    x = torch.ones(1, 1, 128, dtype=BF16, device="cuda")
    q, k = x.expand(1 << 28, 16, 128), x.expand(1 << 28, 1, 128)           # 1.1 TB of q
    offsets = torch.tensor([0, 1 << 28], dtype=torch.int32, device="cuda")
    for call in (lambda: mc.qk_attention_packed_forward(q, k, k, offsets), lambda: mc.qk_norm_rope(q, k)):
        with pytest.raises(torch.cuda.OutOfMemoryError):
            call()
    y, _, _ = mc.qk_norm_rope(x)
    torch.cuda.synchronize()
    assert torch.isfinite(y).all()


@pytest.mark.parametrize("lens,H,G,d,dv", [([70, 1, 200], 4, 2, 17, 33), ([300], 6, 2, 90, 20), ([129, 15], 1, 1, 127, 125),
                                           ([512], 16, 1, 30, 18), ([5] * 40, 3, 1, 100, 63)])
def test_widths_that_are_no_multiple_of_eight(lens, H, G, d, dv):
    """Rows padded to whole 16 bytes: what lies behind the features (NaN here) is neither read nor
    written, and outputs that the call allocates have such rows."""
    def pad(t, fill):
        held = torch.full((*t.shape[:2], (t.shape[2] + 7) // 8 * 8 + 8), fill, dtype=BF16, device="cuda")
        held[..., :t.shape[2]] = t
        return held[..., :t.shape[2]], held[..., t.shape[2]:]

    q, k, v, do, offsets = features(lens, H, G, d, dv, seed=d, sharp=4.0)
    (q, _), (k, _), (v, _), (do, _) = (pad(t, float("nan")) for t in (q, k, v, do))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = mc.qk_attention_packed_forward(q, k, v, offsets, lse=True, status=st)
    torch.cuda.synchronize()
    assert st.item() == 0 and got[0].stride(1) % 8 == 0
    check_forward(got, q, k, v, offsets)
    out, rest = pad(torch.zeros_like(got[0]), 7.0)
    mc.qk_attention_packed_forward(q, k, v, offsets, out=out)
    assert torch.equal(out, got[0]) and torch.all(rest == 7.0)
    o, lse, _ = got
    args = (q, k, v, o, lse, do, offsets)
    grads = mc.qk_attention_packed_backward(*args, status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    check_backward(grads, *args)
    held = [pad(torch.zeros_like(t), 7.0) for t in (q, k, v)]
    again = mc.qk_attention_packed_backward(*args, dq=held[0][0], dk=held[1][0], dv=held[2][0])
    assert all(torch.equal(x, y) for x, y in zip(again, grads)) and all(torch.all(r == 7.0) for _, r in held)
