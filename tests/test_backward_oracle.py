"""Pins of the oracle's gradients that are independent of their formulas:
central differences of the oracle's forward functions, and closed forms."""
import numpy as np
import pytest

import oracle as O


def rnd(rng, *shape):
    return rng.standard_normal(shape)


@pytest.mark.parametrize("causal,dr", [(True, 0), (False, 0), (True, 4)])
def test_attention_backward_matches_differences(causal, dr):
    rng = np.random.default_rng(3)
    B, S, H, dk, dv = 2, 5, 3, 4, 6
    Q, K, V, dO = rnd(rng, B, S, H, dk + dr), rnd(rng, B, S, H, dk), rnd(rng, B, S, H, dv), rnd(rng, B, S, H, dv)
    Ks = rnd(rng, B, S, dr) if dr else None

    def loss():
        return float(np.sum(O.attention_forward(Q, K, V, Ks, causal=causal)[0] * dO))

    out, lse, _ = O.attention_forward(Q, K, V, Ks, causal=causal)
    grads = O.attention_backward(Q, K, V, out, lse, dO, Ks, causal=causal)
    eps = 1e-5
    for x, g in zip((Q, K, V, Ks), grads):
        if x is None:
            assert g is None
            continue
        assert g.shape == x.shape
        for idx in np.ndindex(*x.shape):
            if rng.random() > 0.3:
                continue
            keep = x[idx]
            x[idx] = keep + eps
            up = loss()
            x[idx] = keep - eps
            down = loss()
            x[idx] = keep
            assert abs((up - down) / (2 * eps) - g[idx]) < 1e-7, (idx, g[idx])


def test_attention_backward_closed_forms():
    """One token: the output is v whatever q and k are.  Equal keys: dV of an
    unmasked layer is the mean of dO over the queries, dQ is zero."""
    rng = np.random.default_rng(4)
    Q, K, V, dO = (rnd(rng, 1, 1, 2, 8) for _ in range(4))
    out, lse, _ = O.attention_forward(Q, K, V)
    dQ, dK, dV, _ = O.attention_backward(Q, K, V, out, lse, dO)
    assert np.allclose(dV, dO) and np.allclose(dQ, 0) and np.allclose(dK, 0)
    S = 7
    Q, V, dO = rnd(rng, 1, S, 1, 8), rnd(rng, 1, S, 1, 8), rnd(rng, 1, S, 1, 8)
    K = np.broadcast_to(rnd(rng, 1, 1, 1, 8), (1, S, 1, 8))
    out, lse, _ = O.attention_forward(Q, K, V, causal=False)
    dQ, dK, dV, _ = O.attention_backward(Q, K, V, out, lse, dO, causal=False)
    assert np.allclose(dV, np.broadcast_to(dO.mean(axis=1, keepdims=True), dV.shape))
    assert np.allclose(dQ, 0)          # sum_j ds_ij = 0 and every key is the same


@pytest.mark.parametrize("mistake", ["scale", "delta", "causal", "shared_mean"])
def test_attention_backward_catches_planted_mistakes(mistake):
    """A dropped scale, a dropped delta, a missing mask and a mean over the heads
    each move some gradient by far more than the differences' error."""
    rng = np.random.default_rng(5)
    B, S, H, dk, dr, dv = 1, 6, 2, 4, 2, 4
    Q, K, V, dO = rnd(rng, B, S, H, dk + dr), rnd(rng, B, S, H, dk), rnd(rng, B, S, H, dv), rnd(rng, B, S, H, dv)
    Ks = rnd(rng, B, S, dr)
    out, lse, _ = O.attention_forward(Q, K, V, Ks)
    right = O.attention_backward(Q, K, V, out, lse, dO, Ks)
    wrong = {
        "scale": lambda: O.attention_backward(Q, K, V, out, lse, dO, Ks, scale=1.0),
        "delta": lambda: O.attention_backward(Q, K, V, 0 * out, lse, dO, Ks),
        "causal": lambda: O.attention_backward(Q, K, V, out, lse, dO, Ks, causal=False),
        "shared_mean": lambda: right[:3] + (right[3] / H,),
    }[mistake]()
    assert max(np.max(np.abs(a - b)) for a, b in zip(right, wrong)) > 1e-2


def test_rms_norm_backward_matches_differences():
    rng = np.random.default_rng(6)
    h, w, dy = rnd(rng, 3, 7), 1 + 0.3 * rnd(rng, 7), rnd(rng, 3, 7)
    eps = 0.05
    rstd = 1 / np.sqrt(np.mean(h * h, 1) + eps)
    loss = lambda: float(np.sum(O.rms_norm(h, eps) * w * dy))  # noqa: E731
    dx, dw = O.rms_norm_backward(dy, h, rstd, w)
    for x, g in ((h, dx), (w, dw)):
        for idx in np.ndindex(*x.shape):
            keep = x[idx]
            x[idx] = keep + 1e-5
            up = loss()
            x[idx] = keep - 1e-5
            down = loss()
            x[idx] = keep
            assert abs((up - down) / 2e-5 - g[idx]) < 1e-8
    assert np.allclose(O.rms_norm_backward(dy, h, rstd, w, dres=h)[0], dx + h)
    # a missing mean term or weight is far off
    assert np.max(np.abs(rstd[:, None] * dy * w - dx)) > 1e-2
    assert np.max(np.abs(O.rms_norm_backward(dy, h, rstd)[0] - dx)) > 1e-2


def test_rope_backward_is_the_transpose():
    """<rope(x), dy> = <x, rope_backward(dy)>, and it undoes the rotation."""
    rng = np.random.default_rng(7)
    x, dy = rnd(rng, 2, 9, 3, 6), rnd(rng, 2, 9, 3, 6)
    assert abs(np.sum(O.rope(x) * dy) - np.sum(x * O.rope_backward(dy))) < 1e-10
    assert np.allclose(O.rope_backward(O.rope(x, 77.0), 77.0), x)
    assert np.max(np.abs(O.rope(dy) - O.rope_backward(dy))) > 0.1     # the direction matters


def test_e4m3_rounding():
    """Every e4m3 value is kept, midpoints go to even, small ones to the 2^-9 grid."""
    vals = sorted({m / 8 * 2.0 ** e for e in range(-6, 9) for m in range(8, 16)} | {m * 2.0 ** -9 for m in range(8)})
    vals = np.array([v for v in vals if v <= 448.0])
    assert len(vals) == 127                               # 7 f is NaN
    assert np.array_equal(O.round_to_e4m3(vals), vals) and np.array_equal(O.round_to_e4m3(-vals), -vals)
    mid = (vals[1:] + vals[:-1]) / 2
    got = O.round_to_e4m3(mid)
    even = np.where(np.arange(len(mid)) % 2 == 0, vals[:-1], vals[1:])
    assert np.array_equal(got, even)
    assert np.array_equal(O.round_to_e4m3(mid * (1 + 1e-9)), vals[1:])
    assert O.round_to_e4m3(1e9) == 448.0
