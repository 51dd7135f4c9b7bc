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
