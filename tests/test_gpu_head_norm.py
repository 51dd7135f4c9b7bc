"""GPU parity of mc_head_norm_rope and its gradient with 64-bit references.

Bounds (w = 2^-24, u = half a step of the stored type, s = |a| + |b| over a pair):
  * rstd: a lane adds at most 8 squares, then at most 5 shuffle sums, all positive, the
    mean's product, eps, root and quotient: 14 w of the mean, half after the root, 3 w
  * z = x rstd w: two more products: 12 w
  * rotation: the turn rounded to fp32 (pi w of the angle), sine and cosine to 2 w, a
    product and an fma: 8 w s; so y within 20 w s of the exact pair, then u.  bf16 takes
    the hardware's sine and cosine: an angle rounded twice more (2 pi w) and 2^-21.1 (8 w)
    absolute, 12 w s more
  * dz = R^T dy: 8 w s (bf16 20 w s); g = w dz and xhat a rounding each; mean(g xhat): 14 w of its
    magnitudes' sum and 10 w of each term; dx: each term to 4 w; u at the end
  * dw: fp32 sums over tokens and heads in some order: (N + 80) w of the magnitudes
"""
import numpy as np
import pytest
import torch

from muon_qk_clip_gb300 import abi, build
from muon_qk_clip_gb300 import binding as mc
from muon_qk_clip_gb300 import synth
from tests.gpu_helpers import assert_rounded_within, f64

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
W = 2.0 ** -24
EPS, THETA = 1e-6, 10000.0


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    abi.load()


def normal(shape, std, key, dtype):
    return synth.normal(shape, std, key, 5).to(dtype).cuda()


def turns(pos, rot, theta=THETA):
    a = np.outer(np.asarray(pos, np.float64), theta ** (-np.arange(0, rot, 2) / max(rot, 1)))
    return np.cos(a)[:, None], np.sin(a)[:, None]


def rotated(x, cos, sin):
    """(rotated x, |a| + |b| of each feature's pair; of the features that are not rotated, |x|)"""
    at = x.shape[-1] - 2 * cos.shape[-1]
    a, b = x[..., at::2], x[..., at + 1::2]
    y, s = x.copy(), np.abs(x)
    y[..., at::2], y[..., at + 1::2] = a * cos - b * sin, a * sin + b * cos
    s[..., at::2] = s[..., at + 1::2] = np.abs(a) + np.abs(b)
    return y, s


def check_forward(x, w, y, rstd, pos, rot, theta=THETA, eps=EPS):
    X = f64(x)
    ref = 1 / np.sqrt(np.mean(X * X, -1) + eps)
    assert np.all(np.abs(f64(rstd) - ref) <= 10 * W * ref)
    z = X * ref[..., None] * (1.0 if w is None else f64(w))
    want, s = rotated(z, *turns(pos, rot, theta))
    assert_rounded_within(y, want, (32 if x.dtype == BF16 else 20) * W * s + 1e-40)


def check_backward(dy, x, rstd, w, dx, dw, pos, rot, theta=THETA):
    X, r = f64(x), f64(rstd)[..., None]
    cos, sin = turns(pos, rot, theta)
    dz, s = rotated(f64(dy), cos, -sin)
    wt = np.ones(X.shape[-1]) if w is None else f64(w)
    xhat, g = X * r, dz * wt
    mean = np.mean(g * xhat, -1, keepdims=True)
    mag = np.mean(np.abs(wt) * s * np.abs(xhat), -1, keepdims=True)
    more = 12 if x.dtype == BF16 else 0
    tol = np.abs(r) * ((14 + more) * W * np.abs(wt) * s + np.abs(xhat) * (30 + more) * W * mag)
    assert_rounded_within(dx, r * (g - xhat * mean), tol + 1e-40)
    if w is None:
        assert dw is None
        return
    n = X.shape[0] * X.shape[1]
    assert np.all(np.abs(f64(dw) - (dz * xhat).sum((0, 1))) <= (n + 80) * W * (s * np.abs(xhat)).sum((0, 1)))


# T, query heads, key heads, d, rot
SHAPES = [(1, 1, 1, 2, 2), (1, 64, 8, 128, 128), (5, 3, 1, 128, 64), (33, 5, 2, 80, 80), (7, 2, 2, 90, 30), (130, 4, 4, 64, 0),
          (3, 9, 1, 256, 256), (2, 3, 5, 192, 64), (6, 7, 3, 254, 100), (1000, 2, 1, 16, 8), (5000, 1, 0, 24, 24), (65, 31, 3, 40, 6)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,H,G,d,rot", SHAPES)
def test_parity(T, H, G, d, rot, dtype):
    q, k = normal((T, H, d), 2.0, "q", dtype), normal((T, G, d), 0.5, "k", dtype) if G else None
    wq, wk = ((1 + normal((d,), 0.2, n, F32)).to(dtype) for n in ("wq", "wk"))
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 37 % 1009
    dyq, dyk = normal((T, H, d), 1e-2, "dq", dtype), normal((T, G, d), 1e-2, "dk", dtype) if G else None
    for weights in (True, False):
        a, b = (wq, wk if G else None) if weights else (None, None)
        for p in (pos, None):
            at = np.arange(T) if p is None else pos.cpu().numpy()
            yq, yk, rstd = mc.qk_norm_rope(q, k, a, b, positions=p, rot=rot, theta=THETA, eps=EPS)
            dq, dk, dwq, dwk = mc.qk_norm_rope_backward(dyq, dyk, q, k, rstd, a, b, positions=p, rot=rot, theta=THETA)
            torch.cuda.synchronize()
            check_forward(q, a, yq, rstd[:, :H], at, rot)
            check_backward(dyq, q, rstd[:, :H], a, dq, dwq, at, rot)
            if G:
                check_forward(k, b, yk, rstd[:, H:], at, rot)
                check_backward(dyk, k, rstd[:, H:], b, dk, dwk, at, rot)
            else:
                assert yk is None and dk is None and dwk is None
            again = mc.qk_norm_rope_backward(dyq, dyk, q, k, rstd, a, b, positions=p, rot=rot, theta=THETA)
            for x, y in zip((dq, dk, dwq, dwk), again):
                assert (x is None) == (y is None) and (x is None or torch.equal(x, y))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shift", [0, 8, 1, 2])
def test_views_of_one_projection_and_in_place(dtype, shift):
    """q and k as head ranges of one buffer, aligned or not, normed in place; the values between
    them stay as they are."""
    T, H, G, d = 19, 6, 2, 64
    buf = torch.full((T, (H + 2 * G) * d + 16), 7.0, dtype=dtype, device="cuda")
    both = buf[:, shift:shift + (H + 2 * G) * d].unflatten(1, (H + 2 * G, d))
    both.copy_(normal((T, H + 2 * G, d), 1.0, "buf", dtype))
    before = buf.clone()
    q, k = both[:, :H], both[:, H:H + G]
    q0, k0 = q.clone(), k.clone()
    w = (1 + normal((d,), 0.2, "w", F32)).to(dtype)
    yq, yk, rstd = mc.qk_norm_rope(q, k, w, w, out_q=q, out_k=k)
    torch.cuda.synchronize()
    assert yq.data_ptr() == q.data_ptr()
    check_forward(q0, w, q, rstd[:, :H], np.arange(T), d)
    check_forward(k0, w, k, rstd[:, H:], np.arange(T), d)
    assert torch.equal(both[:, H + G:], before[:, shift:].narrow(1, (H + G) * d, G * d).unflatten(1, (G, d)))
    assert torch.equal(buf[:, :shift], before[:, :shift]) and torch.equal(buf[:, shift + (H + 2 * G) * d:], before[:, shift + (H + 2 * G) * d:])
    # the gradient, in place over the outputs' gradients in the same kind of buffer
    both.copy_(normal((T, H + 2 * G, d), 1e-2, "gbuf", dtype))
    dyq, dyk = q.clone(), k.clone()
    dq, dk, dwq, dwk = mc.qk_norm_rope_backward(q, k, q0, k0, rstd, w, w, dq=q, dk=k)
    torch.cuda.synchronize()
    check_backward(dyq, q0, rstd[:, :H], w, q, dwq, np.arange(T), d)
    check_backward(dyk, k0, rstd[:, H:], w, k, dwk, np.arange(T), d)


def test_heads_of_transposed_layouts():
    """[H, T, d] storage seen as [T, H, d]: head strides larger than token strides."""
    T, H, G, d = 21, 3, 2, 72
    q, k = normal((H, T, d), 1.0, "tq", BF16).transpose(0, 1), normal((G, T, d), 1.0, "tk", BF16).transpose(0, 1)
    out_q = torch.zeros(H, T, d, dtype=BF16, device="cuda").transpose(0, 1)
    yq, yk, rstd = mc.qk_norm_rope(q, k, out_q=out_q, rot=48)
    torch.cuda.synchronize()
    check_forward(q, None, out_q, rstd[:, :H], np.arange(T), 48)
    check_forward(k, None, yk, rstd[:, H:], np.arange(T), 48)


def test_far_and_negative_positions():
    """Any 32-bit position: the turn is taken modulo one in integers, so far positions are as good
    as near ones (frequencies in fp64: 2^31 positions of at most a radian to 2^-21)."""
    pos = torch.tensor([0, 1, -1, 1 << 20, (1 << 24) + 1, 2147483647, -2147483648], dtype=torch.int32, device="cuda")
    x = normal((7, 2, 32), 1.0, "far", F32)
    y, _, rstd = mc.qk_norm_rope(x, positions=pos, rot=32)
    torch.cuda.synchronize()
    P = pos.cpu().numpy().astype(np.float64)
    X = f64(x)
    z = X / np.sqrt(np.mean(X * X, -1, keepdims=True) + EPS)
    want, s = rotated(z, *turns(P, 32))
    # the frequencies' 2^-52 relative, here and in the reference, times the angle
    tol = (20 * W + np.abs(P)[:, None, None] * 2.0 ** -51) * s
    assert np.all(np.abs(f64(y) - want) <= tol + W * np.abs(want))


def test_theta_below_one():
    x = normal((9, 1, 16), 1.0, "low", F32)
    y, _, rstd = mc.qk_norm_rope(x, theta=0.25)
    torch.cuda.synchronize()
    check_forward(x, None, y, rstd, np.arange(9), 16, theta=0.25)


def test_zero_and_nonfinite_heads():
    """A head of zeros gives zeros (eps alone under the root); NaN and infinity stay in their head."""
    q = normal((4, 3, 64), 1.0, "nf", BF16)
    clean, _, r0 = mc.qk_norm_rope(q)
    bad = q.clone()
    bad[1, 1, 5], bad[2, 0, 7] = float("nan"), float("inf")
    bad[3, 2] = 0
    y, _, rstd = mc.qk_norm_rope(bad)
    torch.cuda.synchronize()
    keep = torch.ones(4, 3, dtype=torch.bool, device="cuda")
    keep[1, 1] = keep[2, 0] = keep[3, 2] = False
    assert torch.equal(y[keep], clean[keep]) and torch.equal(rstd[keep], r0[keep])
    assert torch.all(y[3, 2] == 0) and torch.isnan(y[1, 1]).all() and torch.isnan(y[2, 0]).any()


def test_no_tokens():
    q = torch.empty(0, 2, 64, dtype=BF16, device="cuda")
    w = torch.ones(64, dtype=BF16, device="cuda")
    y, _, rstd = mc.qk_norm_rope(q, wq=w)
    dq, _, dw, _ = mc.qk_norm_rope_backward(q, None, q, None, rstd, wq=w, dwq=torch.full((64,), 7.0, device="cuda"))
    torch.cuda.synchronize()
    assert y.shape == q.shape and dq.shape == q.shape and torch.all(dw == 0)


def test_gradient_against_differences():
    """sum(dy * y) as a function of x and w, differentiated numerically in 64 bits by the oracle
    formula, agrees with the kernel's gradient."""
    T, H, d, rot = 2, 2, 10, 6
    x, w, dy = normal((T, H, d), 1.0, "fx", F32), 1 + normal((d,), 0.2, "fw", F32), normal((T, H, d), 1.0, "fd", F32)
    _, _, rstd = mc.qk_norm_rope(x, wq=w, rot=rot)
    dx, _, dw, _ = mc.qk_norm_rope_backward(dy, None, x, None, rstd, wq=w, rot=rot)
    torch.cuda.synchronize()

    def f(X, Wt):
        z = X / np.sqrt(np.mean(X * X, -1, keepdims=True) + EPS) * Wt
        return float((rotated(z, *turns(np.arange(T), rot))[0] * f64(dy)).sum())

    X, Wt, h = f64(x), f64(w), 1e-5
    for i in np.ndindex(X.shape):
        e = np.zeros_like(X)
        e[i] = h
        # central differences: h^2 times third derivatives of order 10, 2^-52 / h of the sum
        assert abs((f(X + e, Wt) - f(X - e, Wt)) / (2 * h) - f64(dx)[i]) < 1e-5
    for i in range(d):
        e = np.zeros(d)
        e[i] = h
        assert abs((f(X, Wt + e) - f(X, Wt - e)) / (2 * h) - f64(dw)[i]) < 1e-5


def test_offsets_past_32_bits():
    """Token strides that reach beyond 2^31 elements."""
    base = torch.zeros((1 << 31) + 4096, dtype=BF16, device="cuda")
    x = base.as_strided((2, 2, 128), (1 << 31, 128, 1))
    x.copy_(normal((2, 2, 128), 1.0, "big", BF16))
    y, _, rstd = mc.qk_norm_rope(x)
    dx, _, _, _ = mc.qk_norm_rope_backward(x, None, x, None, rstd)
    torch.cuda.synchronize()
    check_forward(x, None, y, rstd, np.arange(2), 128)
    check_backward(x, x, rstd, None, dx, None, np.arange(2), 128)


def test_streams_and_graph():
    q, k = normal((300, 8, 128), 1.0, "gq", BF16), normal((300, 2, 128), 1.0, "gk", BF16)
    w = (1 + normal((128,), 0.2, "gw", F32)).to(BF16)
    want = mc.qk_norm_rope(q, k, w, w)
    grad = mc.qk_norm_rope_backward(*want[:2], q, k, want[2], w, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mc.qk_norm_rope(q, k, w, w, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = mc.qk_norm_rope(q, k, w, w)
        g = mc.qk_norm_rope_backward(*y[:2], q, k, y[2], w, w)
    for t in (*y, *g):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*want, *grad), (*y, *g)))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_without_keys_their_pointers_are_not_looked_at(dtype):
    """heads_k of 0 at the C ABI: k, wk, yk, dyk, dk and dwk may be anything, here an odd address of
    nothing; the results are those of null pointers."""
    T, H, d = 40, 3, 64
    q, dy = normal((T, H, d), 1.0, "nk", dtype), normal((T, H, d), 1e-2, "nkd", dtype)
    w = (1 + normal((d,), 0.2, "nkw", F32)).to(dtype)
    want = mc.qk_norm_rope(q, None, w)
    grad = mc.qk_norm_rope_backward(dy, None, q, None, want[2], w)
    lib, stale = abi.load(), 0x7f0000000001
    h = abi.McHeads(T, H, 0, d, d, abi.MC_BF16 if dtype == BF16 else abi.MC_F32, EPS, THETA, None)
    y, dx, rstd = torch.empty_like(q), torch.empty_like(q), torch.empty(T, H, device="cuda")
    dw, ws = torch.empty(d, device="cuda"), torch.empty(mc.head_norm_backward_workspace_size(d), dtype=torch.uint8, device="cuda")
    at = lambda t: (t.data_ptr(), H * d, d)  # noqa: E731
    none, s = (stale, 1, 1), torch.cuda.current_stream().cuda_stream
    assert lib.mc_head_norm_rope(h, *at(q), *none, w.data_ptr(), stale, *at(y), *none, rstd.data_ptr(), s) == abi.MC_OK
    assert lib.mc_head_norm_rope_backward(h, *at(dy), *none, *at(q), *none, rstd.data_ptr(), w.data_ptr(), stale, *at(dx), *none,
                                          dw.data_ptr(), stale, ws.data_ptr(), ws.numel(), s) == abi.MC_OK
    torch.cuda.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(rstd, want[2]) and torch.equal(dx, grad[0]) and torch.equal(dw, grad[2])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,H,G,d,rot", [(1, 1, 1, 2, 2), (33, 5, 2, 80, 80), (7, 2, 2, 90, 30), (130, 4, 0, 64, 0), (300, 9, 1, 256, 128)])
def test_without_the_norm(T, H, G, d, rot, dtype):
    """Rotation and weights alone: y = R (x w), dx = w R^T dy, dw = sum R^T dy x; bounds as with the
    norm, which takes more roundings.  Infinite features reach their own rows of y and dw, no dx."""
    q, k = normal((T, H, d), 2.0, "q", dtype), normal((T, G, d), 0.5, "k", dtype) if G else None
    wq, wk = ((1 + normal((d,), 0.2, n, F32)).to(dtype) for n in ("wq", "wk"))
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 37 % 1009
    dyq, dyk = normal((T, H, d), 1e-2, "dq", dtype), normal((T, G, d), 1e-2, "dk", dtype) if G else None
    cos, sin = turns(pos.cpu().numpy(), rot)
    more = (32 if dtype == BF16 else 20) * W
    for weights in (True, False):
        a, b = (wq, wk if G else None) if weights else (None, None)
        yq, yk, rstd = mc.qk_norm_rope(q, k, a, b, positions=pos, rot=rot, norm=False)
        grads = mc.qk_norm_rope_backward(dyq, dyk, q, k, None, a, b, positions=pos, rot=rot, norm=False)
        torch.cuda.synchronize()
        assert rstd is None
        for x, w, y, dy, dx, dw in ((q, a, yq, dyq, grads[0], grads[2]), (k, b, yk, dyk, grads[1], grads[3])):
            if x is None:
                continue
            wt = np.ones(d) if w is None else f64(w)
            want, s = rotated(f64(x) * wt, cos, sin)
            assert_rounded_within(y, want, more * s + 1e-40)
            dz, s = rotated(f64(dy), cos, -sin)
            assert_rounded_within(dx, dz * wt, more * s * np.abs(wt) + 1e-40)
            if w is not None:
                n = x.shape[0] * x.shape[1]
                assert np.all(np.abs(f64(dw) - (dz * f64(x)).sum((0, 1))) <= (n + 80) * W * (s * np.abs(f64(x))).sum((0, 1)))
    clean = mc.qk_norm_rope_backward(dyq, None, q, None, None, rot=rot, norm=False)
    q[0, 0] = float("inf")
    bad = mc.qk_norm_rope_backward(dyq, None, q, None, None, rot=rot, norm=False)
    assert torch.equal(clean[0], bad[0])
    with pytest.raises(ValueError, match="rstd"):
        mc.qk_norm_rope_backward(dyq, None, q, None, None, rot=rot)
    with pytest.raises(ValueError, match="rstd"):
        mc.qk_norm_rope(q, rstd=torch.empty(T, H, device="cuda"), norm=False)
