"""GPU parity of mc_add_rms_norm, mc_rms_norm_backward and mc_rope_backward with
64-bit references.

Bounds (w = 2^-24, u = half a step of the stored type relative: 2^-24 fp32,
2^-8 bf16):
  * h is the rounding of the fp32 sum: equal bits
  * rstd: a lane adds at most L = max(32, cols / 256) squares, then 5 shuffle
    and 8 warp sums, all positive: relative (L + 13) w for the mean square, half
    of it after the root, and 4 w for division, root and reciprocal
  * y: rstd's, 2 w for the products, u
  * e4m3: the scale within twice y's fp32 error, 2 w; q a rounding of a value
    within that of y / scale (rounding is monotone)
  * dx: with xhat and g correct to 2 w, mean(g xhat) to (L + 16) w of the mean
    of magnitudes, each of the three terms to 4 w of itself; u at the end
  * dw: fp32 sums over the rows in some order: (rows + 60) w of the magnitudes
  * rotary gradient: angles within half a turn rounded to fp32 (pi w), sines to
    2 ulp, one product and one fma: 8 w (|a| + |b|), u of the result
"""
import ctypes

import numpy as np
import pytest
import torch

import oracle as O
from muon_qk_clip_gb300 import abi, build
from muon_qk_clip_gb300 import binding as mc
from muon_qk_clip_gb300 import synth
from tests.gpu_helpers import f64

pytestmark = pytest.mark.gpu
BF16, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
W = 2.0 ** -24
U = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    abi.load()


def normal(shape, std, key, dtype):
    return synth.normal(shape, std, key, 7).to(dtype).cuda()


def pitched(t, extra, shift=0):
    """t as a column slice of a wider buffer of sevens."""
    base = torch.full((t.shape[0], t.shape[1] + extra), 7, dtype=t.dtype, device="cuda")
    view = base[:, shift:shift + t.shape[1]]
    view.copy_(t)
    return base, view


def chain(cols):
    return max(32, cols / 256)


def check_add(x, r, w, y, scales, h, rstd, eps=EPS):
    cols = x.shape[1]
    want = x if r is None else (x.float() + r.float()).to(x.dtype)
    assert torch.equal(h, want)
    H = f64(want)
    ref = 1 / np.sqrt(np.mean(H * H, 1) + eps)
    e = ((chain(cols) + 13) / 2 + 4) * W
    assert np.all(np.abs(f64(rstd) - ref) <= e * ref)
    Y = H * ref[:, None] * (1.0 if w is None else f64(w))
    e += 2 * W
    if scales is None:
        assert np.all(np.abs(f64(y) - Y) <= (e + U[y.dtype]) * np.abs(Y) + 1e-40)
        return
    assert scales.shape == (x.shape[0], -(-cols // 128))
    q, s = y.float().double().cpu().numpy(), f64(scales)
    for t in range(s.shape[1]):
        part = Y[:, 128 * t:128 * t + 128]
        sref = np.maximum(np.abs(part).max(1) / 448.0, 2.0 ** -100)
        assert np.all(np.abs(s[:, t] - sref) <= (e + 2 * W) * sref)
        z = part / sref[:, None]
        tol = (2 * e + 4 * W) * np.abs(z)
        got = q[:, 128 * t:128 * t + 128]
        assert np.all(got >= O.round_to_e4m3(z - tol)) and np.all(got <= O.round_to_e4m3(z + tol))


SHAPES = [(1, 1), (1, 7168), (3, 128), (5, 129), (7, 127), (64, 512), (33, 1536), (9, 1537), (4, 2048), (130, 96),
          (2, 8192), (3, 8200), (2, 12001), (1000, 24)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_add_rms_norm_parity(rows, cols, dtype):
    x, r = normal((rows, cols), 1.0, "nx", dtype), normal((rows, cols), 3.0, "nr", dtype)
    w = (1 + normal((cols,), 0.2, "nw", F32)).to(dtype)
    for res, wt, out in ((r, w, F8), (r, None, None), (None, w, None), (None, None, F8)):
        y, s, h, rstd = mc.add_rms_norm(x, res, wt, eps=EPS, out_dtype=out)
        torch.cuda.synchronize()
        check_add(x, res, wt, y, s, h, rstd)
        again = mc.add_rms_norm(x, res, wt, eps=EPS, out_dtype=out)
        assert torch.equal(again[0].view(torch.uint8), y.view(torch.uint8)) and torch.equal(again[3], rstd)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shift,extra", [(0, 16), (8, 24), (3, 5)])
def test_add_rms_norm_pitches_and_in_place(dtype, shift, extra):
    """Column slices of wider buffers, 16-byte aligned or not; h over the
    residual and y over x; nothing beside the slices is written."""
    rows, cols = 37, 640
    x, r = normal((rows, cols), 1.0, "px", dtype), normal((rows, cols), 2.0, "pr", dtype)
    w = (1 + normal((cols,), 0.2, "pw", F32)).to(dtype)
    bx, vx = pitched(x, extra, shift)
    br, vr = pitched(r, extra, shift)
    bs = torch.full((rows, 9), 7.0, device="cuda")
    y, s, h, rstd = mc.add_rms_norm(vx, vr, w, eps=EPS, out_dtype=F8, h=vr, scales=bs[:, 2:7])
    torch.cuda.synchronize()
    check_add(x, r, w, y, s, vr, rstd)
    assert torch.all(bs[:, :2] == 7) and torch.all(bs[:, 7:] == 7) and torch.equal(vx, x)
    br, vr = pitched(r, extra, shift)
    y, _, h, rstd = mc.add_rms_norm(vx, vr, w, eps=EPS, h=vr, out=vx)
    torch.cuda.synchronize()
    check_add(x, r, w, vx, None, vr, rstd)
    for base in (bx, br):
        assert torch.all(base[:, :shift] == 7) and torch.all(base[:, shift + cols:] == 7)


def test_add_rms_norm_agrees_with_rms_norm():
    """Without residual and weight it is rms_norm (another order of the sum)."""
    x = normal((50, 1536), 2.0, "ag", F32)
    y = mc.add_rms_norm(x, eps=EPS)[0]
    assert torch.allclose(y, mc.rms_norm(x, eps=EPS), rtol=1e-5, atol=0)


def test_add_rms_norm_extreme_rows():
    """Zero rows, rows of tiny and of huge values, and a NaN and an infinity that
    stay in their own rows."""
    x = normal((8, 384), 1.0, "ex", F32)
    x[0] = 0
    x[1] *= 1e-30
    x[2] *= 1e15
    x[3, 5] = float("nan")
    x[4, 7] = float("inf")
    x[5, :128] = 0
    y, s, _, rstd = mc.add_rms_norm(x, eps=EPS, out_dtype=F8)
    torch.cuda.synchronize()
    good = [0, 1, 2, 5, 6, 7]
    check_add(x[good], None, None, y[good], s[good], x[good], rstd[good])
    assert torch.all(s[0] == 2.0 ** -100) and torch.all(y[0].float() == 0) and s[5, 0] == 2.0 ** -100
    assert torch.isnan(y[3].float()).all() and torch.isnan(s[3]).all()
    assert rstd[4] == 0 and torch.isnan(y[4, 7].float())


def test_add_rms_norm_single_tokens_match_the_batch():
    x, r = normal((6, 7168), 1.0, "st", BF16), normal((6, 7168), 2.0, "sr", BF16)
    y, s, h, rstd = mc.add_rms_norm(x, r, eps=EPS, out_dtype=F8)
    for i in range(6):
        yi, si, hi, ri = mc.add_rms_norm(x[i:i + 1], r[i:i + 1], eps=EPS, out_dtype=F8)
        assert torch.equal(yi.view(torch.uint8), y[i:i + 1].view(torch.uint8)) and torch.equal(si, s[i:i + 1])
        assert torch.equal(hi, h[i:i + 1]) and torch.equal(ri, rstd[i:i + 1])


def check_back(dy, h, rstd, w, dres, dx, dw):
    rows, cols = dy.shape
    D, Hh, rs = f64(dy), f64(h), f64(rstd)[:, None]
    wt = 1.0 if w is None else f64(w)
    ref, dwref = O.rms_norm_backward(D, Hh, rs[:, 0], wt if w is not None else None, None if dres is None else f64(dres))
    xh, g = np.abs(Hh * rs), np.abs(D * wt)
    m = np.mean(g * xh, 1, keepdims=True)
    d = np.zeros_like(ref) if dres is None else np.abs(f64(dres))
    tol = rs * (4 * W * g + xh * m * (chain(cols) + 16 + 8) * W) + 4 * W * d + U[dy.dtype] * np.abs(ref) + 1e-38
    err = np.abs(f64(dx) - ref)
    assert np.all(err <= tol), (np.max(err - tol), np.max(err))
    if dw is not None:
        assert np.all(np.abs(f64(dw) - dwref) <= (rows + 60) * W * np.sum(np.abs(D) * xh, 0) + 1e-38)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", SHAPES + [(2500, 256), (700, 2048), (613, 40)])
def test_rms_norm_backward_parity(rows, cols, dtype):
    h, dy = normal((rows, cols), 3.0, "bh", dtype), normal((rows, cols), 0.01, "bd", dtype)
    dres = normal((rows, cols), 0.01, "br", dtype)
    w = (1 + normal((cols,), 0.2, "bw", F32)).to(dtype)
    rstd = torch.rsqrt(h.float().square().mean(1) + EPS)
    for wt, res in ((w, dres), (None, None), (w, None)):
        dx, dw = mc.rms_norm_backward(dy, h, rstd, weight=wt, dres=res)
        torch.cuda.synchronize()
        assert (dw is None) == (wt is None)
        check_back(dy, h, rstd, wt, res, dx, dw)
        again = mc.rms_norm_backward(dy, h, rstd, weight=wt, dres=res)
        assert torch.equal(again[0], dx) and (dw is None or torch.equal(again[1], dw))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shift,extra", [(0, 16), (3, 5)])
@pytest.mark.parametrize("over", ["dy", "h", "dres", "none"])
def test_rms_norm_backward_in_place_and_pitched(dtype, shift, extra, over):
    rows, cols = 45, 640
    t = {"h": normal((rows, cols), 3.0, "ih", dtype), "dy": normal((rows, cols), 0.01, "id", dtype),
         "dres": normal((rows, cols), 0.01, "ir", dtype), "none": torch.zeros(rows, cols, dtype=dtype, device="cuda")}
    w = (1 + normal((cols,), 0.2, "iw", F32)).to(dtype)
    rstd = torch.rsqrt(t["h"].float().square().mean(1) + EPS)
    wide = {n: pitched(x, extra, shift) for n, x in t.items()}
    ws = torch.full((304 * cols,), float("nan"), device="cuda")
    dx, dw = mc.rms_norm_backward(wide["dy"][1], wide["h"][1], rstd, weight=w, dres=wide["dres"][1], dx=wide[over][1],
                                  workspace=ws)
    torch.cuda.synchronize()
    check_back(t["dy"], t["h"], rstd, w, t["dres"], dx, dw)
    base = wide[over][0]
    assert torch.all(base[:, :shift] == 7) and torch.all(base[:, shift + cols:] == 7)
    alone = mc.rms_norm_backward(t["dy"], t["h"], rstd, dweight=torch.empty(cols, device="cuda"))
    check_back(t["dy"], t["h"], rstd, None, None, *alone)          # a weight gradient of ones


def test_rms_norm_backward_of_no_rows():
    e = torch.empty(0, 64, device="cuda")
    dx, dw = mc.rms_norm_backward(e, e, torch.empty(0, device="cuda"), weight=torch.ones(64, device="cuda"))
    torch.cuda.synchronize()
    assert dx.shape == (0, 64) and torch.all(dw == 0)
    y, s, h, rstd = mc.add_rms_norm(e, e, out_dtype=F8)
    assert y.shape == (0, 64) and rstd.shape == (0,)


def check_rope(dy, out, theta):
    ref = O.rope_backward(f64(dy), theta)
    x = f64(dy)
    pair = np.repeat(np.abs(x[..., 0::2]) + np.abs(x[..., 1::2]), 2, axis=-1)
    assert np.all(np.abs(f64(out) - ref) <= 8 * W * pair + U[dy.dtype] * np.abs(ref) + 1e-40)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,S,nh,d,skip,theta", [
    (1, 1, 1, 2, 0, 10000.0), (2, 700, 3, 64, 128, 10000.0), (1, 5000, 1, 64, 0, 10000.0), (3, 17, 5, 6, 1, 500.0),
    (1, 33, 2, 4096, 0, 1e6), (2, 9, 70, 30, 2, 10000.0), (1, 40000, 1, 16, 0, 10000.0),
    (1, 1 << 20, 1, 4, 0, 0.25), (1, 200, 3, 8, 0, 1e-4)])
def test_rope_backward_parity(B, S, nh, d, skip, theta, dtype):
    """Out of place and in place, on the rotary columns of wider heads, at
    positions up to 2^20 and angles up to 2^22; aligned and unaligned slices."""
    full = normal((B, S, nh, skip + d), 0.5, "rd", dtype)
    keep = full.clone()
    dy = full[..., skip:]
    out = mc.rope_backward(dy, theta)
    torch.cuda.synchronize()
    assert torch.equal(full, keep)
    check_rope(dy, out, theta)
    assert mc.rope_backward(dy, theta, out=dy) is dy
    torch.cuda.synchronize()
    assert torch.equal(dy, out) and torch.equal(full[..., :skip], keep[..., :skip])


def test_rope_backward_undoes_rope():
    """rope_ then rope_backward returns the features, to the two roundings; the
    shared key's three-axis form."""
    x = normal((2, 300, 64), 1.0, "ru", F32)
    y = mc.rope_backward(mc.rope_(x.clone()))
    assert torch.allclose(x, y, atol=4e-6)


def test_norm_and_rope_calls_in_a_cuda_graph_and_on_a_stream():
    x, r = normal((96, 640), 1.0, "gx", BF16), normal((96, 640), 2.0, "gr", BF16)
    w = (1 + normal((640,), 0.2, "gw", F32)).to(BF16)
    dy = normal((96, 640), 0.01, "gd", BF16)
    ws = torch.empty(304 * 640, device="cuda")
    o = dict(h=torch.empty_like(x), out=torch.empty(96, 640, dtype=F8, device="cuda"),
             scales=torch.empty(96, 5, device="cuda"), rstd=torch.empty(96, device="cuda"))
    dx, dw = torch.empty_like(x), torch.empty(640, device="cuda")
    rx = torch.empty(1, 96, 10, 64, dtype=BF16, device="cuda")

    def calls(stream=None):
        mc.add_rms_norm(x, r, w, out_dtype=F8, stream=stream, **o)
        mc.rms_norm_backward(dy, o["h"], o["rstd"], weight=w, dres=dy, dx=dx, dweight=dw, workspace=ws, stream=stream)
        mc.rope_backward(dx.view(1, 96, 10, 64), out=rx, stream=stream)

    graph = torch.cuda.CUDAGraph()
    calls()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        calls()
    x.add_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (o["out"].view(torch.uint8), o["scales"], o["h"], dx, dw, rx)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    calls(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, (o["out"].view(torch.uint8), o["scales"], o["h"], dx, dw, rx)))


def test_norm_gradient_on_another_stream_keeps_its_memory():
    """As for the attention's gradient: the partial weight sums of a call on a
    given stream are not handed out while it runs."""
    dy, h = normal((96, 640), 0.01, "gd", BF16), normal((96, 640), 1.0, "gx", BF16)
    w = (1 + normal((640,), 0.2, "gw", F32)).to(BF16)
    rstd = mc.add_rms_norm(h)[3]
    want = mc.rms_norm_backward(dy, h, rstd, weight=w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)      # about 10 ms
    got = mc.rms_norm_backward(dy, h, rstd, weight=w, stream=side)
    taken = [torch.full((mc.rms_norm_backward_workspace_size(640) // 4,), float("nan"), device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert len(taken) == 4 and all(torch.equal(a, b) for a, b in zip(want, got))
    with pytest.raises(ValueError, match="contiguous"):
        mc.rms_norm_backward(dy, h, rstd, weight=w, workspace=torch.empty(1, device="cuda").expand(304 * 640))


def test_calls_wait_for_what_their_inputs_come_from():
    """The kernels may be scheduled before the work in front of them has ended, and
    wait for it: behind a long kernel, a copy, a fill, another stream's work and
    each other, eagerly and captured, they see its results."""
    src, w = normal((3000, 1024), 1.0, "dx", BF16), (1 + normal((1024,), 0.2, "dw", F32)).to(BF16)
    host = src.cpu().pin_memory()
    x, r, dy = torch.empty_like(src), torch.empty_like(src), torch.empty_like(src)
    side = torch.cuda.Stream()
    big = torch.empty(64 << 20, device="cuda")

    def chain(seed):
        big.fill_(seed)                                    # a kernel that outlasts the launches behind it
        x.copy_(src)
        y, _, h, rstd = mc.add_rms_norm(x, weight=w)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            big.fill_(seed + 1)
            dy.copy_(y)
        torch.cuda.current_stream().wait_stream(side)
        dx, dw = mc.rms_norm_backward(dy, h, rstd, weight=w)
        r.zero_()
        r.add_(dx)
        y2, s2, h2, _ = mc.add_rms_norm(y, r, w, out_dtype=F8)
        out = mc.rope_backward(h2.view(1, 3000, 16, 64))
        big.fill_(seed + 2)
        x.copy_(host, non_blocking=True)
        z = mc.add_rms_norm(x, out.view(3000, 1024), w)[0]
        return dx, dw, y2.view(torch.uint8), s2, out, z

    torch.cuda.synchronize()
    steps = []
    real = mc._run

    def one_by_one(*a):
        torch.cuda.synchronize()
        real(*a)
        torch.cuda.synchronize()
    mc._run = one_by_one
    try:
        want = [t.clone() for t in chain(1.0)]
    finally:
        mc._run = real
    for _ in range(3):
        steps.append(chain(2.0))
    torch.cuda.synchronize()
    for got in steps:
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(3.0)
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_norm_and_rope_offsets_past_32_bits():
    """Rows and positions so far apart that element offsets pass 2^31."""
    rows, cols, ld = 3, 384, (1 << 31) + 8
    far = torch.empty((rows - 1) * ld + 4 * cols, dtype=BF16, device="cuda")
    x, r, dy = (normal((rows, cols), 1.0, n, BF16) for n in ("fx", "fr", "fd"))
    w = (1 + normal((cols,), 0.2, "fw", F32)).to(BF16)
    place = [far.as_strided((rows, cols), (ld, 1), i * cols) for i in range(4)]
    y, _, h, rstd = mc.add_rms_norm(x, r, w)
    dx, dw = mc.rms_norm_backward(dy, h, rstd, weight=w)
    place[0].copy_(x)
    place[1].copy_(r)
    y2, _, h2, rstd2 = mc.add_rms_norm(place[0], place[1], w, h=place[2], out=place[3])
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(h, h2) and torch.equal(rstd, rstd2)
    place[0].copy_(dy)
    dx2, dw2 = mc.rms_norm_backward(place[0], h2, rstd, weight=w, dx=place[1])
    torch.cuda.synchronize()
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    want = mc.rope_backward(dy.view(1, rows, 3, 128))
    got = mc.rope_backward(place[0].as_strided((1, rows, 3, 128), (0, ld, 128, 1), 0),
                           out=torch.empty_like(far).as_strided((1, rows, 3, 128), (0, ld, 128, 1), 0))
    torch.cuda.synchronize()
    assert torch.equal(want, got)


@pytest.mark.parametrize("shift,extra", [(0, 24), (3, 5)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_add_rms_norm_e4m3_is_the_rounded_quotient(dtype, shift, extra):
    """Rows of +-1 with eps = 0 have rstd = 1, so y is +-w exactly: the scale has the
    bits of the fp32 quotient max|w| / 448 and the codes those of e4m3(w / scale),
    on weights next to the values where e4m3 changes its code."""
    tiles, cols = 41, 40 * 128 + 40
    g = np.random.default_rng(5)
    top = g.integers(128, 256, tiles) * 2.0 ** g.integers(-110, 3, tiles)
    tie = (2 * g.integers(8, 16, (tiles, 128)) + 1) * 2.0 ** g.integers(-11, 4, (tiles, 128))
    w = np.minimum(tie / 448, 1.0) * top[:, None]
    w[:, 5] = top
    w[7] = 0
    w = torch.from_numpy(w.reshape(-1)[:cols]).to(dtype).cuda()
    x = torch.where(torch.rand(3, cols, device="cuda") < 0.5, -1.0, 1.0).to(dtype)
    _, vx = pitched(x, extra, shift)
    y, s, _, rstd = mc.add_rms_norm(vx, weight=w, eps=0.0, out_dtype=F8)
    torch.cuda.synchronize()
    assert torch.all(rstd == 1)
    v = np.zeros(tiles * 128, np.float32)
    v[:cols] = w.float().cpu().numpy()
    v = v.reshape(tiles, 128)
    scale = np.maximum(np.abs(v).max(1) / np.float32(448), np.float32(2.0 ** -100))
    code = O.round_to_e4m3((v / scale[:, None]).astype(np.float64)).reshape(-1)[:cols]
    assert scale.dtype == np.float32 and np.array_equal(s.cpu().numpy(), np.broadcast_to(scale, (3, tiles)))
    assert np.array_equal(y.float().double().cpu().numpy(), f64(x) * code)


def test_an_older_error_of_the_runtime_is_not_the_calls_own():
    """A runtime call of the program's own has failed and left its error to be
    fetched: a launch that succeeds says so, and leaves that error where it was."""
    cudart = ctypes.CDLL("libcudart.so.13")
    x, dy = normal((5, 640), 1.0, "er", F32), normal((5, 640), 0.1, "ed", F32)
    y, _, _, rstd = mc.add_rms_norm(x)
    dx = mc.rms_norm_backward(dy, x, rstd)[0]
    out, r2, dx2, rx = torch.empty_like(x), torch.empty_like(rstd), torch.empty_like(x), torch.empty_like(x)
    torch.cuda.synchronize()
    assert cudart.cudaSetDevice(1 << 20) != 0
    try:
        pending = cudart.cudaPeekAtLastError()
        mc.add_rms_norm(x, out=out, rstd=r2)
        mc.rms_norm_backward(dy, x, rstd, dx=dx2)
        mc.rope_backward(dy.view(1, 5, 10, 64), out=rx.view(1, 5, 10, 64))
        assert pending != 0 and cudart.cudaPeekAtLastError() == pending
    finally:
        cudart.cudaGetLastError()
    torch.cuda.synchronize()
    assert torch.equal(out, y) and torch.equal(r2, rstd) and torch.equal(dx2, dx)
    assert torch.equal(rx.view(1, 5, 10, 64), mc.rope_backward(dy.view(1, 5, 10, 64)))


@pytest.mark.parametrize("rows,cols,dtype", [(700, 7168, BF16), (613, 8200, BF16), (650, 7167, BF16), (613, 2100, F32),
                                             (700, 7168, F32)])
def test_rms_norm_backward_of_wide_rows_over_many_rows(rows, cols, dtype):
    """Rows wider than a block's registers hold, several to every block: the
    weight's sums are carried from row to row."""
    h, dy = normal((rows, cols), 3.0, "wh", dtype), normal((rows, cols), 0.01, "wd", dtype)
    dres = normal((rows, cols), 0.01, "wr", dtype)
    w = (1 + normal((cols,), 0.2, "ww", F32)).to(dtype)
    rstd = torch.rsqrt(h.float().square().mean(1) + EPS)
    dx, dw = mc.rms_norm_backward(dy, h, rstd, weight=w, dres=dres)
    torch.cuda.synchronize()
    check_back(dy, h, rstd, w, dres, dx, dw)
    again = mc.rms_norm_backward(dy, h, rstd, weight=w, dres=dres, dx=dres)      # in place
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
