"""GPU parity of mc_adamw_step with a 64-bit reference.

Bounds (w = 2^-24; A = |beta1 m| + |(1 - beta1) g|, the magnitudes of the new m):
  * m: both factors rounded once, a product, the sum, and before them grad_scale's
    product and an 8-bit state's code * scale: 6 w A
  * v: as many roundings, the gradient's twice, the stored root's twice, all terms
    positive: 10 w v
  * the update u = m i1 / (sqrt(v) i2 + eps): m's, half of v's, a rounding each for
    the root, i1, i2 and the fma, and 2 ulp (4 w) for the quotient:
    (8 w A i1 + 16 w |m| i1) / denominator
  * p: lr (u's + 4 w (|u| + decay |p|)), then one rounding to its type
  * 8-bit states: the scale within the largest value's relative error and 2 w; the
    code a rounding of a value within that and 4 w of x / scale (rounding is monotone)
"""
import numpy as np
import pytest
import torch

import oracle as O
from muon_qk_clip_gb300 import abi, build
from muon_qk_clip_gb300 import binding as mc
from muon_qk_clip_gb300 import synth
from tests.gpu_helpers import assert_rounded_within, f64

pytestmark = pytest.mark.gpu
BF16, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
W = 2.0 ** -24
LEAST, SCALE_MIN = 2.0 ** -9, 2.0 ** -100


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    abi.load()


def normal(shape, std, key):
    return synth.normal(shape, std, key, 11)


def copy_of(state):
    return {k: v and [t.clone() for t in v] for k, v in state.items()}


def make(sizes, p_dtype, g_dtype, bits, steps_before=3):
    """Parameters, gradients and a state that has seen a few steps; some gradients are exactly zero."""
    P = [normal((n,), 0.02, f"p{i}").to(p_dtype).cuda() for i, n in enumerate(sizes)]
    G = [(normal((n,), 1e-3, f"g{i}") * torch.exp(normal((n,), 1.0, f"l{i}"))).to(g_dtype).cuda() for i, n in enumerate(sizes)]
    for g in G:
        g[::7] = 0.0
    s = mc.adamw_state(P, bits)
    for t in range(steps_before):
        mc.adamw_step([p.clone() for p in P], [g * (1.0 - 0.3 * t) for g in G], hp=mc.AdamHparams(), step=t + 1, **s)
    return P, G, s


def values(code, scale):
    """The values that codes stand for, in 64 bits."""
    n = code.numel()
    return code.float().double().cpu().numpy().ravel() * np.repeat(f64(scale), 128)[:n]


def reference(p, g, m, r_or_v, hp, step, bits, gs=1.0):
    """(p, m, v and the bounds of p and m) of one tensor, from 64-bit copies of what the state holds."""
    p, g = f64(p).ravel(), f64(g).ravel() * gs
    v = r_or_v ** 2 if bits == 8 else r_or_v
    A = np.abs(hp.beta1 * m) + np.abs((1 - hp.beta1) * g)
    m = hp.beta1 * m + (1 - hp.beta1) * g
    v = hp.beta2 * v + (1 - hp.beta2) * g * g
    i1 = 1 / (1 - hp.beta1 ** step)
    den = np.sqrt(v / (1 - hp.beta2 ** step)) + hp.eps
    u = m * i1 / den
    tu = (8 * W * A * i1 + 16 * W * np.abs(m) * i1) / den
    tp = abs(hp.lr) * (tu + 4 * W * (np.abs(u) + hp.weight_decay * np.abs(p)))
    return p - hp.lr * (u + hp.weight_decay * p), m, v, tp, 6 * W * A


def check_codes(code, scale, x, tol, root):
    n = x.size
    pad = lambda t: np.pad(t, (0, -n % 128)).reshape(-1, 128)  # noqa: E731
    X, T = pad(x), pad(tol)
    top = np.abs(X).max(1)
    ref = np.maximum(top / 448.0, SCALE_MIN)
    ts = T.max(1) / 448.0 + 2 * W * ref
    s = f64(scale)
    assert np.all(np.abs(s - ref) <= ts)
    y = X / ref[:, None]
    ty = T / ref[:, None] + np.abs(y) * ((ts / ref)[:, None] + 4 * W)
    lo, hi = O.round_to_e4m3(y - ty), O.round_to_e4m3(y + ty)
    if root:                              # a root that is not zero has at least the least code
        some = y > 0
        lo, hi = np.where(some, np.maximum(lo, LEAST), 0.0), np.where(some, np.maximum(hi, LEAST), 0.0)
    got = pad(code.float().double().cpu().numpy().ravel())
    assert np.all((got >= lo) & (got <= hi))


def check(P, before, G, s, hp, step, bits, gs=1.0):
    for i, p in enumerate(P):
        if p.numel() == 0:
            continue
        p0, m0, v0 = before[i]
        ref, m, v, tp, tm = reference(p0, G[i], m0, v0, hp, step, bits, gs)
        assert_rounded_within(p.flatten(), ref, tp, f"p[{i}]")
        if bits == 32:
            assert np.all(np.abs(f64(s["M"][i]).ravel() - m) <= tm + 1e-44)
            assert np.all(np.abs(f64(s["V"][i]).ravel() - v) <= 10 * W * v + 1e-44)
        else:
            check_codes(s["M"][i], s["m_scales"][i], m, tm, False)
            r = np.sqrt(v)
            check_codes(s["V"][i], s["v_scales"][i], r, 6 * W * r, True)


def snapshot(P, s, bits):
    if bits == 32:
        return [(p.clone(), f64(m).ravel(), f64(v).ravel()) for p, m, v in zip(P, s["M"], s["V"])]
    return [(p.clone(), values(m, ms), values(v, vs))
            for p, m, v, ms, vs in zip(P, s["M"], s["V"], s["m_scales"], s["v_scales"])]


SIZES = [1, 2, 127, 128, 129, 4095, 4096, 4097, 8200, 0, 5]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p_dtype", [BF16, F32])
@pytest.mark.parametrize("g_dtype", [BF16, F32])
def test_parity(p_dtype, g_dtype, bits):
    P, G, s = make(SIZES, p_dtype, g_dtype, bits)
    before = snapshot(P, s, bits)
    hp = mc.AdamHparams(lr=1e-3)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mc.adamw_step(P, G, hp=hp, step=4, status=status, **s)
    torch.cuda.synchronize()
    assert status.item() == 0
    check(P, before, G, s, hp, 4, bits)


@pytest.mark.parametrize("bits", [32, 8])
def test_first_step_moves_by_lr(bits):
    """From zero states m / (1 - beta1) is g and the root of v / (1 - beta2) its magnitude: a step
    of lr against its sign, and of nothing where g is 0 (0 / eps, no 0 / 0)."""
    P, G, s = make([1000], F32, F32, bits, steps_before=0)
    p0 = P[0].clone()
    mc.adamw_step(P, G, hp=mc.AdamHparams(lr=0.5, weight_decay=0.0, eps=1e-30), step=1, **s)
    torch.cuda.synchronize()
    assert torch.allclose(P[0] - p0, -0.5 * torch.sign(G[0]), rtol=1e-5, atol=1e-7)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("count", [16, 17, 128, 129, 504, 600])
def test_many_tensors(count, bits):
    """Every size of the launch's table, and more tensors than one launch takes."""
    sizes = [(i * 37) % 300 + 1 for i in range(count)]
    flat = normal((sum(sizes),), 0.02, "flat").cuda()
    grad = normal((sum(sizes),), 1e-3, "gradient").cuda()
    P, G = list(flat.split(sizes)), list(grad.split(sizes))      # views at any multiple of four bytes
    s = mc.adamw_state(P, bits)
    before = snapshot(P, s, bits)
    hp = mc.AdamHparams()
    mc.adamw_step(P, G, hp=hp, step=1, **s)
    torch.cuda.synchronize()
    check(P, before, G, s, hp, 1, bits)


@pytest.mark.parametrize("bits", [32, 8])
def test_nothing_beside_the_tensors_is_written(bits):
    for lead in (0, 1, 2, 3, 5, 8):
        n = 300
        base = {k: torch.full((n + 32,), 7.0, device="cuda") for k in "pg"}
        state_type = F32 if bits == 32 else F8
        base |= {k: torch.full((n + 32,), 2.0, device="cuda").to(state_type) for k in "mv"}
        cut = lambda t: t[lead:lead + n]  # noqa: E731
        s = dict(M=[cut(base["m"])], V=[cut(base["v"])], m_scales=None, v_scales=None)
        scales = torch.full((2, 5), 3.0, device="cuda")
        if bits == 8:
            s.update(m_scales=[scales[0, 1:4]], v_scales=[scales[1, 1:4]])
        mc.adamw_step([cut(base["p"])], [cut(base["g"])], hp=mc.AdamHparams(lr=0.1), step=2, **s)
        torch.cuda.synchronize()
        for k, t in base.items():
            outside = torch.cat([t.float()[:lead], t.float()[lead + n:]])
            assert torch.all(outside == (7.0 if k in "pg" else 2.0)), (lead, k)
        assert torch.all(base["g"] == 7.0) and torch.all(cut(base["p"]) != 7.0)
        assert torch.all(scales[:, 0] == 3.0) and torch.all(scales[:, 4] == 3.0)


@pytest.mark.parametrize("bits", [32, 8])
def test_grad_scale_and_shapes(bits):
    P = [normal((33, 5), 0.02, "sp").cuda(), normal((4, 3, 2), 0.02, "sq").to(BF16).cuda()]
    G = [normal((33, 5), 1.0, "sg").cuda(), normal((4, 3, 2), 1.0, "sh").cuda()]
    s = mc.adamw_state(P, bits)
    before = snapshot(P, s, bits)
    scale = torch.tensor([0.125], device="cuda")
    hp = mc.AdamHparams()
    mc.adamw_step(P, G, hp=hp, step=1, grad_scale=scale, **s)
    torch.cuda.synchronize()
    check(P, before, G, s, hp, 1, bits, gs=0.125)


def test_nonfinite_gradient_stays_in_its_place():
    for bits in (32, 8):
        P, G, s = make([700], F32, F32, bits)
        Q, H, z = make([700], F32, F32, bits)
        G[0][300] = float("nan")
        G[0][10] = float("inf")
        H[0][300], H[0][10] = 0.0, 0.0
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        mc.adamw_step(P, G, hp=mc.AdamHparams(), step=4, status=status, **s)
        mc.adamw_step(Q, H, hp=mc.AdamHparams(), step=4, **z)
        torch.cuda.synchronize()
        assert status.item() == abi.MC_STATUS_NONFINITE_UPDATE
        keep = torch.ones(700, dtype=torch.bool, device="cuda")
        keep[[10, 300]] = False
        assert torch.equal(P[0][keep], Q[0][keep]) and not torch.isfinite(P[0][300])
        if bits == 8:                    # of the state, its block of 128
            keep[:128] = False
            keep[256:384] = False
            assert torch.isnan(s["m_scales"][0][2]) and torch.isfinite(s["m_scales"][0][1])
        for k in "MV":
            assert torch.equal(s[k][0].float()[keep], z[k][0].float()[keep])


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_step_counts_on(bits):
    """A captured step that reads its number from the device, replayed, equals steps one by one."""
    P, G, s = make([5000, 33], BF16, F32, bits, steps_before=0)
    Q, z = [p.clone() for p in P], copy_of(s)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    hp = mc.AdamHparams(lr=1e-2)
    mc.adamw_step([p.clone() for p in P], G, hp=hp, step=step, **copy_of(s))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.add_(1)
        mc.adamw_step(P, G, hp=hp, step=step, **s)
    step.zero_()
    for _ in range(3):
        graph.replay()
    for t in range(3):
        mc.adamw_step(Q, G, hp=hp, step=t + 1, **z)
    torch.cuda.synchronize()
    assert step.item() == 3
    for a, b in zip(P, Q):               # the factors of t come from two libraries' expm1: an ulp of the update at most
        assert torch.all((a.float() - b.float()).abs() <= 2.0 ** -8 * b.float().abs() + 1e-12)
    for a, b in zip(s["M"] + s["V"], z["M"] + z["V"]):
        assert torch.equal(a.float(), b.float())


def test_equal_inputs_give_equal_bits_on_any_stream():
    P, G, s = make([40000, 777], BF16, BF16, 8)
    Q, z = [p.clone() for p in P], copy_of(s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    mc.adamw_step(P, G, hp=mc.AdamHparams(), step=4, **s)
    mc.adamw_step(Q, G, hp=mc.AdamHparams(), step=4, stream=side, **z)
    torch.cuda.synchronize()
    for a, b in zip(P + s["M"] + s["V"], Q + z["M"] + z["V"]):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_tensor_of_more_than_2_to_31_values():
    n = (1 << 31) + 4099
    p = torch.zeros(n, dtype=BF16, device="cuda")
    g = torch.zeros(n, dtype=BF16, device="cuda")
    at = torch.tensor([0, (1 << 31) - 1, 1 << 31, n - 1], device="cuda")
    p[at] = 1.0
    g[at] = 0.5
    s = mc.adamw_state([p], 8)
    mc.adamw_step([p], [g], hp=mc.AdamHparams(lr=0.25, weight_decay=0.0), step=1, **s)
    torch.cuda.synchronize()
    assert torch.all(p[at] == 0.75) and int((p != 0).sum()) == 4 and int((s["M"][0].view(torch.uint8) != 0).sum()) == 4


def test_eight_bit_states_equal_operations_of_one_rounding_each():
    """m, v and their scales have the bits of elementary fp32 operations in the order of the
    formulas, step after step: no products and sums contracted to one rounding."""
    n = 1 << 20
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    P = [torch.randn(n, generator=g, device="cuda").to(BF16)]
    s, hp = mc.adamw_state(P, 8), mc.AdamHparams()
    m8, v8, ms, vs = (s[k][0].clone() for k in ("M", "V", "m_scales", "v_scales"))
    rows = lambda t: t.view(-1, 128)  # noqa: E731

    def codes(x, least):
        scale = (rows(x).abs().amax(1) * torch.tensor(1 / 448, device="cuda")).clamp(min=SCALE_MIN)
        y = rows(x) * (1.0 / scale)[:, None]
        if least:
            y = torch.where((y > 0) & (y < LEAST), torch.full_like(y, LEAST), y)
        return y.to(F8).flatten(), scale

    for t in range(1, 4):
        G = (torch.randn(n, generator=g, device="cuda") * 1e-3).to(BF16)
        mc.adamw_step(P, [G], hp=hp, step=t, **s)
        gf = G.float()
        m = (rows(m8.float()) * ms[:, None]).flatten()
        r = (rows(v8.float()) * vs[:, None]).flatten()
        a, b = m * hp.beta1, gf * (1.0 - hp.beta1)
        m = a + b
        a, b = (r * r) * hp.beta2, (gf * gf) * (1.0 - hp.beta2)
        v = a + b
        (m8, ms), (v8, vs) = codes(m, False), codes(v.sqrt(), True)
        for name, own, want in (("m", s["M"][0], m8), ("v", s["V"][0], v8)):
            assert torch.equal(own.view(torch.uint8), want.view(torch.uint8)), (t, name)
        assert torch.equal(s["m_scales"][0], ms) and torch.equal(s["v_scales"][0], vs), t


@pytest.mark.parametrize("gradients", ["alike", "uneven", "falling"])
def test_eight_bit_states_follow_32_bit_ones_over_many_steps(gradients):
    """400 steps at the default betas, Gaussian gradients of one scale, of scales that differ from value
    to value, and of which every other falls tenfold after 100 steps.  The header's formulas, run on the
    CPU, give a median of v between 0.99 and 1.11 times the 32-bit state's, updates' norms of 0.95 to
    1.01 times and a correlation of 0.995; the bounds leave twice these distances."""
    n, hp = 1 << 17, mc.AdamHparams(lr=0.0, weight_decay=0.0)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(6)
    scale = torch.exp(torch.randn(n, generator=gen, device="cuda")) if gradients == "uneven" else torch.ones(n, device="cuda")
    P = [torch.ones(n, device="cuda")]
    small, wide = mc.adamw_state(P, 8), mc.adamw_state(P, 32)
    for t in range(1, 401):
        if gradients == "falling" and t == 101:
            scale[1::2] *= 0.1
        G = [torch.randn(n, generator=gen, device="cuda") * scale]
        for s in (small, wide):
            mc.adamw_step(P, G, hp=hp, step=t, **s)
    m = values(small["M"][0], small["m_scales"][0])
    r = values(small["V"][0], small["v_scales"][0])
    M, V = f64(wide["M"][0]), f64(wide["V"][0])
    for part in (slice(0, None, 2), slice(1, None, 2)):
        u, U = m[part] / (r[part] + 1e-8), M[part] / (np.sqrt(V[part]) + 1e-8)
        assert 0.9 <= np.median(r[part] ** 2 / V[part]) <= 1.22
        assert 0.9 <= np.linalg.norm(u) / np.linalg.norm(U) <= 1.02 and np.dot(u, U) >= 0.99 * np.linalg.norm(u) * np.linalg.norm(U)


@pytest.mark.parametrize("beta1,beta2", [(0.9, 0.95), (0.0, 0.999), (0.5, 0.0), (0.999, 0.9999), (1 - 1e-7, 1 - 1e-9)])
def test_step_on_the_device_at_any_number(beta1, beta2):
    """The factors of a step that is read on the device, from 1 to numbers whose powers are 0: the
    update m i1 / (sqrt(v) i2 + eps) of m = v = g = 1 (which they stay, to 2 w) within 4 w for m and
    v's root, 5 w for i1 (2 ulp and a quotient), 4 w for i2 (half of 2 ulp, root, quotient), 2 w for
    fma and product and 4 w for the quotient: 20 w."""
    hp = mc.AdamHparams(lr=1.0, beta1=beta1, beta2=beta2, eps=0.0, weight_decay=0.0)
    one = lambda: [torch.ones(5, device="cuda")]  # noqa: E731
    for t in (-3, 0, 1, 2, 3, 10, 1000, 12345, 10 ** 6, (1 << 24) + 1, (1 << 31) + 5, 1 << 40, (1 << 62) + 1, (1 << 63) - 1):
        P = [torch.zeros(5, device="cuda")]
        mc.adamw_step(P, one(), one(), one(), hp=hp, step=torch.tensor([t], device="cuda"))
        torch.cuda.synchronize()
        n = np.float64(max(t, 1))
        power = lambda b: np.expm1(n * np.log(b)) if b else -1.0  # noqa: E731
        u = -1.0 / power(beta1) * np.sqrt(-power(beta2))
        assert np.all(np.abs(f64(P[0]) + u) <= 20 * W * u), (t, P[0], u)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p_dtype", [BF16, F32])
@pytest.mark.parametrize("g_dtype", [BF16, F32])
def test_large_dense_tensors(p_dtype, g_dtype, bits):
    """25 million values in three tensors of odd sizes, one operand of each an element off every
    alignment: chunks of the most steps, ragged ends inside a late one, scale blocks in all of them.
    m, v, codes and scales have the bits of elementary fp32 operations; p lies within its rounding and
    lr's share of 20 roundings of the update."""
    sizes, off = (12_000_037, 9_000_001, 4_000_003), ("p", "g", "m")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(8)

    def place(x, shifted):
        held = torch.empty(x.numel() + 32, dtype=x.dtype, device="cuda")
        got = held[1:1 + x.numel()] if shifted else held[:x.numel()]
        return got.copy_(x)

    def codes(x, least):
        n = x.numel()
        rows = torch.nn.functional.pad(x, (0, -n % 128)).view(-1, 128)
        scale = (rows.abs().amax(1) * torch.tensor(1 / 448, device="cuda")).clamp(min=SCALE_MIN)
        y = rows * (1.0 / scale)[:, None]
        if least:
            y = torch.where((y > 0) & (y < LEAST), torch.full_like(y, LEAST), y)
        return y.to(F8).flatten()[:n], scale

    wide = lambda c, s: (c.float() * s.repeat_interleave(128)[:c.numel()])  # noqa: E731
    P, G, M, V, ms, vs = [], [], [], [], [], []
    for n, o in zip(sizes, off):
        loud = torch.exp(torch.randn(n, generator=gen, device="cuda"))
        P.append(place((torch.randn(n, generator=gen, device="cuda") * 0.02).to(p_dtype), o == "p"))
        G.append(place((torch.randn(n, generator=gen, device="cuda") * 1e-3 * loud).to(g_dtype), o == "g"))
        m, r = torch.randn(n, generator=gen, device="cuda") * 3e-4 * loud, 1e-3 * loud * (0.2 + torch.rand(n, generator=gen, device="cuda"))
        if bits == 8:
            (m, a), (r, b) = codes(m, False), codes(r, True)
            ms.append(a)
            vs.append(b)
        M.append(place(m, o == "m"))
        V.append(place(r if bits == 8 else r * r, False))
    before = [(p.clone(), wide(m, a) if bits == 8 else m.clone(), wide(v, b).square() if bits == 8 else v.clone())
              for p, m, v, a, b in zip(P, M, V, ms or sizes, vs or sizes)]
    hp, t = mc.AdamHparams(lr=1e-2), 50
    mc.adamw_step(P, G, M, V, hp=hp, step=t, m_scales=ms or None, v_scales=vs or None)
    for i, (p0, m, v) in enumerate(before):
        g = G[i].float()
        a, b = m * hp.beta1, g * (1.0 - hp.beta1)
        m = a + b
        a, b = v * hp.beta2, (g * g) * (1.0 - hp.beta2)
        v = a + b
        if bits == 8:
            for own, scale, x, least in ((M[i], ms[i], m, False), (V[i], vs[i], v.sqrt(), True)):
                want, s = codes(x, least)
                assert torch.equal(own.view(torch.uint8), want.view(torch.uint8)) and torch.equal(scale, s), i
        else:
            assert torch.equal(M[i], m) and torch.equal(V[i], v), i
        u = m.double() / (1 - hp.beta1 ** t) / ((v.double() / (1 - hp.beta2 ** t)).sqrt() + hp.eps)
        p = p0.double() - hp.lr * (u + hp.weight_decay * p0.double())
        tol = hp.lr * 20 * W * (u.abs() + p0.double().abs()) + 1.0001 * torch.finfo(p_dtype).eps / 2 * p.abs()
        assert torch.all((P[i].double() - p).abs() <= tol), i


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("at", [0, 17, 1999, 2002])
def test_overflow_in_the_rounding_of_p_sets_the_status(bits, at):
    """A step that takes a bf16 value beyond the largest by more than half a step: finite in fp32,
    infinite as stored.  One that stays below half a step sets nothing."""
    top = float(torch.finfo(BF16).max)                     # 2^128 - 2^120; infinity begins at 2^128 - 2^119
    for lr, status in ((2.0 ** 119 * 1.25, abi.MC_STATUS_NONFINITE_UPDATE), (2.0 ** 119 * 0.5, 0)):
        P, G = [torch.zeros(2003, dtype=BF16, device="cuda")], [torch.zeros(2003, device="cuda")]
        P[0][at], G[0][at] = top, -1.0
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        s = mc.adamw_state(P, bits)
        mc.adamw_step(P, G, hp=mc.AdamHparams(lr=lr, weight_decay=0.0), step=1, status=st, **s)
        torch.cuda.synchronize()
        assert st.item() == status and bool(torch.isinf(P[0][at])) == bool(status)
        assert int((P[0] != 0).sum()) == 1


def test_small_roots_stay_above_zero_while_their_squares_are_in_range():
    """Blocks whose scale is 2^e, every positive code among them, without a gradient: a root of 2^-74 or
    more does not become zero, in one step or in 400 (which lower the scale by 2^-15); smaller ones may,
    as v may in a 32-bit state, since their squares are below 2^-149."""
    codes = torch.arange(1, 127, dtype=torch.uint8, device="cuda").view(F8)      # 2^-9 .. 448
    for e in (0, -40, -65, -66, -80, -100):
        V = torch.zeros(128, dtype=F8, device="cuda")
        V[:126] = codes
        r0 = f64(V.float()) * 2.0 ** e
        s = dict(M=[torch.zeros(128, dtype=F8, device="cuda")], V=[V], m_scales=[torch.ones(1, device="cuda")],
                 v_scales=[torch.full((1,), 2.0 ** e, device="cuda")])
        wide = dict(M=[torch.zeros(128, device="cuda")], V=[torch.tensor(r0 * r0).float().cuda()])
        for t in range(400 if e >= -40 else 1):
            for state in (s, wide):
                mc.adamw_step([torch.ones(128, device="cuda")], [torch.zeros(128, device="cuda")], step=t + 1, **state)
        torch.cuda.synchronize()
        safe, r = r0 >= 2.0 ** -74, values(s["V"][0], s["v_scales"][0])
        assert np.all(r[safe] > 0) and np.all(r[r0 == 0] == 0)
        assert np.all(f64(wide["V"][0])[safe] > 0)
