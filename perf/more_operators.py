"""The operators around a packed training step, as measured: causal attention over packed sequences with
grouped heads (forward with the per-head max logit, backward), the norm of every query and key head with
its rotary embedding in one pass (forward, backward), and the AdamW step of the parameters that Muon
leaves out (states in 32 or in 8 bits).

own = False runs them in plain torch (fp32, products and sums written out); own = True makes the calls
of muon_qk_clip_gb300 that a training step makes.  Inputs follow the repository's workloads: bf16
features of N(0, 1), one head in four with its queries scaled so that its softmax is nearly one-hot
(the heads QK-Clip is about), gradients of N(0, 1e-2).
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
E4M3_LEAST = 2.0 ** -9
SCALE_MIN = 2.0 ** -100
BLOCK = 128                     # values per scale of an 8-bit state
EPS = 1e-6
THETA = 10000.0
BETA1, BETA2, ADAM_EPS, LR, DECAY = 0.9, 0.95, 1e-8, 2e-4, 0.1


# ------------------------------------------------------------------------------------------- cases
def listed():
    fwd, bwd = dict(op="packed_forward"), dict(op="packed_backward")
    norm, norm_back = dict(op="norm_rope"), dict(op="norm_rope_backward")
    adam = dict(op="adamw")
    return [
        # four short prompts: launch latency decides
        dict(name="packed_fwd_prompts", **fwd, T=366, nseq=4, cut=3, Hq=8, Hkv=2, d=64, dv=64),
        # documents packed into the tokens of a training batch, four query heads per key head
        dict(name="packed_fwd_documents", **fwd, T=16384, nseq=8, cut=5, Hq=32, Hkv=8, d=128, dv=128),
        # one long sequence, eight query heads per key head, a length off every tile
        dict(name="packed_fwd_long", **fwd, T=24571, nseq=1, cut=0, Hq=16, Hkv=2, d=128, dv=128),
        # the documents' gradients
        dict(name="packed_bwd_documents", **bwd, T=16384, nseq=8, cut=5, Hq=32, Hkv=8, d=128, dv=128),
        # many short samples of a fine-tuning batch, three query heads per key head, odd widths
        dict(name="packed_bwd_samples", **bwd, T=4093, nseq=31, cut=7, Hq=6, Hkv=2, d=80, dv=48),
        # one decoded token of a 64-head layer
        dict(name="norm_rope_token", **norm, T=1, Hq=64, Hkv=8, d=128, rot=128, dtype="bf16", weight=True, fused=True),
        # a training batch, q and k as views of one projection
        dict(name="norm_rope_batch", **norm, T=16384, Hq=32, Hkv=8, d=128, rot=128, dtype="bf16", weight=True, fused=True),
        # its gradient, with the weights'
        dict(name="norm_rope_bwd_batch", **norm_back, T=16384, Hq=32, Hkv=8, d=128, rot=128, dtype="bf16", weight=True, fused=True),
        # partly rotated heads of an odd width in fp32, a short odd batch
        dict(name="norm_rope_bwd_odd_fp32", **norm_back, T=1021, Hq=5, Hkv=1, d=90, rot=30, dtype="fp32", weight=True, fused=False),
        # the norm weights of a deep stack, 122 vectors of a 7168-wide layer: many small tensors
        dict(name="adamw_norm_weights", **adam, tables=0, rows=1, cols=1, vecs=122, vlen=7168, p="fp32", g="fp32", bits=32, step=1),
        # embedding and output tables of a 2048-wide block, with its norms
        dict(name="adamw_tables", **adam, tables=2, rows=65536, cols=2048, vecs=48, vlen=2048, p="bf16", g="bf16", bits=32, step=1000),
        # the same with 8-bit states, a row count off every block
        dict(name="adamw_tables_8bit", **adam, tables=2, rows=65521, cols=2048, vecs=48, vlen=1531, p="bf16", g="bf16", bits=8, step=1000),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["packed_forward", "packed_forward", "packed_backward", "packed_backward", "norm_rope", "norm_rope_backward", "adamw", "adamw"])
    if op.startswith("packed"):
        c = dict(op=op, T=_log(rng, 1, 24571), nseq=_log(rng, 1, 48), cut=rng.randint(1, 1 << 20), Hq=1, Hkv=rng.randint(1, 8),
                 d=8 * rng.randint(2, 16), dv=8 * rng.randint(2, 16))
        if rng.random() < 0.4:
            c.update(d=rng.choice([64, 128]))
            c.update(dv=c["d"])
        group = rng.randint(1, 8)
        while True:
            c["Hq"] = c["Hkv"] * group
            longest = max(lengths(c))
            pairs = c["Hq"] * sum(n * n for n in lengths(c))
            if pairs <= 3.6e9 and c["nseq"] * c["Hq"] * longest ** 2 <= 8e9:
                return c
            if group > 1:
                group -= 1
            elif c["Hkv"] > 1:
                c["Hkv"] -= 1
            else:
                c["T"] = c["T"] * 2 // 3
    if op.startswith("norm_rope"):
        d = 2 * rng.randint(8, 128) if rng.random() < 0.5 else rng.choice([64, 128, 192, 256])
        c = dict(op=op, T=_log(rng, 1, 32768), Hq=rng.randint(1, 64), Hkv=rng.randint(1, 8), d=d, rot=rng.choice([d, d, 2 * rng.randint(0, d // 2)]),
                 dtype=rng.choice(["bf16", "bf16", "fp32"]), weight=rng.random() < 0.8, fused=rng.random() < 0.5)
        c["T"] = max(1, min(c["T"], 16384 * 40 * 128 // (c["d"] * (c["Hq"] + c["Hkv"]) * (1 if c["dtype"] == "bf16" else 2))))
        return c
    c = dict(op=op, tables=rng.randint(0, 3), rows=_log(rng, 1, 40000), cols=_log(rng, 16, 8192), vecs=rng.randint(1, 64), vlen=_log(rng, 1, 8192),
             p=rng.choice(["bf16", "bf16", "fp32"]), g=rng.choice(["bf16", "fp32"]), bits=rng.choice([8, 32]), step=_log(rng, 1, 20000))
    c["rows"] = max(1, min(c["rows"], 60_000_000 // c["cols"]))
    return c


def lengths(c):
    """The lengths of a packed case's sequences: T tokens cut into nseq parts of very different sizes (some may be empty)."""
    rng = random.Random(c["cut"])
    shares = [rng.expovariate(1.0) for _ in range(c["nseq"])]
    at, cuts, total = 0.0, [0], sum(shares)
    for s in shares:
        at += s
        cuts.append(int(round(c["T"] * at / total)))
    cuts[-1] = c["T"]
    return [b - a for a, b in zip(cuts, cuts[1:])]


def sizes(c):
    """(values, place) of an AdamW case's tensors in their flat buffers, each on a boundary of 128 values."""
    got, at = [], 0
    for n in [c["rows"] * c["cols"]] * c["tables"] + [c["vlen"]] * c["vecs"]:
        got.append((n, at))
        at += -(-n // BLOCK) * BLOCK
    return got, at


def _bytes(name):
    return 2 if name == "bf16" else 4


def work(c):
    if c["op"].startswith("packed"):
        H, G, d, dv, T = c["Hq"], c["Hkv"], c["d"], c["dv"], c["T"]
        pairs = H * sum(n * (n + 1) // 2 for n in lengths(c))
        read = 2 * T * (H * d + G * (d + dv))
        if c["op"] == "packed_forward":
            return {"bytes": read + 2 * T * H * dv + 4 * T * H + 4 * H, "flops": 2 * pairs * (d + dv)}
        return {"bytes": 2 * read + 4 * T * H * dv + 4 * T * H, "flops": pairs * (6 * d + 4 * dv)}
    if c["op"].startswith("norm_rope"):
        es, rows = _bytes(c["dtype"]), c["T"] * (c["Hq"] + c["Hkv"])
        back = c["op"] == "norm_rope_backward"
        vectors = 2 * c["d"] * (es + 4 * back) if c["weight"] else 0
        return {"bytes": rows * (c["d"] * es * (3 if back else 2) + 4) + 4 * c["T"] + vectors, "flops": rows * c["d"] * (12 if back else 7)}
    n = sum(x for x, _ in sizes(c)[0])
    blocks = sum(-(-x // BLOCK) for x, _ in sizes(c)[0])
    state = 16 * n if c["bits"] == 32 else 4 * n + 16 * blocks
    return {"bytes": n * (2 * _bytes(c["p"]) + _bytes(c["g"])) + state, "flops": 14 * n}


# ------------------------------------------------------------------------------------------ inputs
def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device="cuda") * std

    s = {"case": c}
    if c["op"].startswith("packed"):
        T, H, G, d, dv = (c[n] for n in ("T", "Hq", "Hkv", "d", "dv"))
        sharp = 1.0 + 11.0 * (torch.arange(H, device="cuda") % 4 == 1)
        s["q"] = (normal(T, H, d) * sharp[:, None]).bfloat16()
        s["k"], s["v"] = normal(T, G, d).bfloat16(), normal(T, G, dv).bfloat16()
        ends = torch.tensor([0] + lengths(c), dtype=torch.int64).cumsum(0)
        s["offsets"] = ends.to(torch.int32).cuda()
        s["scale"] = 1.0 / math.sqrt(d)
        # where token i of sequence b stands, for the plain form: a padded batch, and which of its places exist
        longest = max(lengths(c))
        i = torch.arange(longest)
        s["there"] = (i[None, :] < (ends[1:] - ends[:-1])[:, None]).cuda()
        s["rows"] = (ends[:-1, None] + i).clamp(max=T - 1).cuda()
        if c["op"] == "packed_backward":
            s["do"] = normal(T, H, dv, std=1e-2).bfloat16()
            s["o"], s["lse"], _ = _plain_packed_forward(s)
    elif c["op"].startswith("norm_rope"):
        T, H, G, d, t = c["T"], c["Hq"], c["Hkv"], c["d"], _dtype(c["dtype"])
        loud = 1.0 + 4.0 * (torch.rand(d, generator=gen, device="cuda") < 0.05)   # a few large channels
        if c["fused"]:
            both = (normal(T, H + 2 * G, d) * loud).to(t)          # queries, keys and values of one projection
            s["q"], s["k"] = both[:, :H], both[:, H:H + G]
        else:
            s["q"], s["k"] = (normal(T, H, d) * loud).to(t), (normal(T, G, d) * loud).to(t)
        s["wq"], s["wk"] = ((1.0 + 0.1 * normal(d)).to(t) for _ in range(2)) if c["weight"] else (None, None)
        # packed sequences: positions begin again at a few places
        breaks = torch.rand(T, generator=gen, device="cuda") < 4.0 / T
        at = torch.arange(T, device="cuda")
        s["positions"] = (at - torch.where(breaks, at, torch.zeros_like(at)).cummax(0).values).to(torch.int32)
        if c["op"] == "norm_rope_backward":
            s["dyq"], s["dyk"] = normal(T, H, d, std=1e-2).to(t), normal(T, G, d, std=1e-2).to(t)
            s["rstd"] = torch.cat([_rstd(s["q"].float()), _rstd(s["k"].float())], 1)
    else:
        parts, total = sizes(c)
        first = c["step"] == 1
        loud = torch.exp(normal(total // BLOCK))[:, None].expand(-1, BLOCK).reshape(-1)   # tensors' rows differ in scale
        s["p"] = normal(total, std=0.02).to(_dtype(c["p"]))
        s["g"] = (normal(total, std=1e-3) * loud).to(_dtype(c["g"]))
        m = torch.zeros(total, device="cuda") if first else normal(total, std=3e-4) * loud
        v = torch.zeros(total, device="cuda") if first else (1e-3 * loud * (0.2 + normal(total).abs())).square()
        if c["bits"] == 8:
            s["m"], s["ms"] = _quantise(m, False)
            s["v"], s["vs"] = _quantise(v.sqrt(), True)
        else:
            s["m"], s["v"], s["ms"], s["vs"] = m, v, None, None
        cut = lambda t: None if t is None else [t[a:a + n] for n, a in parts]  # noqa: E731
        blocks = lambda t: None if t is None else [t[a // BLOCK:a // BLOCK + -(-n // BLOCK)] for n, a in parts]  # noqa: E731
        s["lists"] = dict(P=cut(s["p"]), G=cut(s["g"]), M=cut(s["m"]), V=cut(s["v"]), m_scales=blocks(s["ms"]), v_scales=blocks(s["vs"]))
        inside = torch.zeros(total, dtype=torch.bool)
        for n, a in parts:
            inside[a:a + n] = True
        s["inside"] = None if bool(inside.all()) else inside.cuda()   # between the tensors lies nothing of theirs
    return s


# -------------------------------------------------------------------------------------- plain forms
def _grouped(s, name):
    """[batch, key heads, heads per key head, position, feature] of a packed tensor, in fp32."""
    x, G = s[name], s["case"]["Hkv"]
    return x[s["rows"]].float().unflatten(2, (G, x.shape[1] // G)).permute(0, 2, 3, 1, 4)


def _packed(s, x):
    """The tokens [T, heads, feature] of a grouped padded batch."""
    return x.permute(0, 3, 1, 2, 4).flatten(2, 3)[s["there"]]


def _logits(s):
    x = torch.matmul(_grouped(s, "q"), _grouped(s, "k").transpose(3, 4)).mul_(s["scale"])
    i = torch.arange(x.shape[-1], device=x.device)
    seen = (i[None, :] <= i[:, None]) & s["there"][:, :, None]
    return x.masked_fill_(~seen[:, None, None], -math.inf)


def _plain_packed_forward(s):
    x = _logits(s)
    top = x.amax(-1, keepdim=True)
    smax = top.amax((0, 3, 4)).flatten()
    top = top.clamp(min=-3e38)                                     # rows that do not exist
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x, _grouped(s, "v")).div_(total)
    lse = _packed(s, top + total.log())[..., 0].t().contiguous()
    return _packed(s, o).to(s["q"].dtype), lse, smax


def _plain_packed_backward(s):
    t, G = s["q"].dtype, s["case"]["Hkv"]
    lse = s["lse"].t()[s["rows"]].unflatten(2, (G, -1)).permute(0, 2, 3, 1)
    p = _logits(s).sub_(lse[..., None]).exp_()
    do = _grouped(s, "do") * s["there"][:, None, None, :, None]
    dv = torch.matmul(p.transpose(3, 4), do).sum(2, keepdim=True)
    delta = (do * _grouped(s, "o")).sum(-1, keepdim=True)
    ds = torch.matmul(do, _grouped(s, "v").transpose(3, 4)).sub_(delta).mul_(p)
    ds[..., 0, :] = 0.0                                            # one key: the softmax is 1 whatever its logit
    dq = torch.matmul(ds, _grouped(s, "k")) * s["scale"]
    dk = torch.matmul(ds.transpose(3, 4), _grouped(s, "q")).sum(2, keepdim=True) * s["scale"]
    return _packed(s, dq).to(t), _packed(s, dk).to(t), _packed(s, dv).to(t)


def _rstd(x):
    return 1.0 / torch.sqrt((x * x).mean(-1) + EPS)


def _turns(s):
    """Cosine and sine [T, 1, rot / 2] of every position's angles, from 64 bits."""
    rot = s["case"]["rot"]
    freq = THETA ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / max(rot, 1))
    angle = s["positions"].double()[:, None] * freq
    return angle.cos().float()[:, None], angle.sin().float()[:, None]


def _rotate(x, cos, sin):
    """The last 2 cos.shape[-1] features of x, as interleaved pairs, turned."""
    rest, last = x[..., :x.shape[-1] - 2 * cos.shape[-1]], x[..., x.shape[-1] - 2 * cos.shape[-1]:]
    a, b = last[..., 0::2], last[..., 1::2]
    return torch.cat([rest, torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)], -1)


def _plain_norm_rope(s):
    cos, sin = _turns(s)
    q, k = s["q"].float(), s["k"].float()
    rq, rk = _rstd(q), _rstd(k)
    q, k = q * rq[..., None], k * rk[..., None]
    if s["wq"] is not None:
        q, k = q * s["wq"].float(), k * s["wk"].float()
    return _rotate(q, cos, sin).to(s["q"].dtype), _rotate(k, cos, sin).to(s["q"].dtype), torch.cat([rq, rk], 1)


def _norm_rope_gradient(x, dy, rstd, w, cos, sin):
    xhat = x.float() * rstd[..., None]
    dz = _rotate(dy.float(), cos, -sin)
    g = dz if w is None else dz * w.float()
    dx = (g - xhat * (g * xhat).mean(-1, keepdim=True)) * rstd[..., None]
    return dx.to(x.dtype), None if w is None else (dz * xhat).sum((0, 1))


def _plain_norm_rope_backward(s):
    cos, sin = _turns(s)
    rq, rk = s["rstd"].split([s["case"]["Hq"], s["case"]["Hkv"]], 1)
    dq, dwq = _norm_rope_gradient(s["q"], s["dyq"], rq, s["wq"], cos, sin)
    dk, dwk = _norm_rope_gradient(s["k"], s["dyk"], rk, s["wk"], cos, sin)
    return dq, dk, dwq, dwk


def _codes(x, least):
    """x [blocks, 128] in e4m3 with one scale per block; with `least` (the root of v, which divides), no
    positive value becomes zero."""
    scale = (x.abs().amax(-1) / E4M3_MAX).clamp(min=SCALE_MIN)
    y = x * (1.0 / scale)[:, None]
    if least:
        y = torch.where((y > 0) & (y < E4M3_LEAST), torch.full_like(y, E4M3_LEAST), y)
    return y.to(torch.float8_e4m3fn), scale


def _quantise(x, least):
    codes, scales = _codes(x.view(-1, BLOCK), least)
    return codes.flatten(), scales


def _plain_adamw(s):
    c = s["case"]
    g, p = s["g"].float(), s["p"].float()
    if c["bits"] == 8:
        m = (s["m"].float().view(-1, BLOCK) * s["ms"][:, None]).flatten()
        r = (s["v"].float().view(-1, BLOCK) * s["vs"][:, None]).flatten()
        v = r * r
    else:
        m, v = s["m"], s["v"]
    if s["inside"] is not None:
        g = torch.where(s["inside"], g, torch.zeros_like(g))
    m = m * BETA1 + g * (1.0 - BETA1)
    v = v * BETA2 + g * g * (1.0 - BETA2)
    step = (m / (1.0 - BETA1 ** c["step"])) / ((v / (1.0 - BETA2 ** c["step"])).sqrt() + ADAM_EPS) + p * DECAY
    p = p - step * LR
    keep = (lambda new, old: new) if s["inside"] is None else (lambda new, old: torch.where(s["inside"], new, old))
    s["p"].copy_(keep(p.to(s["p"].dtype), s["p"]))
    if c["bits"] == 8:
        r = v.sqrt()
        if s["inside"] is not None:
            m, r = torch.where(s["inside"], m, torch.zeros_like(m)), torch.where(s["inside"], r, torch.zeros_like(r))
        m8, ms = _quantise(m, False)
        v8, vs = _quantise(r, True)
        s["ms"].copy_(ms)
        s["vs"].copy_(vs)
        s["m"].copy_(keep(m8.float(), s["m"].float()).to(torch.float8_e4m3fn))
        s["v"].copy_(keep(v8.float(), s["v"].float()).to(torch.float8_e4m3fn))
    else:
        s["m"].copy_(keep(m, s["m"]))
        s["v"].copy_(keep(v, s["v"]))
    return s["p"], s["m"], s["v"], s["ms"], s["vs"]


# --------------------------------------------------------------------------------------------- run
def run(s):
    c, op = s["case"], s["case"]["op"]
    if not own:
        return {"packed_forward": _plain_packed_forward, "packed_backward": _plain_packed_backward, "norm_rope": _plain_norm_rope,
                "norm_rope_backward": _plain_norm_rope_backward, "adamw": _plain_adamw}[op](s)
    from muon_qk_clip_gb300 import binding as mc
    if op == "packed_forward":
        return mc.qk_attention_packed_forward(s["q"], s["k"], s["v"], s["offsets"], scale=s["scale"], lse=True)
    if op == "packed_backward":
        return mc.qk_attention_packed_backward(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], s["offsets"], scale=s["scale"])
    if op == "norm_rope":
        return mc.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], positions=s["positions"], rot=c["rot"], theta=THETA, eps=EPS)
    if op == "norm_rope_backward":
        return mc.qk_norm_rope_backward(s["dyq"], s["dyk"], s["q"], s["k"], s["rstd"], s["wq"], s["wk"], positions=s["positions"],
                                        rot=c["rot"], theta=THETA)
    hp = mc.AdamHparams(lr=LR, beta1=BETA1, beta2=BETA2, eps=ADAM_EPS, weight_decay=DECAY)
    mc.adamw_step(**s["lists"], hp=hp, step=c["step"])
    return s["p"], s["m"], s["v"], s["ms"], s["vs"]


# ------------------------------------------------------------------------------------------- exact
def exact(c, seed):
    s = prepare(c, seed)
    if c["op"].startswith("packed"):
        return _exact_packed(c, s)
    if c["op"].startswith("norm_rope"):
        return _exact_norm_rope(c, s)
    p, m, v, ms, vs = (None if s[n] is None else s[n].double() for n in ("p", "m", "v", "ms", "vs"))
    for n, a in sizes(c)[0]:
        at, blocks = slice(a, a + n), slice(a // BLOCK, a // BLOCK + -(-n // BLOCK))
        wide = lambda t: t[blocks].repeat_interleave(BLOCK)[:n]  # noqa: E731
        gr = s["g"][at].double()
        m1 = m[at] if ms is None else m[at] * wide(ms)
        v1 = v[at] if vs is None else (v[at] * wide(vs)).pow(2)
        m1 = BETA1 * m1 + (1 - BETA1) * gr
        v1 = BETA2 * v1 + (1 - BETA2) * gr.pow(2)
        update = m1 / (1 - BETA1 ** c["step"]) / (torch.sqrt(v1 / (1 - BETA2 ** c["step"])) + ADAM_EPS)
        p[at] -= LR * (update + DECAY * p[at])
        if ms is None:
            m[at], v[at] = m1, v1
            continue
        for state, scales, x in ((m, ms, m1), (v, vs, v1.sqrt())):
            top = torch.nn.functional.pad(x.abs(), (0, -n % BLOCK)).view(-1, BLOCK).max(-1).values
            scales[blocks] = torch.clamp(top / E4M3_MAX, min=SCALE_MIN)
            y = x / wide(scales)
            state[at] = _to_e4m3(torch.clamp(y, min=E4M3_LEAST) * (y > 0) if state is v else y)
    return p, m, v, ms, vs


def _to_e4m3(x):
    """The e4m3 value nearest to x, ties to even: 4 significand bits, quanta of 2^-9 below 2^-6."""
    e = torch.frexp(x)[1].clamp(min=-5) - 4
    quantum = torch.ldexp(torch.ones_like(x), e)
    return (torch.round(x / quantum) * quantum).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_norm_rope(c, s):
    rot, d = c["rot"], c["d"]
    n = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    angle = torch.outer(s["positions"].double(), torch.exp(-2.0 * n / max(rot, 1) * math.log(THETA)))

    def turned(x, sign):
        z = torch.view_as_complex(x[..., d - rot:].unflatten(-1, (-1, 2)).contiguous()) if rot else None
        if rot:
            z = z * torch.polar(torch.ones_like(angle), sign * angle)[:, None]
            x = torch.cat([x[..., :d - rot], torch.view_as_real(z).flatten(-2)], -1)
        return x

    out, rs, dws = [], [], []
    for x, w, dy in ((s["q"], s["wq"], s.get("dyq")), (s["k"], s["wk"], s.get("dyk"))):
        x = x.double()
        w = torch.ones(d, device="cuda", dtype=torch.float64) if w is None else w.double()
        if dy is None:
            r = (x.pow(2).sum(-1) / d + EPS).pow(-0.5)
            out.append(turned(torch.einsum("thc,th,c->thc", x, r, w), 1.0))
            rs.append(r)
            continue
        r = s["rstd"].double()
        r = r[:, c["Hq"]:] if out else r[:, :c["Hq"]]
        dz = turned(dy.double(), -1.0)
        inner = torch.einsum("thc,c,thc,th->th", dz, w, x, r) / d
        out.append(dz * w * r[..., None] - x * (r * r * inner)[..., None])
        dws.append(torch.einsum("thc,thc,th->c", dz, x, r) if c["weight"] else None)
    return (*out, *dws) if dws else (*out, torch.cat(rs, 1))


def _exact_packed(c, s):
    H, group, back = c["Hq"], c["Hq"] // c["Hkv"], c["op"] == "packed_backward"
    if H * sum(n * n for n in lengths(c)) * (c["d"] + c["dv"]) * (5 if back else 2) > 1.2e13:
        return None
    new = lambda like, *shape: torch.zeros(*(shape or like.shape), device="cuda", dtype=torch.float64)  # noqa: E731
    o, lse, smax = new(None, c["T"], H, c["dv"]), new(None, H, c["T"]), torch.full((H,), -math.inf, device="cuda", dtype=torch.float64)
    dq, dk, dv = new(s["q"]), new(s["k"]), new(s["v"])
    at = 0
    for n in lengths(c):
        rows, at = slice(at, at + n), at + n
        if n == 0:
            continue
        for h in range(H):
            q, k, v = s["q"][rows, h].double(), s["k"][rows, h // group].double(), s["v"][rows, h // group].double()
            x = s["scale"] * (q @ k.T)
            seen = torch.ones(n, n, device="cuda", dtype=torch.bool).tril()
            if not back:
                x = torch.where(seen, x, -math.inf)
                smax[h] = torch.maximum(smax[h], x.max())
                lse[h, rows] = torch.logsumexp(x, -1)
                o[rows, h] = torch.exp(x - lse[h, rows, None]) @ v
                continue
            p = torch.exp(torch.where(seen, x - s["lse"][h, rows].double()[:, None], -math.inf))
            do = s["do"][rows, h].double()
            dv[rows, h // group] += p.T @ do
            p *= do @ v.T - torch.einsum("ic,ic->i", do, s["o"][rows, h].double())[:, None]
            dq[rows, h] = s["scale"] * (p @ k)
            dk[rows, h // group] += s["scale"] * (p.T @ q)
    return (dq, dk, dv) if back else (o, lse, smax)
