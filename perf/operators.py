"""The gradient operators of an attention block, as measured: attention's backward pass, the RMS norm
with the residual's addition (and e4m3 output), the norm's gradient and the rotary embedding's.

own = False runs them in plain torch (fp32, products and sums written out); own = True makes the calls
of muon_qk_clip_gb300 that a training step makes.  Inputs follow the repository's workloads: bf16
features of N(0, 1), one head in four with its queries scaled so that its softmax is nearly one-hot
(the heads QK-Clip is about), gradients of N(0, 1e-2).
"""
import math

import torch

own = False

E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -100
TILE = 128


# ------------------------------------------------------------------------------------------- cases
def listed():
    attn = dict(op="attention_backward")
    add = dict(op="add_rms_norm")
    back = dict(op="rms_norm_backward")
    rope = dict(op="rope_backward")
    return [
        # the tiny layer of the tests: a few CTAs' work, launch latency decides
        dict(name="attn_bwd_tiny", **attn, B=2, S=128, H=4, dh=64, dr=0, dv=64, causal=True),
        # the dense_block workload's attention layer, the ordinary training size
        dict(name="attn_bwd_dense_block", **attn, B=4, S=4096, H=16, dh=128, dr=0, dv=128, causal=True),
        # the k2_mla_layer workload: 64 heads, one rotary key shared by all of them
        dict(name="attn_bwd_mla_layer", **attn, B=1, S=4096, H=64, dh=128, dr=64, dv=128, causal=True),
        # long context (long_mla's length), two of its heads: what one rank of a head split holds
        dict(name="attn_bwd_mla_long", **attn, B=1, S=32768, H=2, dh=128, dr=64, dv=128, causal=True),
        # no mask, lengths and widths off every tile size: an encoder's ragged batch
        dict(name="attn_bwd_odd", **attn, B=3, S=1021, H=5, dh=80, dr=0, dv=48, causal=False),
        # pre-norm of a 7168-wide layer over 4096 tokens, stored in 8 bits for the expert products
        dict(name="add_norm_fp8_layer", **add, rows=4096, cols=7168, dtype="bf16", y="e4m3", residual=True, weight=True),
        # one decoded token of the same layer
        dict(name="add_norm_fp8_token", **add, rows=1, cols=7168, dtype="bf16", y="e4m3", residual=True, weight=True),
        # odd rows and columns in fp32, output in the inputs' type
        dict(name="add_norm_odd_fp32", **add, rows=3001, cols=1537, dtype="fp32", y="same", residual=True, weight=True),
        # gradient of dense_block's pre-norm with the residual stream's own gradient added
        dict(name="norm_bwd_block", **back, rows=16384, cols=2048, dtype="bf16", weight=True, dres=True),
        # gradient of the weightless norm of the MLA query latent, a short odd batch in fp32
        dict(name="norm_bwd_latent_fp32", **back, rows=777, cols=1536, dtype="fp32", weight=False, dres=False),
        # rotary columns of dQ, a strided view into [B, S, H, 192]
        dict(name="rope_bwd_queries", **rope, B=1, S=4096, nh=64, d=64, skip=128, dtype="bf16"),
        # gradient of the shared rotary key of a small batch
        dict(name="rope_bwd_shared_key", **rope, B=2, S=1001, nh=1, d=64, skip=0, dtype="fp32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention_backward", "attention_backward", "add_rms_norm", "rms_norm_backward", "rope_backward"])
    if op == "attention_backward":
        c = dict(op=op, B=rng.randint(1, 4), S=_log(rng, 1, 16384), H=rng.randint(1, 24))
        if rng.random() < 0.5:
            c.update(dh=rng.choice([64, 128]), dr=8 * rng.randint(1, 8), dv=8 * rng.randint(2, 16))
        else:
            c.update(dh=8 * rng.randint(2, 24), dr=0, dv=8 * rng.randint(2, 16))
        c["causal"] = rng.random() < 0.7
        most = 2 * 32768 ** 2 if c["causal"] else 32768 ** 2      # pairs of the largest listed case
        while c["B"] * c["H"] * c["S"] ** 2 > most // 2:
            if c["B"] > 1:
                c["B"] -= 1
            elif c["H"] > 1:
                c["H"] -= 1
            else:
                c["S"] //= 2
        return c
    if op in ("add_rms_norm", "rms_norm_backward"):
        cols = _log(rng, 16, 8192)
        if rng.random() < 0.6:
            cols = (cols + 15) // 16 * 16
        rows = min(_log(rng, 1, 32768), (4096 * 7168) // cols)
        c = dict(op=op, rows=rows, cols=cols, dtype=rng.choice(["bf16", "bf16", "fp32"]), weight=rng.random() < 0.7)
        if op == "add_rms_norm":
            c.update(y=rng.choice(["e4m3", "same"]), residual=rng.random() < 0.7)
        else:
            c.update(dres=rng.random() < 0.7)
        return c
    return dict(op=op, B=rng.randint(1, 4), S=_log(rng, 1, 8192), nh=rng.randint(1, 32), d=2 * rng.randint(4, 64),
                skip=8 * rng.randint(0, 16), dtype=rng.choice(["bf16", "fp32"]))


def work(c):
    es = 2 if c.get("dtype", "bf16") == "bf16" else 4
    if c["op"] == "attention_backward":
        rows, D = c["B"] * c["S"] * c["H"], c["dh"] + c["dr"]
        shared = c["B"] * c["S"] * c["dr"]
        pairs = c["B"] * c["H"] * (c["S"] * (c["S"] + 1) // 2 if c["causal"] else c["S"] ** 2)
        read = 2 * (rows * (D + c["dh"] + 3 * c["dv"]) + shared) + 4 * rows
        write = 2 * (rows * (D + c["dh"] + c["dv"]) + shared)
        return {"bytes": read + write, "flops": pairs * (6 * D + 4 * c["dv"])}
    if c["op"] == "rope_backward":
        n = c["B"] * c["S"] * c["nh"] * c["d"]
        return {"bytes": 2 * es * n, "flops": 3 * n}
    n = c["rows"] * c["cols"]
    if c["op"] == "add_rms_norm":
        planes = 2 * es if c["residual"] else 0                    # residual in, h out
        out = n + 4 * c["rows"] * -(-c["cols"] // TILE) if c["y"] == "e4m3" else es * n
        return {"bytes": n * (es + planes) + out + 4 * c["rows"] + es * c["cols"] * c["weight"], "flops": 6 * n}
    return {"bytes": n * es * (3 + c["dres"]) + 4 * c["rows"] + (es + 4) * c["cols"] * c["weight"], "flops": 9 * n}


# ------------------------------------------------------------------------------------------ inputs
def _dtype(c):
    return torch.bfloat16 if c.get("dtype", "bf16") == "bf16" else torch.float32


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=None):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype or _dtype(c))

    s = {"case": c}
    if c["op"] == "attention_backward":
        B, S, H, dh, dr, dv = (c[n] for n in ("B", "S", "H", "dh", "dr", "dv"))
        sharp = 1.0 + 11.0 * (torch.arange(H, device="cuda") % 4 == 1)
        s["q"] = (torch.randn(B, S, H, dh + dr, generator=g, device="cuda") * sharp[:, None]).to(torch.bfloat16)
        if dr:                                     # k^C and V are views of one projection, as project_mla gives them
            kv = normal(B, S, H, dh + dv)
            s["k"], s["v"], s["ks"] = kv[..., :dh], kv[..., dh:], normal(B, S, dr)
        else:
            s["k"], s["v"], s["ks"] = normal(B, S, H, dh), normal(B, S, H, dv), None
        s["do"] = normal(B, S, H, dv, std=1e-2)
        s["scale"] = 1.0 / math.sqrt(dh + dr)
        p, lse = _probabilities(s)
        s["lse"] = lse.contiguous()
        s["o"] = _weighted(p, s["v"].float()).to(torch.bfloat16).contiguous()
    elif c["op"] == "rope_backward":
        s["dy"] = normal(c["B"], c["S"], c["nh"], c["skip"] + c["d"], std=1e-2)[..., c["skip"]:]
    else:
        rows, cols = c["rows"], c["cols"]
        s["w"] = (1.0 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(_dtype(c)) if c["weight"] else None
        if c["op"] == "add_rms_norm":
            # a residual stream that has grown over the layers, with a few large channels
            loud = 1.0 + 20.0 * (torch.rand(cols, generator=g, device="cuda") < 0.005)
            s["x"] = normal(rows, cols)
            s["r"] = (3.0 * torch.randn(rows, cols, generator=g, device="cuda") * loud).to(_dtype(c)) if c["residual"] else None
        else:
            s["h"] = normal(rows, cols, std=3.0)
            s["rstd"] = torch.rsqrt(s["h"].float().square().mean(-1) + 1e-6)
            s["dy"] = normal(rows, cols, std=1e-2)
            s["dres"] = normal(rows, cols, std=1e-2) if c["dres"] else None
    return s


# -------------------------------------------------------------------------------------- plain forms
def _keys(s):
    k = s["k"].float()
    if s["ks"] is None:
        return k
    B, S, H, _ = k.shape
    return torch.cat([k, s["ks"].float()[:, :, None, :].expand(B, S, H, -1)], dim=-1)


def _heads_first(t):
    return t.permute(0, 2, 1, 3)


def _weighted(p, v):
    """sum_j p[b, h, i, j] v[b, j, h] as [B, S, H, d]"""
    return torch.matmul(p, _heads_first(v)).permute(0, 2, 1, 3)


def _logits(s):
    x = torch.matmul(_heads_first(s["q"].float()), _heads_first(_keys(s)).transpose(2, 3)).mul_(s["scale"])
    if s["case"]["causal"]:
        i = torch.arange(x.shape[-1], device=x.device)
        x.masked_fill_(i[None, :] > i[:, None], -math.inf)
    return x


def _probabilities(s):
    x = _logits(s)
    top = x.amax(-1, keepdim=True)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    return x.div_(total), (top + total.log())[..., 0]


def _plain_attention_backward(s):
    p = _logits(s).sub_(s["lse"][..., None]).exp_()
    do, q = s["do"].float(), s["q"].float()
    dv = _weighted(p.transpose(2, 3), do)
    ds = torch.matmul(_heads_first(do), _heads_first(s["v"].float()).transpose(2, 3))
    delta = (do * s["o"].float()).sum(-1).permute(0, 2, 1)
    ds.sub_(delta[..., None]).mul_(p)
    dq = _weighted(ds, _keys(s)) * s["scale"]
    dk = _weighted(ds.transpose(2, 3), q) * s["scale"]
    dh, t = s["case"]["dh"], torch.bfloat16
    dks = None if s["ks"] is None else dk[..., dh:].sum(2).to(t)
    return dq.to(t), dk[..., :dh].to(t), dv.to(t), dks


def _plain_add_rms_norm(s):
    c = s["case"]
    h = s["x"] if s["r"] is None else (s["x"].float() + s["r"].float()).to(s["x"].dtype)
    f = h.float()
    rstd = 1.0 / torch.sqrt((f * f).mean(-1) + 1e-6)
    y = f * rstd[:, None]
    if s["w"] is not None:
        y = y * s["w"].float()
    if c["y"] == "same":
        return y.to(h.dtype), None, h, rstd
    rows, cols = y.shape
    tiles = -(-cols // TILE)
    y = torch.nn.functional.pad(y, (0, tiles * TILE - cols)).view(rows, tiles, TILE)
    scale = (y.abs().amax(-1) / E4M3_MAX).clamp(min=SCALE_MIN)
    y = (y / scale[..., None]).view(rows, tiles * TILE)[:, :cols]
    return y.to(torch.float8_e4m3fn), scale, h, rstd


def _plain_rms_norm_backward(s):
    xhat = s["h"].float() * s["rstd"][:, None]
    dy = s["dy"].float()
    gr = dy if s["w"] is None else dy * s["w"].float()
    dx = (gr - xhat * (gr * xhat).mean(-1, keepdim=True)) * s["rstd"][:, None]
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    dw = None if s["w"] is None else (dy * xhat).sum(0)
    return dx.to(s["h"].dtype), dw


def _plain_rope_backward(s):
    dy = s["dy"].float()
    _, S, _, d = dy.shape
    freq = 10000.0 ** (-torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d)
    angle = torch.arange(S, device="cuda", dtype=torch.float64)[:, None] * freq
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    a, b = dy[..., 0::2], dy[..., 1::2]
    return torch.stack([a * cos + b * sin, b * cos - a * sin], dim=-1).flatten(-2).to(s["dy"].dtype)


# --------------------------------------------------------------------------------------------- run
def run(s):
    op = s["case"]["op"]
    if not own:
        return {"attention_backward": _plain_attention_backward, "add_rms_norm": _plain_add_rms_norm,
                "rms_norm_backward": _plain_rms_norm_backward, "rope_backward": _plain_rope_backward}[op](s)
    from muon_qk_clip_gb300 import binding as mc
    if op == "attention_backward":
        return mc.qk_attention_backward(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], k_shared=s["ks"],
                                        causal=s["case"]["causal"], scale=s["scale"])
    if op == "add_rms_norm":
        out = torch.float8_e4m3fn if s["case"]["y"] == "e4m3" else None
        return mc.add_rms_norm(s["x"], s["r"], s["w"], eps=1e-6, out_dtype=out)
    if op == "rms_norm_backward":
        return mc.rms_norm_backward(s["dy"], s["h"], s["rstd"], weight=s["w"], dres=s["dres"])
    return mc.rope_backward(s["dy"], theta=10000.0)


# ------------------------------------------------------------------------------------------- exact
def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "attention_backward":
        return _exact_attention(c, s)
    if c["op"] == "rope_backward":
        z = torch.view_as_complex(s["dy"].double().unflatten(-1, (-1, 2)).contiguous())
        k = torch.arange(c["d"] // 2, device="cuda", dtype=torch.float64)
        angle = torch.outer(torch.arange(c["S"], device="cuda", dtype=torch.float64),
                            torch.exp(-2.0 * k / c["d"] * math.log(10000.0)))
        z = z * torch.polar(torch.ones_like(angle), -angle)[None, :, None, :]
        return torch.view_as_real(z).flatten(-2)
    w = 1.0 if s["w"] is None else s["w"].double()
    if c["op"] == "add_rms_norm":
        # the stored sum is a rounding by definition; everything after it is in 64 bits
        h = s["x"] if s["r"] is None else (s["x"].double() + s["r"].double()).to(s["x"].dtype)
        d = h.double()
        rstd = (d.pow(2).sum(-1) / c["cols"] + 1e-6).pow(-0.5)
        y = torch.einsum("rc,r->rc", d, rstd) * w
        if c["y"] == "same":
            return y, None, d, rstd
        parts, scales = [], []
        for part in y.split(TILE, dim=-1):
            scale = torch.clamp(part.abs().max(-1).values / E4M3_MAX, min=SCALE_MIN)
            parts.append(_to_e4m3(part / scale[:, None]))
            scales.append(scale)
        return torch.cat(parts, -1), torch.stack(scales, -1), d, rstd
    d, r, dy = s["h"].double(), s["rstd"].double(), s["dy"].double()
    inner = torch.einsum("rc,rc,r->r", dy * w, d, r) / c["cols"]
    dx = (dy * w) * r[:, None] - d * (r * r * inner)[:, None]
    if s["dres"] is not None:
        dx = dx + s["dres"].double()
    return dx, None if s["w"] is None else torch.einsum("rc,rc,r->c", dy, d, r)


def _to_e4m3(x):
    """The e4m3 value nearest to x, ties to even: 4 significand bits, quanta of 2^-9 below 2^-6."""
    e = torch.frexp(x)[1].clamp(min=-5) - 4
    quantum = torch.ldexp(torch.ones_like(x), e)
    return (torch.round(x / quantum) * quantum).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_attention(c, s):
    B, S, H, dh, dr, dv = (c[n] for n in ("B", "S", "H", "dh", "dr", "dv"))
    new = lambda *shape: torch.zeros(*shape, device="cuda", dtype=torch.float64)  # noqa: E731
    dq, dk, dvv = new(B, S, H, dh + dr), new(B, S, H, dh), new(B, S, H, dv)
    dks = new(B, S, dr) if dr else None
    for b in range(B):
        for h in range(H):
            q, v, do = (s[n][b, :, h].double() for n in ("q", "v", "do"))
            k = s["k"][b, :, h].double()
            if dr:
                k = torch.cat([k, s["ks"][b].double()], -1)
            p = torch.exp(s["scale"] * (q @ k.T) - s["lse"][b, h].double()[:, None])
            if c["causal"]:
                p = p.tril()
            dvv[b, :, h] = p.T @ do
            p *= do @ v.T - torch.einsum("ic,ic->i", do, s["o"][b, :, h].double())[:, None]
            dq[b, :, h] = s["scale"] * (p @ k)
            full = s["scale"] * (p.T @ q)
            dk[b, :, h] = full[:, :dh]
            if dr:
                dks[b] += full[:, dh:]
    return dq, dk, dvv, dks
