"""Host-only checks of the gradient calls: every refusal happens before a launch
(fake, aligned device addresses that are never dereferenced)."""
import ctypes

import pytest
import torch

from muon_qk_clip_gb300 import abi
from muon_qk_clip_gb300 import binding as mc
from muon_qk_clip_gb300.abi import McAttnDesc, McAttnGrad

STEP = 1 << 32
FAKE = 0x7f0000000000
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from muon_qk_clip_gb300 import build
    build.build()
    return abi.load()


ROWS = [16 * 2 * 64, 2 * 64, 64]           # [B, S = 16, H = 2, 64], contiguous


def attn(**kw):
    d = McAttnDesc()
    d.B, d.S, d.H, d.d_head, d.d_shared, d.dtype, d.causal = 2, 16, 2, 64, 0, abi.MC_BF16, 1
    d.scale = 0.125
    d.q, d.k = FAKE, FAKE + STEP
    d.q_strides[:] = ROWS
    d.k_strides[:] = ROWS
    for k, v in kw.items():
        if k.endswith("strides"):
            getattr(d, k)[:] = v
        else:
            setattr(d, k, v)
    return d


def grad(**kw):
    g = McAttnGrad()
    for n, name in enumerate(("v", "o", "d_o", "dq", "dk", "dv")):
        setattr(g, name, FAKE + (2 + n) * STEP)
    g.lse = FAKE + 10 * STEP
    g.d_v = 64
    for name in ("v", "o", "do", "dq", "dk", "dv"):
        getattr(g, name + "_strides")[:] = ROWS
    g.dq_strides[:] = [2 * x for x in ROWS]          # room for a shared part
    for k, v in kw.items():
        if k.endswith("strides"):
            getattr(g, k)[:] = v
        else:
            setattr(g, k, v)
    return g


def call(lib, d, g, workspace=FAKE + 20 * STEP, nbytes=1 << 40):
    return lib.qk_attention_backward(ctypes.byref(d), ctypes.byref(g), P(workspace), nbytes, None, None)


INV, UNS, WS = abi.MC_ERR_INVALID_ARG, abi.MC_ERR_UNSUPPORTED, abi.MC_ERR_WORKSPACE


@pytest.mark.parametrize("dkw,gkw,code,needle", [
    (dict(S=0), {}, INV, "S"),
    (dict(H=0), {}, INV, "H"),
    (dict(dtype=abi.MC_F32), {}, UNS, "bf16"),
    (dict(dtype=7), {}, INV, "dtype"),
    (dict(scale=0.0), {}, INV, "scale"),
    (dict(scale=float("nan")), {}, INV, "scale"),
    (dict(d_head=256), {}, UNS, "q.k length"),
    (dict(d_head=8), {}, UNS, "q.k length"),
    (dict(d_head=96, d_shared=64, k_shared=FAKE + 8 * STEP), {}, UNS, "multiple of 64"),
    (dict(d_shared=64), {}, INV, "k_shared is null"),
    (dict(d_shared=64, k_shared=FAKE + 8 * STEP, ks_strides=[1024, 64]), {}, INV, "dk_shared is null"),
    (dict(q=None), {}, INV, "q is null"),
    (dict(S=(1 << 30) + 1), {}, UNS, "too large"),
    (dict(k=FAKE + STEP + 8), {}, UNS, "k must be 16-byte"),
    (dict(q_strides=[2048, 132, 64]), {}, UNS, "multiples of 8"),
    (dict(k_strides=[2048, -128, 64]), {}, INV, "negative"),
    ({}, dict(d_v=256), UNS, "d_v"),
    ({}, dict(d_v=8), UNS, "d_v"),
    ({}, dict(v=None), INV, "v is null"),
    ({}, dict(d_o=None), INV, "d_o is null"),
    ({}, dict(lse=None), INV, "lse"),
    ({}, dict(lse=FAKE + 2), INV, "lse"),
    ({}, dict(dv=FAKE + 7 * STEP + 2), UNS, "dv must be 16-byte"),
    ({}, dict(dk_strides=[2048, 128, 0]), INV, "dk share"),          # a broadcast output
    ({}, dict(dq_strides=[2048, 64, 64]), INV, "dq share"),          # heads over tokens
    ({}, dict(dq_strides=[2048, 64, 1024 - 64]), INV, "dq share"),
    ({}, dict(dq=FAKE), INV, "dq overlaps q"),                       # in place over the queries
    ({}, dict(dk=FAKE + 2 * STEP + 256), INV, "dk overlaps v"),
    ({}, dict(dk=FAKE + 5 * STEP), INV, "same memory"),
])
def test_attention_backward_refuses(lib, dkw, gkw, code, needle):
    assert call(lib, attn(**dkw), grad(**gkw)) == code
    assert needle in lib.mc_last_error().decode()


DQ, DK, DV, LSE, WSP = (FAKE + n * STEP for n in (5, 6, 7, 10, 20))
KV = [16 * 2 * 128, 2 * 128, 128]          # [B, S, H, 64 + 64]
BHSD = [2 * 16 * 64, 64, 16 * 64]          # heads outside the sequence


@pytest.mark.parametrize("gkw,needle", [
    (dict(dv=DK + 16), "dk and dv share"),                           # an overlap that does not begin together
    (dict(dv=DK + 64, dk_strides=KV, dv_strides=KV), "dk and dv share"),
    (dict(dv=DK + 128, dk_strides=KV, dv_strides=[16 * 2 * 128, 2 * 128, 64]), "dk and dv share"),
    (dict(dv=DK + 128, dk_strides=KV, dv_strides=[16 * 2 * 128, 128, 16 * 128]), "dk and dv share"),
    (dict(dv=DK + 256 - 32, dk_strides=KV, dv_strides=KV), "dk and dv share"),        # into the next head's dk
    (dict(dk=LSE + 64), "dk overlaps lse"),
    (dict(lse=WSP + 64), "lse, status and workspace"),
    (dict(dv=WSP - 16), "workspace overlaps dv"),
    (dict(v=WSP + 256), "workspace overlaps v"),
    (dict(q_strides=[1 << 36, 1 << 36, 64], S=1 << 20), "too large"),
])
def test_attention_backward_refuses_shared_memory(lib, gkw, needle):
    d = attn(**{k: gkw.pop(k) for k in ("q_strides", "S") if k in gkw})
    assert call(lib, d, grad(**gkw)) in (INV, UNS)
    assert needle in lib.mc_last_error().decode()


@pytest.mark.parametrize("gkw", [
    dict(dv=DK + 128, dk_strides=KV, dv_strides=KV),                                  # [B, S, H, dk | dv]
    dict(dk=DV + 128, dk_strides=KV, dv_strides=KV),
    dict(dv=DK + 2 * 64 * 2, dk_strides=[16 * 256, 256, 64], dv_strides=[16 * 256, 256, 64]),   # [B, S, 2, H, 64]
    dict(dv=DK + 16 * 64 * 2, dk_strides=[4096, 64, 2048], dv_strides=[4096, 64, 2048]),        # [B, H, 2, S, 64]
    dict(dv=DK + 2 * 2048 * 2, dk_strides=BHSD, dv_strides=BHSD),                     # one after the other
])
def test_attention_backward_takes_outputs_that_interleave(lib, gkw):
    """These pass the checks of memory: the next refusal, of the workspace's size, is the one that is met."""
    assert call(lib, attn(), grad(**gkw), nbytes=0) == WS


@pytest.mark.parametrize("status,needle", [
    (FAKE + 20 * STEP + 64, "lse, status and workspace"), (LSE + 8, "lse, status and workspace"),
    (FAKE + 4 * STEP + 4, "status overlaps d_o"), (DQ + 4, "status overlaps dq"), (FAKE + 30 * STEP + 2, "4-byte")])
def test_attention_backward_refuses_a_status_among_its_operands(lib, status, needle):
    d, g = attn(), grad()
    assert lib.qk_attention_backward(ctypes.byref(d), ctypes.byref(g), P(WSP), 1 << 40, P(status), None) == INV
    assert needle in lib.mc_last_error().decode()


def test_attention_backward_workspace(lib):
    n, d = ctypes.c_size_t(0), attn()
    assert lib.qk_attention_backward_workspace_size(ctypes.byref(d), ctypes.byref(n)) == abi.MC_OK
    assert n.value >= 2 * 4 * 2 * 2 * 16
    assert call(lib, d, grad(), nbytes=n.value - 1) == WS
    assert call(lib, d, grad(), workspace=FAKE + 20 * STEP + 16) == WS
    assert call(lib, d, grad(), workspace=None) == WS
    m = ctypes.c_size_t(0)
    shared = attn(d_shared=64)
    assert lib.qk_attention_backward_workspace_size(ctypes.byref(shared), ctypes.byref(m)) == abi.MC_OK
    assert m.value >= n.value + 4 * 2 * 2 * 16 * 64
    assert lib.qk_attention_backward_workspace_size(ctypes.byref(attn(S=0)), ctypes.byref(n)) == INV
    assert lib.qk_attention_backward_workspace_size(ctypes.byref(d), None) == INV


@pytest.mark.parametrize("kw", [dict(d_head=8), dict(d_head=200), dict(d_shared=192),
                                dict(B=1 << 10, S=1 << 20, H=1 << 10, d_shared=(1 << 31) - 1)])   # would overflow
def test_attention_backward_workspace_of_unsupported_widths(lib, kw):
    n = ctypes.c_size_t(0)
    assert lib.qk_attention_backward_workspace_size(ctypes.byref(attn(**kw)), ctypes.byref(n)) == UNS
    assert n.value == 0 and "q.k length" in lib.mc_last_error().decode()


def test_binding_refuses_host_tensors_and_shapes():
    x = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        mc.qk_attention_backward(x, x, x, x, torch.zeros(1, 2, 4), x)


def test_grad_struct_layout(tmp_path):
    import os
    import subprocess
    header = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "muonclip.h")
    src = tmp_path / "l.c"
    src.write_text(f'#include <stdio.h>\n#include <stddef.h>\n#include "{header}"\nint main(void) {{'
                   'printf("%zu %zu %zu %zu", sizeof(mc_attn_grad), offsetof(mc_attn_grad, lse),'
                   'offsetof(mc_attn_grad, dk_shared), offsetof(mc_attn_grad, dv)); return 0; }')
    subprocess.run(["gcc", "-std=c99", str(src), "-o", str(tmp_path / "l")], check=True)
    got = subprocess.run([str(tmp_path / "l")], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in got] == [ctypes.sizeof(McAttnGrad), McAttnGrad.lse.offset, McAttnGrad.dk_shared.offset,
                                     McAttnGrad.dv.offset]


# ------------------------------------------------------------- norms and the rotary gradient
X, R, H, Y, SC, RS, WT = (P(FAKE + i * STEP) for i in range(7))
BF, F32, F8 = abi.MC_BF16, abi.MC_F32, abi.MC_F8E4M3


def add(**kw):
    a = dict(x=X, ldx=256, r=R, ldr=256, w=WT, h=H, ldh=256, y=Y, ldy=256, sc=None, lds=0, rs=RS, rows=4, cols=256,
             dt=BF, yt=BF, eps=1e-6, stream=None)
    a.update(kw)
    return tuple(a.values())


@pytest.mark.parametrize("kw,needle", [
    (dict(dt=5), "dtype 5"),
    (dict(yt=F32), "y_dtype"),
    (dict(yt=F8), "scales"),
    (dict(sc=SC, lds=2), "scales"),
    (dict(yt=F8, sc=SC, lds=1), "pitch"),
    (dict(rows=-1), "rows -1"),
    (dict(cols=0), "cols 0"),
    (dict(ldx=255), "pitch"),
    (dict(ldh=100), "pitch"),
    (dict(eps=-1.0), "eps"),
    (dict(eps=float("inf")), "eps"),
    (dict(h=None), "together"),
    (dict(r=None), "together"),
    (dict(x=None), "null"),
    (dict(y=None), "null"),
    (dict(x=P(FAKE + 1)), "aligned"),
    (dict(rs=P(FAKE + 5 * STEP + 2)), "aligned"),
    (dict(y=H), "h overlaps y"),
    (dict(h=P(FAKE + 512)), "h overlaps x"),                # another row of x
    (dict(h=X, ldh=512), "h overlaps x"),                   # x's memory at another pitch
    (dict(y=WT), "y overlaps weight"),
    (dict(yt=F8, sc=SC, lds=2, y=X), "y overlaps x"),       # 8-bit rows over wider ones
    (dict(rs=P(FAKE + 4)), "rstd overlaps x"),
])
def test_add_rms_norm_refuses(lib, kw, needle):
    assert lib.mc_add_rms_norm(*add(**kw)) == INV
    assert needle in lib.mc_last_error().decode()


def test_norm_calls_on_no_rows_launch_nothing(lib):
    assert lib.mc_add_rms_norm(*add(rows=0)) == abi.MC_OK
    assert lib.mc_rms_norm_backward(*back(rows=0, dw=None)) == abi.MC_OK


def back(**kw):
    a = dict(dy=X, lddy=256, h=R, ldh=256, rs=RS, w=WT, dres=H, ldr=256, dx=Y, lddx=256, dw=SC, rows=4, cols=256, dt=BF,
             ws=P(FAKE + 8 * STEP), n=1 << 30, stream=None)
    a.update(kw)
    return tuple(a.values())


@pytest.mark.parametrize("kw,code,needle", [
    (dict(dt=F8), INV, "dtype"),
    (dict(rows=-2), INV, "rows -2"),
    (dict(cols=-1), INV, "cols -1"),
    (dict(lddy=10), INV, "pitch"),
    (dict(ldr=10), INV, "pitch"),
    (dict(dy=None), INV, "null"),
    (dict(rs=None), INV, "null"),
    (dict(dx=None), INV, "null"),
    (dict(h=P(FAKE + STEP + 1)), INV, "aligned"),
    (dict(dw=P(FAKE + 3)), INV, "aligned"),
    (dict(ws=None), WS, "workspace"),
    (dict(n=304 * 256 * 4 - 1), WS, "workspace"),
    (dict(ws=P(FAKE + 8 * STEP + 8)), WS, "workspace"),
    (dict(dx=P(FAKE + 512)), INV, "dx overlaps dy"),
    (dict(dx=R, lddx=512), INV, "dx overlaps h"),
    (dict(dw=RS), INV, "dweight overlaps rstd"),
    (dict(ws=X), INV, "workspace overlaps dy"),
])
def test_rms_norm_backward_refuses(lib, kw, code, needle):
    assert lib.mc_rms_norm_backward(*back(**kw)) == code
    assert needle in lib.mc_last_error().decode()


def test_rms_norm_backward_workspace_size(lib):
    n = ctypes.c_size_t(0)
    assert lib.mc_rms_norm_backward_workspace_size(256, ctypes.byref(n)) == abi.MC_OK and n.value == 304 * 256 * 4
    assert lib.mc_rms_norm_backward_workspace_size(0, ctypes.byref(n)) == INV
    assert lib.mc_rms_norm_backward_workspace_size(256, None) == INV


def rope(**kw):
    a = dict(dy=X, yb=8192, ys=1024, yh=64, dx=Y, xb=8192, xs=1024, xh=64, B=2, S=8, nh=16, d=64, dt=BF, theta=1e4,
             stream=None)
    a.update(kw)
    return tuple(a.values())


@pytest.mark.parametrize("kw,needle", [
    (dict(dt=F8), "dtype"),
    (dict(d=63), "d 63"),
    (dict(d=0), "d 0"),
    (dict(d=8192), "d 8192"),
    (dict(nh=0), "heads 0"),
    (dict(S=-1), "S -1"),
    (dict(theta=0.0), "theta"),
    (dict(theta=float("inf")), "theta"),
    (dict(dy=None), "null"),
    (dict(dx=None), "null"),
    (dict(dx=P(FAKE + 3 * STEP + 1)), "aligned"),
    (dict(ys=-1024), "negative"),
    (dict(xh=0), "share"),
    (dict(xs=512), "share"),
    (dict(dx=P(FAKE + 64)), "overlaps"),
    (dict(dx=X, xs=2048, xb=16384), "overlaps"),            # in place with other strides
])
def test_rope_backward_refuses(lib, kw, needle):
    assert lib.mc_rope_backward(*rope(**kw)) == INV
    assert needle in lib.mc_last_error().decode()


@pytest.mark.parametrize("kw", [
    dict(B=1, S=(1 << 24) + 1, nh=1, d=2, ys=2, xs=2),      # a position that fp32 does not hold
    dict(theta=1e-7),                                       # 8 positions of up to 1e7 radians each
    dict(theta=1e-300)])
def test_rope_backward_refuses_angles_that_it_cannot_hold(lib, kw):
    assert lib.mc_rope_backward(*rope(**kw)) == UNS
    assert "angles" in lib.mc_last_error().decode()


def test_rope_backward_of_nothing_is_a_no_op(lib):
    assert lib.mc_rope_backward(*rope(B=0, dy=None, dx=None)) == abi.MC_OK


def test_norm_bindings_refuse_host_tensors():
    x = torch.zeros(2, 8)
    for call in (lambda: mc.add_rms_norm(x), lambda: mc.rms_norm_backward(x, x, x[:, 0].contiguous()),
                 lambda: mc.rope_backward(torch.zeros(1, 2, 8))):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_packed_descriptors_match_the_structures():
    """The binding packs the attention descriptors by format: every field arrives."""
    assert mc._ATTN_DESC.size == ctypes.sizeof(McAttnDesc) and mc._ATTN_GRAD.size == ctypes.sizeof(McAttnGrad)
    d = McAttnDesc.from_buffer_copy(mc._ATTN_DESC.pack(*range(1, 8), 0.5, *range(9, 20)))
    assert [d.B, d.S, d.H, d.d_head, d.d_shared, d.dtype, d.causal, d.scale] == [1, 2, 3, 4, 5, 6, 7, 0.5]
    assert [d.q, d.k, d.k_shared, *d.q_strides, *d.k_strides, *d.ks_strides] == list(range(9, 20))
    n = len(mc._ATTN_GRAD.unpack(bytes(mc._ATTN_GRAD.size)))
    g = McAttnGrad.from_buffer_copy(mc._ATTN_GRAD.pack(*range(1, n + 1)))
    flat = []
    for name, _ in McAttnGrad._fields_:
        x = getattr(g, name)
        flat += list(x) if hasattr(x, "__len__") else [x]
    assert flat == list(range(1, n + 1))


def test_products_refuse_rows_that_share_memory():
    """Broadcast rows would be read past their storage."""
    x, w = torch.zeros(1, 8).expand(4, 8), torch.zeros(3, 8)
    for call in (lambda: mc.matmul(x, w), lambda: mc.matmul(w, x), lambda: mc.rms_norm(x)):
        with pytest.raises(ValueError, match="share memory"):
            call()


def test_descriptor_scale_beyond_fp32_is_left_to_the_library(lib):
    x = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    d = mc.attn_desc(x, x, scale=1e300)
    assert d.scale == float("inf")
    d.q, d.k = FAKE, FAKE + STEP
    assert call(lib, d, grad()) == INV and "scale" in lib.mc_last_error().decode()


def test_projections_run_on_their_tensors_device():
    """The projections and their gradients launch on the device that their tensors
    are on, whichever is current, and refuse tensors of several devices."""
    from types import SimpleNamespace

    from muon_qk_clip_gb300 import forward
    on = lambda name: SimpleNamespace(device=torch.device(name))  # noqa: E731
    assert forward._on_device(on("cuda:1"), on("cuda:1")).idx == 1
    with pytest.raises(ValueError, match="one device"):
        forward._on_device(on("cuda:0"), on("cuda:1"))
    with pytest.raises(ValueError, match="device tensors"):
        forward._on_device(on("cuda:0"), on("cpu"))
