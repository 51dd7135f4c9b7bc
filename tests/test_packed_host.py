"""Host-only checks of the packed attention, the head norms and AdamW: every refusal
happens before a launch (fake, aligned device addresses that are never dereferenced)."""
import ctypes
import os
import subprocess

import pytest
import torch

from muon_qk_clip_gb300 import abi
from muon_qk_clip_gb300 import binding as mc
from muon_qk_clip_gb300.abi import McAdamHparams, McAdamTensor, McHeads, McPackedDesc, McPackedGrad

STEP = 1 << 32
FAKE = 0x7f0000000000
P = ctypes.c_void_p
INV, UNS, WS = abi.MC_ERR_INVALID_ARG, abi.MC_ERR_UNSUPPORTED, abi.MC_ERR_WORKSPACE
BF, F32, F8 = abi.MC_BF16, abi.MC_F32, abi.MC_F8E4M3
Q, K, V, O, DO, DQ, DK, DV, LSE, SMAX, WSP, OFF, STATUS = (FAKE + i * STEP for i in range(13))


@pytest.fixture(scope="module")
def lib():
    from muon_qk_clip_gb300 import build
    build.build()
    return abi.load()


def fill(s, kw):
    for k, v in kw.items():
        if k.endswith("strides"):
            getattr(s, k)[:] = v
        else:
            assert hasattr(s, k)
            setattr(s, k, v)
    return s


QS, KS = [4 * 64, 64], [2 * 64, 64]           # [T = 64, H = 4, 64] and [T, H_kv = 2, 64], contiguous


def packed(**kw):
    d = McPackedDesc(64, 3, 4, 2, 64, 64, BF, 0.125, OFF, Q, K, V)
    return fill(fill(d, dict(q_strides=QS, k_strides=KS, v_strides=KS)), kw)


def grads(**kw):
    g = McPackedGrad(o=O, lse=LSE, d_o=DO, dq=DQ, dk=DK, dv=DV)
    return fill(fill(g, dict(o_strides=QS, do_strides=QS, dq_strides=QS, dk_strides=KS, dv_strides=KS)), kw)


def forward(lib, d, o=O, os=QS, lse=LSE, smax=SMAX, ws=WSP, nbytes=1 << 40, status=None):
    return lib.qk_attention_packed_forward(d, o, (ctypes.c_int64 * 2)(*os), lse, smax, 0, ws, nbytes, status, None)


def backward(lib, d, g, ws=WSP, nbytes=1 << 40, status=None):
    return lib.qk_attention_packed_backward(d, g, ws, nbytes, status, None)


SHAPES = [
    (dict(T=-1), INV, "T -1"), (dict(nseq=0), INV, "nseq 0"), (dict(H=0), INV, "H 0"), (dict(H_kv=0), INV, "H_kv 0"),
    (dict(H_kv=3), INV, "multiple"), (dict(dtype=F32), UNS, "bf16"), (dict(dtype=F8), INV, "dtype"),
    (dict(d=8), UNS, "widths"), (dict(d=144), UNS, "widths"), (dict(d_v=8), UNS, "widths"), (dict(d_v=256), UNS, "widths"),
    (dict(T=(1 << 30) + 1), UNS, "too large"), (dict(nseq=(1 << 22) + 1), UNS, "too large"),
    (dict(H=1 << 17, H_kv=1), UNS, "too large"), (dict(T=1 << 30, H=1 << 10), UNS, "too large")]
LAYOUTS = [
    (dict(scale=0.0), INV, "scale"), (dict(scale=float("inf")), INV, "scale"), (dict(scale=float("nan")), INV, "scale"),
    (dict(offsets=None), INV, "offsets"), (dict(offsets=OFF + 2), INV, "offsets"), (dict(q=None), INV, "q"),
    (dict(k=K + 8), UNS, "k"), (dict(v=None), INV, "v"), (dict(q_strides=[257, 64]), UNS, "q"),
    (dict(k_strides=[-128, 64]), INV, "k"), (dict(v_strides=[1 << 34, 64]), UNS, "too large")]


@pytest.mark.parametrize("kw,code,needle", SHAPES + LAYOUTS)
def test_packed_attention_refuses(lib, kw, code, needle):
    for call in (lambda: forward(lib, packed(**kw)), lambda: backward(lib, packed(**kw), grads())):
        assert call() == code and needle in lib.mc_last_error().decode()


@pytest.mark.parametrize("kw", [kw for kw, _, _ in SHAPES])
def test_packed_workspace_size_refuses(lib, kw):
    n = ctypes.c_size_t(0)
    for back in (0, 1):
        assert lib.qk_attention_packed_workspace_size(packed(**kw), back, n) in (INV, UNS)


@pytest.mark.parametrize("kw,needle", [
    (dict(smax=None), "smax"), (dict(smax=SMAX + 2), "4-byte"), (dict(lse=LSE + 1), "4-byte"), (dict(status=STATUS + 2), "4-byte"),
    (dict(o=None), "o"), (dict(o=O + 2), "o"), (dict(os=[256, 32]), "o"), (dict(os=[0, 64]), "o"), (dict(o=Q), "o overlaps q"),
    (dict(o=K + 16), "o overlaps k"), (dict(lse=V + 4), "lse overlaps v"), (dict(smax=OFF + 8), "smax overlaps offsets"),
    (dict(smax=LSE + 1020), "overlaps"), (dict(status=SMAX + 4), "overlaps"), (dict(status=WSP + 4), "overlaps"),
    (dict(lse=WSP + 256), "overlaps")])
def test_packed_forward_refuses_outputs(lib, kw, needle):
    assert forward(lib, packed(), **kw) == (UNS if kw == dict(o=O + 2) else INV) and needle in lib.mc_last_error().decode()


@pytest.mark.parametrize("kw,needle", [
    (dict(lse=None), "lse"), (dict(lse=LSE + 2), "4-byte"), (dict(o=None), "o"), (dict(d_o=DO + 4), "d_o"), (dict(dq=None), "dq"),
    (dict(dk=DK + 2), "dk"), (dict(dv_strides=[128, 32]), "dv"), (dict(dq=Q), "dq overlaps q"), (dict(dq=DO), "dq overlaps d_o"),
    (dict(dk=DV), "overlaps"), (dict(dk=DQ + 64), "overlaps"), (dict(dv=LSE + 16), "dv overlaps lse")])
def test_packed_backward_refuses_operands(lib, kw, needle):
    code = UNS if kw in (dict(d_o=DO + 4), dict(dk=DK + 2)) else INV          # 16-byte alignment
    assert backward(lib, packed(), grads(**kw)) == code and needle in lib.mc_last_error().decode()


@pytest.mark.parametrize("kw", [
    dict(dk=DQ + 512, dv=DQ + 768, dq_strides=[512, 64], dk_strides=[512, 64], dv_strides=[512, 64]),   # [T, q | k | v heads]
    dict(dv=DK + 128, dk_strides=[256, 128], dv_strides=[256, 128])])                                   # [T, G, dk | dv]
def test_packed_backward_takes_outputs_that_interleave(lib, kw):
    """These pass the checks of memory: the next refusal, of the workspace's size, is met."""
    assert backward(lib, packed(), grads(**kw), nbytes=0) == WS


def test_packed_workspace(lib):
    n, m = ctypes.c_size_t(0), ctypes.c_size_t(0)
    assert lib.qk_attention_packed_workspace_size(packed(), 0, n) == abi.MC_OK
    assert lib.qk_attention_packed_workspace_size(packed(), 1, m) == abi.MC_OK
    assert m.value >= n.value + 2 * 4 * 64 * 4
    assert lib.qk_attention_packed_workspace_size(packed(), 0, None) == INV
    assert lib.qk_attention_packed_workspace_size(None, 0, n) == INV
    for call in (lambda **kw: forward(lib, packed(), **kw), lambda **kw: backward(lib, packed(), grads(), **kw)):
        for kw in (dict(nbytes=n.value - 1), dict(ws=None), dict(ws=WSP + 64)):
            assert call(**kw) == WS
    assert backward(lib, packed(), grads(), nbytes=m.value - 1) == WS
    assert forward(lib, None) == INV and backward(lib, packed(), None) == INV


# ------------------------------------------------------------------ head norms
X, Y, WQ, WK, XO, YO, RSTD, GX, GY, DWQ, DWK = (FAKE + (20 + i) * STEP for i in range(11))


def heads(**kw):
    return fill(McHeads(16, 4, 2, 64, 64, BF, 1e-6, 1e4, None), kw)


def norm(lib, h, q=X, qt=256, qh=64, k=Y, kt=128, kh=64, wq=WQ, wk=WK, oq=XO, oqt=256, oqh=64, ok=YO, okt=128, okh=64, rstd=RSTD):
    return lib.mc_head_norm_rope(h, q, qt, qh, k, kt, kh, wq, wk, oq, oqt, oqh, ok, okt, okh, rstd, None)


def norm_grad(lib, h, dyq=GX, dyk=GY, q=X, k=Y, rstd=RSTD, wq=WQ, wk=WK, dq=XO, dqt=256, dqh=64, dk=YO, dkt=128, dkh=64,
              dwq=DWQ, dwk=DWK, ws=WSP, nbytes=1 << 40):
    return lib.mc_head_norm_rope_backward(h, dyq, 256, 64, dyk, 128, 64, q, 256, 64, k, 128, 64, rstd, wq, wk, dq, dqt, dqh,
                                          dk, dkt, dkh, dwq, dwk, ws, nbytes, None)


@pytest.mark.parametrize("kw,code,needle", [
    (dict(T=-1), INV, "T -1"), (dict(heads_q=0), INV, "heads 0"), (dict(heads_k=-1), INV, "heads"), (dict(d=0), INV, "d 0"),
    (dict(d=63), INV, "d 63"), (dict(d=258), INV, "d 258"), (dict(rot=-2), INV, "rot"), (dict(rot=31), INV, "rot"),
    (dict(rot=66), INV, "rot"), (dict(dtype=F8), INV, "dtype"), (dict(eps=-1.0), INV, "eps"), (dict(eps=float("nan")), INV, "eps"),
    (dict(theta=0.0), INV, "theta"), (dict(theta=float("inf")), INV, "theta"), (dict(theta=1e-7), UNS, "theta"),
    (dict(T=1 << 40), UNS, "too large"), (dict(positions=FAKE + 2), INV, "positions")])
def test_head_norm_refuses_shapes(lib, kw, code, needle):
    for call in (norm, norm_grad):
        assert call(lib, heads(**kw)) == code and needle in lib.mc_last_error().decode()


@pytest.mark.parametrize("kw,code,needle", [
    (dict(q=None), INV, "null"), (dict(k=None), INV, "null"), (dict(oq=None), INV, "null"), (dict(ok=None), INV, "null"),
    (dict(rstd=None), INV, "null"), (dict(q=X + 1), INV, "aligned"), (dict(wk=WK + 1), INV, "aligned"), (dict(rstd=RSTD + 2), INV, "aligned"),
    (dict(qt=-256), INV, "negative"), (dict(kh=1 << 50), UNS, "too large"), (dict(oqt=64), INV, "share addresses"),
    (dict(okh=0), INV, "share addresses"), (dict(oq=X, oqt=512), INV, "overlaps"), (dict(oq=X + 2), INV, "overlaps"),
    (dict(oq=Y), INV, "overlaps"), (dict(ok=X + 64), INV, "overlaps"), (dict(ok=XO + 128), INV, "overlaps"),
    (dict(rstd=XO + 4), INV, "overlaps"), (dict(rstd=WQ), INV, "overlaps"), (dict(oq=WK - 64), INV, "overlaps")])
def test_head_norm_refuses_operands(lib, kw, code, needle):
    assert norm(lib, heads(), **kw) == code and needle in lib.mc_last_error().decode()


@pytest.mark.parametrize("kw,code,needle", [
    (dict(dyq=None), INV, "null"), (dict(dk=None), INV, "null"), (dict(rstd=None), INV, "null"), (dict(dwq=DWQ + 2), INV, "aligned"),
    (dict(dq=GX + 2), INV, "overlaps"), (dict(dq=GY), INV, "overlaps"), (dict(dq=Y - 64), INV, "overlaps"),
    (dict(dqt=64), INV, "share addresses"), (dict(dwq=DWK + 4), INV, "overlaps"), (dict(dwq=WSP + 64), INV, "overlaps"),
    (dict(dwk=WQ), INV, "overlaps"), (dict(ws=None), WS, "workspace"), (dict(ws=WSP + 8), WS, "workspace"), (dict(nbytes=8), WS, "workspace")])
def test_head_norm_gradient_refuses_operands(lib, kw, code, needle):
    assert norm_grad(lib, heads(), **kw) == code and needle in lib.mc_last_error().decode()


def test_head_norm_workspace_and_no_tokens(lib):
    n = ctypes.c_size_t(0)
    assert lib.mc_head_norm_rope_backward_workspace_size(128, n) == abi.MC_OK and n.value >= 2 * 128 * 4
    assert mc.head_norm_backward_workspace_size(128) == n.value
    for d, at in ((0, n), (7, n), (258, n), (64, None)):
        assert lib.mc_head_norm_rope_backward_workspace_size(d, at) == INV
    assert norm(lib, None) == INV and norm_grad(lib, None) == INV
    assert norm(lib, heads(T=0), q=None, oq=None, rstd=None) == abi.MC_OK
    assert norm_grad(lib, heads(T=0), dq=None, dwq=None, dwk=None) == abi.MC_OK


# ----------------------------------------------------------------------- AdamW
def tensor(i=0, **kw):
    p, g, m, v, ms, vs = (FAKE + (40 + 6 * i + j) * STEP for j in range(6))
    t = McAdamTensor(p, g, m, v, None, None, 1000, BF, BF, F32)
    if kw.get("state_dtype") == F8:
        t.m_scale, t.v_scale = ms, vs
    return fill(t, kw)


def adamw(lib, *ts, count=None, scale=None, status=None, **kw):
    hp = fill(McAdamHparams(1e-3, 0.9, 0.95, 1e-8, 0.1, 1, None), kw)
    return lib.mc_adamw_step((McAdamTensor * len(ts))(*ts), len(ts) if count is None else count, hp, scale, status, None)


AT = FAKE + 40 * STEP


@pytest.mark.parametrize("kw", [dict(beta1=0.96), dict(beta2=0.98), dict(beta2=0.999), dict(beta1=0.99, beta2=0.9)])
def test_adamw_refuses_8_bit_states_whose_codes_would_stand_still(lib, kw):
    assert adamw(lib, tensor(), tensor(1, state_dtype=F8), **kw) == UNS
    text = lib.mc_last_error().decode()
    assert "tensor 1" in text and "betas up to 0.95" in text
    # what is left passes that check: a later refusal is met
    assert adamw(lib, tensor(0, state_dtype=F8, g=AT), beta1=0.95, beta2=0.95) == INV and "overlaps" in lib.mc_last_error().decode()
    assert adamw(lib, tensor(0, g=AT), **kw) == INV and "overlaps" in lib.mc_last_error().decode()


@pytest.mark.parametrize("kw,needle", [
    (dict(lr=float("nan")), "lr"), (dict(weight_decay=float("inf")), "lr"), (dict(eps=-1e-8), "eps"), (dict(beta1=1.0), "beta"),
    (dict(beta2=-0.1), "beta"), (dict(beta1=float("nan")), "beta"), (dict(step=0), "step"), (dict(count=-1), "need"),
    (dict(step_device=FAKE + 4), "aligned"), (dict(scale=FAKE + 2), "aligned"), (dict(status=FAKE + 2), "aligned"),
    (dict(status=AT + 8), "overlaps"), (dict(scale=AT + 4), "overlaps"), (dict(step_device=AT + 8), "overlaps")])
def test_adamw_refuses(lib, kw, needle):
    assert adamw(lib, tensor(), **kw) == INV and needle in lib.mc_last_error().decode()


@pytest.mark.parametrize("kw,needle", [
    (dict(n=-1), "values"), (dict(n=1 << 41), "values"), (dict(p_dtype=F8), "dtypes"), (dict(g_dtype=9), "dtypes"),
    (dict(state_dtype=BF), "dtypes"), (dict(p=None), "null"), (dict(g=None), "null"), (dict(m=None), "null"), (dict(v=None), "null"),
    (dict(m_scale=FAKE), "scales"), (dict(state_dtype=F8, v_scale=None), "scales"), (dict(p=AT + 1), "aligned"),
    (dict(m=AT + 2 * STEP + 2), "aligned"), (dict(state_dtype=F8, m_scale=FAKE + 2), "aligned"), (dict(g=AT), "overlaps"),
    (dict(m=AT + 3 * STEP + 4), "overlaps"), (dict(state_dtype=F8, m_scale=AT + 8), "overlaps")])
def test_adamw_refuses_tensors(lib, kw, needle):
    assert adamw(lib, tensor(1), tensor(**kw), tensor(2)) == INV
    text = lib.mc_last_error().decode()
    assert needle in text and "tensor 1" in text


def test_adamw_of_tensors_that_meet_and_of_nothing(lib):
    assert adamw(lib, tensor(), tensor(1, p=AT + 1000)) == INV                    # p of one within p of the other
    assert adamw(lib, tensor(), tensor(1, g=AT + 2 * STEP)) == INV                # a gradient among a moment
    assert adamw(lib, count=0) == abi.MC_OK
    assert adamw(lib, tensor(n=0, p=None, g=None, m=None, v=None)) == abi.MC_OK
    assert lib.mc_adamw_step(None, 1, McAdamHparams(1e-3, 0.9, 0.95, 1e-8, 0.1, 1, None), None, None, None) == INV
    assert lib.mc_adamw_step(None, 0, None, None, None, None) == INV


# --------------------------------------------------------------------- binding
def test_bindings_refuse_host_tensors_and_kinds():
    x, o = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    r = torch.zeros(4, 4)
    for call in (lambda: mc.qk_norm_rope(x, x), lambda: mc.qk_norm_rope_backward(x, x, x, x, r),
                 lambda: mc.qk_attention_packed_forward(x, x, x, o), lambda: mc.qk_attention_packed_backward(x, x, x, x, r, x, o),
                 lambda: mc.adamw_step([x], [x], [x], [x])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for call, needle in (
            (lambda: mc.qk_norm_rope([1]), "must be a tensor"), (lambda: mc.qk_norm_rope(None), "must be a tensor"),
            (lambda: mc.qk_norm_rope(x, x, rot=1.5), "rot"), (lambda: mc.adamw_step([x], [x], [x], []), "one length"),
            (lambda: mc.adamw_step([x], [x], [x], [x], m_scales=[r]), "go together"),
            (lambda: mc.adamw_step([x], [1], [x], [x]), "list of tensors"), (lambda: mc.adamw_state([x], bits=16), "bits"),
            (lambda: mc.packed_workspace_size(x, x[:, :, :32], x, o), "k must be"),
            (lambda: mc.packed_workspace_size(x, x, x, o.long()), "offsets"),
            (lambda: mc.packed_workspace_size(x, x, x, o[:1]), "offsets"),
            (lambda: mc.packed_workspace_size(x[0], x, x, o), "heads, features"),
            (lambda: mc.packed_workspace_size(x, x, x.float(), o), "dtype")):
        with pytest.raises(ValueError, match=needle):
            call()
    with pytest.raises(abi.MuonClipError, match="bf16"):
        mc.packed_workspace_size(*(3 * [x.float()]), o)
    with pytest.raises(TypeError):
        mc.qk_norm_rope(x, x, theta="1")
    mc.adamw_step([], [], [], [])


def test_workspace_size_and_clip_segments():
    x, o = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    n = ctypes.c_size_t(0)
    d = McPackedDesc(4, 2, 2, 2, 64, 64, BF, 0.125)
    assert abi.load().qk_attention_packed_workspace_size(d, 1, n) == abi.MC_OK
    assert mc.packed_workspace_size(x, x, x, o, backward=True) == n.value
    (s,) = mc.gqa_segments(torch.zeros(8 * 16, 4), 8)
    assert (s.offset, s.stride, s.rows, s.exponent) == (0, 16, 16, 1.0)


def test_packed_positions():
    from muon_qk_clip_gb300.forward import packed_positions
    got = packed_positions(torch.tensor([2, 2, 5, 6, 6, 9], dtype=torch.int32), 9)
    assert got.dtype == torch.int32 and got.tolist() == [0, 0, 0, 1, 2, 0, 0, 1, 2]
    assert packed_positions(torch.tensor([0, 0], dtype=torch.int32), 0).shape == (0,)


def test_struct_layouts(tmp_path):
    """Sizes and every field's offset, as the C compiler sees the header."""
    structs = dict(mc_packed_desc=McPackedDesc, mc_packed_grad=McPackedGrad, mc_heads=McHeads, mc_adamw_tensor=McAdamTensor,
                   mc_adamw_hparams=McAdamHparams)
    header = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "muonclip.h")
    lines, want = [], []
    for name, s in structs.items():
        lines.append(f'printf("%zu ", sizeof({name}));')
        want.append(ctypes.sizeof(s))
        for field, _ in s._fields_:
            lines.append(f'printf("%zu ", offsetof({name}, {field}));')
            want.append(getattr(s, field).offset)
    src = tmp_path / "l.c"
    src.write_text(f'#include <stdio.h>\n#include <stddef.h>\n#include "{header}"\nint main(void) {{ {" ".join(lines)} return 0; }}')
    subprocess.run(["gcc", "-std=c99", str(src), "-o", str(tmp_path / "l")], check=True)
    got = subprocess.run([str(tmp_path / "l")], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in got] == want


def test_another_torch_makes_the_build_stale(lib, monkeypatch, tmp_path):
    """_host.so is compiled against one torch's headers: with another version it is built again."""
    from muon_qk_clip_gb300 import build
    assert not build._stale()
    other = tmp_path / "host.torch"
    monkeypatch.setattr(build, "HOST_TORCH", str(other))
    assert build._stale()
    other.write_text("0.0")
    assert build._stale()
