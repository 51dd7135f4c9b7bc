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
