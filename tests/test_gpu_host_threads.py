"""Calls from several host threads at once, each on a stream of its own: the C
entries keep nothing of a call that another one could change, so every call
succeeds and has the bits of the call alone.

A pair of threads runs shapes that need different amounts of shared memory, as
prepared C calls (ctypes leaves the interpreter's lock during them).
"""
import ctypes
import threading

import pytest
import torch

from muon_qk_clip_gb300 import abi, build
from muon_qk_clip_gb300 import binding as mc

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
CALLS = 3000                               # per thread


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    abi.load()


def mk(*shape, dtype=BF16):
    return torch.randn(*shape, device="cuda").to(dtype)


def attention(S, dh, dv):
    """q, k, v, out, lse, do of 2 x S positions and 3 heads."""
    q, k, v, do = mk(2, S, 3, dh), mk(2, S, 3, dh), mk(2, S, 3, dv), mk(2, S, 3, dv)
    out, lse, _ = mc.qk_attention_forward(q, k, v, lse=True)
    return q, k, v, out, lse, do


def backward_call(S, dh, dv):
    a = attention(S, dh, dv)
    outs = [torch.empty_like(t) for t in a[:3]]
    ws = torch.empty(mc.attention_backward_workspace_size(a[0], a[1]), dtype=torch.uint8, device="cuda")
    got, real = [], mc._run
    mc._run = lambda fn, name, index, *args: got.append((fn, args))
    try:
        mc.qk_attention_backward(*a, dq=outs[0], dk=outs[1], dv=outs[2], workspace=ws)
    finally:
        mc._run = real
    fn, args = got[0]
    return (lambda stream: fn(*args, stream)), outs, (a, ws)


def forward_call(S, dh, dv):
    q, k, v, out, lse, _ = attention(S, dh, dv)
    smax, o, d = torch.empty(3, device="cuda"), abi.McAttnOut(), mc.attn_desc(q, k)
    o.v, o.d_v, o.o, o.lse = v.data_ptr(), dv, out.data_ptr(), lse.data_ptr()
    o.v_strides[:], o.o_strides[:] = v.stride()[:3], out.stride()[:3]
    fn = abi.load().qk_attention_forward
    call = lambda stream: fn(ctypes.byref(d), ctypes.byref(o), smax.data_ptr(), 0, None, stream)  # noqa: E731
    return call, [out, lse, smax], (q, k, v)


def max_logit_call(S, dh, dtype, argmax):
    q, k = mk(2, S, 3, dh, dtype=dtype), mk(2, S, 3, dh, dtype=dtype)
    smax, d = torch.empty(3, device="cuda"), mc.attn_desc(q, k)
    where = torch.empty(3, dtype=torch.int64, device="cuda") if argmax else None
    fn = abi.load().qk_max_logit
    call = lambda stream: fn(ctypes.byref(d), smax.data_ptr(), mc._at(where), 0, None, stream)  # noqa: E731
    return call, [smax] + ([where] if argmax else []), (q, k)


def run_at_once(*calls):
    """Every call CALLS times from its own thread; their codes that are not MC_OK."""
    want, codes = [], []
    for call, outs, _ in calls:
        assert call(torch.cuda.current_stream().cuda_stream) == abi.MC_OK
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
        for t in outs:
            t.fill_(7)
    torch.cuda.synchronize()
    start = threading.Barrier(len(calls))

    def work(call, stream):
        start.wait()
        for n in range(CALLS):
            code = call(stream.cuda_stream)
            if code != abi.MC_OK:
                codes.append((code, abi.load().mc_last_error().decode()))
            if n % 100 == 99:
                stream.synchronize()

    streams = [torch.cuda.Stream() for _ in calls]
    threads = [threading.Thread(target=work, args=(c[0], s)) for c, s in zip(calls, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not codes, (len(codes), codes[0])
    for (_, outs, _), w in zip(calls, want):
        assert all(torch.equal(a, b) for a, b in zip(outs, w))


def test_short_attention_backward_from_two_threads():
    run_at_once(backward_call(16, 192, 128), backward_call(2, 16, 16))


def test_attention_backward_of_all_lengths_from_threads():
    run_at_once(backward_call(40, 192, 128), backward_call(16, 128, 128), backward_call(40, 64, 64))


def test_attention_forward_from_two_threads():
    run_at_once(forward_call(40, 128, 128), forward_call(40, 64, 32))


def test_max_logit_from_two_threads():
    run_at_once(max_logit_call(40, 192, BF16, True), max_logit_call(40, 64, BF16, True))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_max_logit_on_cuda_cores_from_two_threads(dtype):
    """Lengths of q.k that the tensor cores do not take (bf16: 12 features, or a
    narrow view of wider rows)."""
    wide = 250 if dtype == BF16 else 256
    run_at_once(max_logit_call(40, wide, dtype, False), max_logit_call(40, 12, dtype, False))


def first_of_a_thread(call):
    """The code of a prepared call that is the first use of CUDA in its thread."""
    codes, stream = [], torch.cuda.current_stream().cuda_stream
    t = threading.Thread(target=lambda: codes.append((call(stream), abi.load().mc_last_error().decode())))
    t.start()
    t.join()
    torch.cuda.synchronize()
    return codes[0]


@pytest.mark.parametrize("S", [40, 16])
def test_attention_calls_as_the_first_of_a_thread(S):
    """A thread that has not used CUDA yet has no context until a call binds one."""
    for call, outs, _ in (backward_call(S, 64, 64), forward_call(S, 64, 64)):
        assert call(torch.cuda.current_stream().cuda_stream) == abi.MC_OK
        want = [t.clone() for t in outs]
        for t in outs:
            t.fill_(7)
        torch.cuda.synchronize()
        assert first_of_a_thread(call) == (abi.MC_OK, "")
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_an_accumulating_max_logit_as_the_first_call_of_a_thread():
    q, k = mk(2, 40, 3, 64), mk(2, 40, 3, 64)
    want, smax, d = mc.qk_max_logit(q, k)[0], torch.full((3,), -1e30, device="cuda"), mc.attn_desc(q, k)
    torch.cuda.synchronize()
    fn = abi.load().qk_max_logit
    assert first_of_a_thread(lambda s: fn(ctypes.byref(d), smax.data_ptr(), None, 1, None, s)) == (abi.MC_OK, "")
    assert torch.equal(smax, want)
