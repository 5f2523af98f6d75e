"""GPU: every call may be the first CUDA work of its host thread.  A thread that has used neither torch's nor the
runtime's GPU calls has no current context of its own yet; the tensor maps are made through the driver, which
wants one."""

import ctypes
import threading

import pytest
import torch

from structured_sparse_attention_cowa_b200 import cowa as cw
from structured_sparse_attention_cowa_b200 import synth

pytestmark = pytest.mark.gpu

PAT = cw.Pattern(8, 60, 256, 2)


def in_a_fresh_thread(f):
    out = []

    def work():
        try:
            out.append(f())
        except Exception as e:  # noqa: BLE001
            out.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    return out[0]


@pytest.mark.parametrize("name", ["fwd", "decode", "decode_fp8", "decode_paged", "decode_paged_fp8", "fwd_paged", "bwd"])
def test_first_call_of_a_thread(cuda_device, name):
    B, N, Hq, Hkv, d, ps = 1, 256, 4, 2, 128, 16
    L, pat = cw.lib(), PAT.c()
    r = lambda s, nm: synth.cuda_normal_bf16(s, synth.seed_of(nm, 131), cuda_device)
    q, k, v = r((B, N, Hq, d), "q"), r((B, N, Hkv, d), "k"), r((B, N, Hkv, d), "v")
    k8, v8 = cw.quantize_e4m3(k, 1 / 64), cw.quantize_e4m3(v, 1 / 64)
    o, lse = torch.zeros_like(q), torch.zeros((B, Hq, N), device=cuda_device)
    fo, fl = cw.cowa_fwd(q, k, v, PAT)
    grads = [torch.zeros_like(x) for x in (q, k, v)]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    pos, cu, start, tab = i32([N - 1]), i32([0, N]), i32([0]), i32([list(range(N // ps))])
    ws, stream = torch.zeros(1 << 24, dtype=torch.uint8, device=cuda_device), torch.cuda.Stream()
    t4 = lambda x: cw.c_tensor(x.data_ptr(), x.stride(0), x.stride(1), x.stride(2))
    pages = lambda x: t4(x.view(N // ps, ps, Hkv, d))
    table = cw.c_page_table(tab.data_ptr(), tab.stride(0), 0, N // ps, ps, N // ps, 0)
    p, tail = ctypes.byref(pat), (ws.data_ptr(), ws.numel(), stream.cuda_stream)
    one = (p, B, Hq, Hkv, d)
    out = (pos.data_ptr(), o.data_ptr(), lse.data_ptr(), *tail)
    qt = q[:, -1].contiguous()
    call = {
        "fwd": lambda: L.cowa_fwd(p, B, N, Hq, Hkv, d, t4(q), t4(k), t4(v), t4(o), lse.data_ptr(), *tail),
        "bwd": lambda: L.cowa_bwd(p, B, N, Hq, Hkv, d, t4(q), t4(k), t4(v), t4(fo), fl.data_ptr(), t4(q),
                                  *(t4(x) for x in grads), *tail),
        "decode": lambda: L.cowa_decode(*one, N, qt.data_ptr(), t4(k), t4(v), *out),
        "decode_fp8": lambda: L.cowa_decode_fp8(*one, N, qt.data_ptr(), t4(k8), t4(v8), 1 / 64, 1 / 64, *out),
        "decode_paged": lambda: L.cowa_decode_paged(*one, qt.data_ptr(), pages(k), pages(v), table, *out),
        "decode_paged_fp8": lambda: L.cowa_decode_paged_fp8(*one, qt.data_ptr(), pages(k8), pages(v8), 1 / 64, 1 / 64,
                                                            table, *out),
        "fwd_paged": lambda: L.cowa_fwd_paged(p, 1, N, Hq, Hkv, d, cu.data_ptr(), start.data_ptr(), t4(q), pages(k),
                                              pages(v), table, t4(o), lse.data_ptr(), *tail),
    }[name]
    torch.cuda.synchronize()
    assert in_a_fresh_thread(call) == 0
    torch.cuda.synchronize()
    assert cw.workspace_status(ws) == 0
    got = [x.clone() for x in (o, lse, *grads)]
    for x in (o, lse, *grads):
        x.zero_()
    torch.cuda.synchronize()
    assert call() == 0
    torch.cuda.synchronize()
    for a, b in zip(got, (o, lse, *grads)):
        assert torch.equal(a, b)
    assert any(x.any() for x in got)


@pytest.mark.parametrize("captured", [False, True])
def test_first_python_call_of_a_thread(cuda_device, captured):
    """The same through the Python calls, also while another thread's stream is being captured."""
    N, Hq, Hkv, d, ps = 64, 4, 2, 128, 16
    r = lambda s, nm: synth.cuda_normal_bf16(s, synth.seed_of(nm, 132), cuda_device)
    q, kp, vp = r((1, Hq, d), "q"), r((N // ps, ps, Hkv, d), "k"), r((N // ps, ps, Hkv, d), "v")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    tab, pos = i32([list(range(N // ps))]), i32([N - 1])
    ws = [torch.zeros(1 << 22, dtype=torch.uint8, device=cuda_device) for _ in range(2)]
    run = lambda w, o, lse: cw.cowa_decode_paged(q, kp, vp, tab, pos, PAT, out=o, lse=lse, workspace=w)
    outs = [(torch.zeros_like(q), torch.zeros((1, Hq), device=cuda_device)) for _ in range(2)]
    wo, wl = run(ws[0], None, None)
    torch.cuda.synchronize()
    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, capture_error_mode="thread_local"):
            run(ws[0], *outs[0])
            got = in_a_fresh_thread(lambda: run(ws[1], *outs[1]))
            run(ws[0], *outs[0])
        g.replay()
    else:
        got = in_a_fresh_thread(lambda: run(ws[1], *outs[1]))
        run(ws[0], *outs[0])
    torch.cuda.synchronize()
    assert not isinstance(got, Exception), got
    for o, lse in outs:
        assert torch.equal(o, wo) and torch.equal(lse, wl)
