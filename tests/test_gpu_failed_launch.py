"""GPU: a launch that the runtime refuses is reported by the call that made it, and by no later one: the runtime
keeps it as the last error, which the check after the next launch would otherwise take for its own.  The launches
are refused because the stream's capture has been broken off (a synchronisation inside it)."""

import pytest
import torch

from structured_sparse_attention_cowa_b200 import cowa as cw
from structured_sparse_attention_cowa_b200 import synth

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["rope", "append", "append_fp8", "decode", "decode_list", "decode_fp8", "fwd_paged", "fwd",
                                  "decode_contiguous"])
def test_a_refused_launch_is_not_remembered(cuda_device, name):
    Hq, Hkv, d, ps, n = 4, 2, 128, 16, 8
    pat, rope = cw.Pattern(4, 50, 128, 2), cw.Rope(cw.rope_frequencies(d, device=cuda_device))
    r = lambda s, nm: synth.cuda_normal_bf16(s, synth.seed_of(nm, 150), cuda_device)
    q, k = r((2, Hq, d), "q"), r((2, Hkv, d), "k")
    pool = r((2 * n, ps, Hkv, d), "v")
    codes_of, codes = pool.clone(), cw.quantize_e4m3(pool, 1 / 64)
    x4, cache = r((1, 64, 2, d), "do"), r((2, Hkv, 128, d), "k_cache")
    o4, lse4 = torch.zeros_like(x4), torch.zeros((1, 2, 64), device=cuda_device)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    tab, pos, cu = torch.arange(2 * n, device=cuda_device).int().view(2, n), i32([100, 7]), i32([0, 1, 2])
    long = torch.cat([tab, torch.full((2, 3000), -1, dtype=torch.int32, device=cuda_device)], 1)
    far = cw.Pattern(4, 50, 400000, 2)
    ws, o = torch.zeros(1 << 24, dtype=torch.uint8, device=cuda_device), torch.zeros_like(q)
    lse, lse2 = torch.zeros((2, Hq), device=cuda_device), torch.zeros((Hq, 2), device=cuda_device)
    call = {
        "rope": lambda: cw.cowa_rope(q[None], None, rope, q_out=o[None]),
        "append": lambda: cw.paged_append(q, k, k, pos, pool, pool, tab, rope=rope, q_out=o),
        "append_fp8": lambda: cw.paged_append_fp8(q, k, k, pos, codes, codes, tab, 1 / 64, 1 / 64, rope=rope, q_out=o),
        "decode": lambda: cw.cowa_decode_paged(q, pool, pool, tab, pos, pat, out=o, lse=lse, workspace=ws),
        "decode_list": lambda: cw.cowa_decode_paged(q, pool, pool, long, pos, far, out=o, lse=lse, workspace=ws),
        "decode_fp8": lambda: cw.cowa_decode_paged_fp8(q, codes, codes, tab, pos, pat, 1 / 64, 1 / 64, out=o, lse=lse,
                                                       workspace=ws),
        "fwd_paged": lambda: cw.cowa_fwd_paged(q, pool, pool, tab, cu, pos, pat, out=o, lse=lse2, workspace=ws),
        "fwd": lambda: cw.cowa_fwd(x4, x4, x4, pat, out=o4, lse=lse4, workspace=ws),
        "decode_contiguous": lambda: cw.cowa_decode(q, cache, cache, pos, pat, out=o, lse=lse, workspace=ws),
    }[name]
    call()
    torch.cuda.synchronize()
    want = cw.cowa_fwd(x4, x4, x4, pat)[0]
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(stream):
        graph.capture_begin()
        with pytest.raises(RuntimeError):
            torch.cuda.synchronize()  # breaks the capture off
        with pytest.raises(cw.CowaError, match="COWA_ERR_CUDA"):
            call()
        with pytest.raises(RuntimeError):
            graph.capture_end()
    # calls that look at the last error after their launch
    cw.quantize_e4m3(codes_of, 1 / 64)
    assert torch.equal(cw.cowa_fwd(x4, x4, x4, pat)[0], want)
    call()
    torch.cuda.synchronize()
