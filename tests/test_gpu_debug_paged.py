"""GPU: the self-checking build over the paged calls, in every way their work is laid out: no check fails, and
every output equals the release build's bit for bit."""

import pytest
import torch

from structured_sparse_attention_cowa_b200 import cowa as cw
from structured_sparse_attention_cowa_b200 import synth
from tests.test_gpu_debug_build import _both, libs  # noqa: F401

pytestmark = pytest.mark.gpu


def rand(shape, name, dev):
    return synth.cuda_normal_bf16(shape, synth.seed_of(name, 140), dev)


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("Hq,Hkv,d,ps,n,pages,pat,pos", [
    (10, 2, 128, 24, 40, 40, cw.Pattern(20, 100, 900, 2), [900, 31, -1, 959]),             # clusters
    (16, 2, 128, 16, 60, 2000, cw.Pattern(20, 100, 400000, 2), [900, 31, -1, 959]),        # a list, joined by pair
    (8, 1, 64, 256, 20, 400, cw.Pattern(4, 9, 90000, 1), [5000, 0, 200, -5]),              # large pages, past the capacity
    (8, 8, 128, 8, 30, 30, cw.Pattern(0, 300, 240, 8), [239, 5, 100, -1, 17, 64, 63] * 20),  # many pairs
])
def test_debug_build_decodes_pages(libs, cuda_device, Hq, Hkv, d, ps, n, pages, pat, pos, e4m3):  # noqa: F811
    if e4m3 and d != 128:
        pytest.skip("E4M3 pages need d = 128")
    B = len(pos)
    tab = torch.full((B, pages), -1, dtype=torch.int32, device=cuda_device)
    tab[:, :n] = torch.randint(0, 64, (B, n), generator=torch.Generator(cuda_device).manual_seed(1), device=cuda_device,
                               dtype=torch.int32)
    pool = [rand((64, ps, Hkv, d), x, cuda_device) for x in ("k", "v")]
    if e4m3:
        pool = [cw.quantize_e4m3(p, 1 / 64) for p in pool]
    pos = [min(p, n * ps - 1) for p in pos]
    q = rand((B, Hq, d), "q", cuda_device)
    if e4m3:
        run = lambda ws: cw.cowa_decode_paged_fp8(q, *pool, tab, i32(pos, cuda_device), pat, 1 / 64, 1 / 64, workspace=ws)
    else:
        run = lambda ws: cw.cowa_decode_paged(q, *pool, tab, i32(pos, cuda_device), pat, workspace=ws)
    _both(libs, run, cuda_device)


@pytest.mark.parametrize("Hq,Hkv,d,ps,n,pat,chunks", [
    (40, 8, 128, 64, 43, cw.Pattern(128, 500, 2048, 8), [(1500, 500), (0, 129)]),
    (3, 1, 64, 16, 170, cw.Pattern(100, 2000, 1000, 1), [(2000, 200), (0, 1), (700, 0), (300, 140)]),  # parts
    (8, 1, 128, 24, 100, cw.Pattern(20, 900, 2400, 1), [(2300, 30)]),                                # parts
    (5, 5, 128, 256, 3, cw.Pattern(0, 1, 700, 5), [(0, 768), (767, 1)]),
    (3, 1, 64, 8, 40, cw.Pattern(30, 100, 320, 1), [(7 * i % 200, 1 + i % 100) for i in range(70)]),  # many sequences
    (4, 2, 64, 16, 20, cw.Pattern(3, 50, 320, 2), [(0, 500), (10**9, 30)]),                          # past the capacity
])
def test_debug_build_chunks_over_pages(libs, cuda_device, Hq, Hkv, d, ps, n, pat, chunks):  # noqa: F811
    B, total = len(chunks), sum(r for _, r in chunks)
    tab = torch.randint(0, 100, (B, n), generator=torch.Generator(cuda_device).manual_seed(2), device=cuda_device,
                        dtype=torch.int32)
    pool = [rand((100, ps, Hkv, d), x, cuda_device) for x in ("k", "v")]
    q = rand((total, Hq, d), "q", cuda_device)
    cu = [0]
    for _, r in chunks:
        cu.append(cu[-1] + r)
    _both(libs, lambda ws: cw.cowa_fwd_paged(q, *pool, tab, i32(cu, cuda_device), i32([s for s, _ in chunks], cuda_device),
                                             pat, workspace=ws), cuda_device)
