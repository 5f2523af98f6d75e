"""GPU: paged decodes issued by several host threads at once, each on its stream with its workspace, which the
library allows.  The calls differ in what their kernels' blocks need (the join takes room for every head of the
group), so no call may leave a setting of a kernel that another one's launch depends on.  The threads are those
of a C program (tests/c_abi/concurrent_decodes.c): Python's take turns at the interpreter."""

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from structured_sparse_attention_cowa_b200 import cowa as cw
from structured_sparse_attention_cowa_b200 import synth

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Job(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("decode", "decode_fp8", "pat", "q", "pos", "o", "lse", "ws")] + \
        [("ws_bytes", ctypes.c_size_t), ("stream", ctypes.c_void_p), ("k", cw.c_tensor), ("v", cw.c_tensor),
         ("table", cw.c_page_table)] + [(n, ctypes.c_int) for n in ("B", "Hq", "Hkv", "d", "calls", "bad")]


@pytest.fixture(scope="module")
def run_jobs(tmp_path_factory):
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    so = str(tmp_path_factory.mktemp("threads") / "concurrent_decodes.so")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pthread", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "c_abi", "concurrent_decodes.c"), "-o", so],
                   check=True, capture_output=True, text=True)
    return ctypes.CDLL(so).run_jobs


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("wide", [False, True])  # the cluster form, the list form
def test_decodes_from_several_threads(cuda_device, run_jobs, e4m3, wide):
    B, Hkv, d, ps, n, calls = 2, 2, 128, 16, 20, 5000
    L, pat = cw.lib(), cw.Pattern(4, 100, 400000 if wide else 320, 1)
    pages = 2000 if wide else n  # (entries of the table; the positions stay below n * ps)
    pool = [synth.cuda_normal_bf16((B * n, ps, Hkv, d), synth.seed_of(x, 130), cuda_device) for x in ("k", "v")]
    if e4m3:
        pool = [cw.quantize_e4m3(p, 1 / 64) for p in pool]
    tab = torch.zeros((B, pages), dtype=torch.int32, device=cuda_device)
    tab[:, :n] = torch.randperm(B * n, device=cuda_device).int().view(B, n)
    pos = torch.tensor([300, 77], dtype=torch.int32, device=cuda_device)
    fn = "cowa_decode_paged_fp8" if e4m3 else "cowa_decode_paged"
    t4 = lambda x: cw.c_tensor(x.data_ptr(), x.stride(0), x.stride(1), x.stride(2))
    table = cw.c_page_table(tab.data_ptr(), tab.stride(0), 0, pages, ps, B * n, 0)
    cpat = pat.c()
    groups = (1, 2, 3, 4, 5, 6, 8)
    jobs, keep = (Job * len(groups))(), []
    for j, grp in zip(jobs, groups):
        Hq = grp * Hkv
        q = synth.cuda_normal_bf16((B, Hq, d), synth.seed_of("q", grp), cuda_device)
        size = getattr(L, fn + "_workspace_size")(ctypes.byref(cpat), B, Hq, Hkv, d, pages, ps)
        x = dict(q=q, o=torch.zeros_like(q), lse=torch.zeros((B, Hq), device=cuda_device),
                 ws=torch.zeros(size, dtype=torch.uint8, device=cuda_device), stream=torch.cuda.Stream())
        keep.append(x)
        setattr(j, "decode_fp8" if e4m3 else "decode", ctypes.cast(getattr(L, fn), ctypes.c_void_p))
        j.pat, j.pos, j.ws_bytes, j.stream = ctypes.addressof(cpat), pos.data_ptr(), size, x["stream"].cuda_stream
        for name in ("q", "o", "lse", "ws"):
            setattr(j, name, x[name].data_ptr())
        j.k, j.v, j.table, j.B, j.Hq, j.Hkv, j.d = t4(pool[0]), t4(pool[1]), table, B, Hq, Hkv, d
    torch.cuda.synchronize()
    want = []
    for i, x in enumerate(keep):
        jobs[i].calls = 1
        assert run_jobs(ctypes.byref(jobs[i]), 1) == 0 and jobs[i].bad == 0
        torch.cuda.synchronize()
        want.append((x["o"].clone(), x["lse"].clone()))
        x["o"].zero_()
        jobs[i].calls = calls
    torch.cuda.synchronize()
    assert run_jobs(jobs, len(jobs)) == 0
    torch.cuda.synchronize()
    assert [j.bad for j in jobs] == [0] * len(jobs)
    for x, (o, lse) in zip(keep, want):
        assert torch.equal(x["o"], o) and torch.equal(x["lse"], lse) and o.any()
        assert cw.workspace_status(x["ws"]) == 0
