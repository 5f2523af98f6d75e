"""GPU: NaN where a query sees it.  A row whose visible scores or values hold a NaN gives NaN in o and lse, as
exact softmax attention does (and the contiguous forward's and decode's o), however the work is cut: a row that
sees NaN only must not pass for one that sees nothing (o 0, lse -inf), and a piece of the work that holds
nothing but NaN must not be dropped when the pieces are joined.  Rows that do not see it keep their bits."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import fp8_kv as f8
from structured_sparse_attention_cowa_b200 import cowa as cw
from tests.gpu_helpers import host_and_device
from tests.test_gpu_paged import make_table, widened, ws_for

pytestmark = pytest.mark.gpu
NAN = float("nan")


def decode_case(dev, e4m3, wide):
    """Three sequences of 700, 64 and no keys, dense causal, pages of their own for each head."""
    B, Hq, Hkv, d, ps, n = 3, 10, 2, 128, 16, 44
    pat, pos = cw.Pattern(0, 5000, 0, 1), [699, 63, -1]
    rng = np.random.default_rng(120)
    tab, n_pages = make_table(rng, B, n, heads=Hkv)
    if wide:
        pat, tab = widened(pat, tab, ps)
    shape = (n_pages, ps, 1, d)
    if e4m3:
        kp, vp = (torch.from_numpy(f8.f64_to_e4m3(rng.standard_normal(shape))).to(dev) for _ in range(2))
    else:
        kp, vp = (host_and_device(shape, x, dev, 120)[1] for x in ("k", "v"))
    q = host_and_device((B, Hq, d), "q", dev, 120)[1]
    fn = "cowa_decode_paged_fp8" if e4m3 else "cowa_decode_paged"
    tabd, posd = torch.from_numpy(tab).to(dev), torch.tensor(pos, dtype=torch.int32, device=dev)
    ws = ws_for(fn, pat, B, Hq, Hkv, d, tab.shape[-1], ps, dev)

    def run(q, kp, vp):
        o, lse = getattr(cw, fn)(q, kp, vp, tabd, posd, pat, *((0.5, 0.5) if e4m3 else ()), workspace=ws)
        assert cw.workspace_status(ws) == 0
        assert (o[2] == 0).all() and (lse[2] == -float("inf")).all()  # the slot without a sequence
        return o, lse

    def put(pool, b, g, s, bad):  # a NaN in row s of sequence b and head g
        pool = pool.clone()
        pool[int(tab[b, g, s // ps]), s % ps, 0, 5] = bad
        return pool

    return q, kp, vp, run, put, 0x7f if e4m3 else NAN


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("wide", [False, True])
def test_decode_of_a_nan_query(cuda_device, e4m3, wide):
    """Every score of one query head is NaN; its group's other heads keep their bits."""
    q, kp, vp, run, _, _ = decode_case(cuda_device, e4m3, wide)
    wo, wl = run(q, kp, vp)
    bad = q.clone()
    bad[0, 3, 7] = bad[1, 9, 0] = NAN
    o, lse = run(bad, kp, vp)
    hit = torch.zeros_like(lse, dtype=torch.bool)
    hit[0, 3] = hit[1, 9] = True
    assert o[hit].isnan().all() and lse[hit].isnan().all()
    assert torch.equal(o[~hit], wo[~hit]) and torch.equal(lse[~hit], wl[~hit])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("rows", [[698], [0], [300], list(range(640, 700)), list(range(700))])
def test_decode_of_nan_keys(cuda_device, e4m3, wide, rows):
    """A visible key that is NaN makes its group's heads NaN: one key, a tile's, all of them."""
    q, kp, vp, run, put, bad = decode_case(cuda_device, e4m3, wide)
    wo, wl = run(q, kp, vp)
    for s in rows:
        kp = put(kp, 0, 1, s, bad)
    o, lse = run(q, kp, vp)
    assert o[0, 5:].isnan().all() and lse[0, 5:].isnan().all()
    hit = torch.zeros_like(lse, dtype=torch.bool)
    hit[0, 5:] = True
    assert torch.equal(o[~hit], wo[~hit]) and torch.equal(lse[~hit], wl[~hit])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("wide", [False, True])
def test_decode_of_a_nan_value(cuda_device, e4m3, wide):
    """A visible value that is NaN makes its column NaN, and nothing else."""
    q, kp, vp, run, put, bad = decode_case(cuda_device, e4m3, wide)
    wo, wl = run(q, kp, vp)
    o, lse = run(q, kp, put(vp, 0, 0, 333, bad))
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[0, :5, 5] = True
    assert o[hit].isnan().all() and torch.equal(o[~hit], wo[~hit]) and torch.equal(lse, wl)


@pytest.mark.parametrize("Hq,Hkv,d,rows,parts", [
    (40, 8, 128, 1000, False),   # pairs of heads and single ones, not cut
    (24, 24, 64, 1000, False),   # single heads
    (3, 1, 64, 300, True),       # key tiles cut into parts
    (2, 1, 128, 300, True),
])
def test_chunk_of_nan_queries_and_keys(cuda_device, Hq, Hkv, d, rows, parts):
    """Query rows that are NaN, and a key that is NaN: the rows that see it, in the heads it belongs to.  Not cut:
    key 0 is a sink, which all rows see (alone in its tile for the far ones), the others are seen through a band
    of 50.  Cut: every key up to the row."""
    ps, n, start, total = 16, 128, 900, rows + 10
    pat = cw.Pattern(1, 50, 2000 if parts else 1, 1)
    tab = torch.from_numpy(make_table(np.random.default_rng(121), 1, n)[0]).to(cuda_device)
    kp, vp = (host_and_device((n + 2, ps, Hkv, d), x, cuda_device, 121)[1] for x in ("k", "v"))
    q = host_and_device((total, Hq, d), "q", cuda_device, 121)[1]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    size = cw.lib().cowa_fwd_paged_workspace_size(ctypes.byref(pat.c()), 1, total, Hq, Hkv, d, n, ps)
    assert (size > 256) == parts
    ws = torch.zeros(size, dtype=torch.uint8, device=cuda_device)

    def run(q, kp):
        out, lse = torch.zeros_like(q), torch.zeros((Hq, total), device=cuda_device)
        cw.cowa_fwd_paged(q, kp, vp, tab, i32([0, rows]), i32([start]), pat, out=out, lse=lse, workspace=ws)
        assert cw.workspace_status(ws) == 0
        return out, lse.t()

    def check(got, want, hit):
        (o, lse), (wo, wl) = got, want
        assert o[hit].isnan().all() and lse[hit].isnan().all()
        assert torch.equal(o[~hit], wo[~hit]) and torch.equal(lse[~hit], wl[~hit])

    want = run(q, kp)
    assert not any(x.isnan().any() for x in want)
    bad = q.clone()
    bad[17, 1, 3] = bad[128, 0, 0] = bad[rows - 1, Hq - 1, 1] = NAN
    hit = torch.zeros((total, Hq), dtype=torch.bool, device=cuda_device)
    hit[17, 1] = hit[128, 0] = hit[rows - 1, Hq - 1] = True
    check(run(bad, kp), want, hit)
    for key, seen in ((0, slice(0, rows)), (1000, slice(100, 150) if not parts else slice(100, rows))):
        bad = kp.clone()
        bad[int(tab[0, key // ps]), key % ps, 0, 2] = NAN
        hit = torch.zeros((total, Hq), dtype=torch.bool, device=cuda_device)
        hit[seen, :Hq // Hkv] = True
        check(run(q, bad), want, hit)
    # nothing but NaN in a tile of keys that some rows see in part: all keys of the last 64 positions
    bad = kp.clone()
    for key in range(start + rows - 64, start + rows):
        bad[int(tab[0, key // ps]), key % ps, 0] = NAN
    hit = torch.zeros((total, Hq), dtype=torch.bool, device=cuda_device)
    hit[rows - 64:rows, :Hq // Hkv] = True
    check(run(q, bad), want, hit)
