"""GPU parity of the paged cache: tokens written to pages (paged_append, bf16 and E4M3) and decode over
them, against the fp64 oracle over the cache the pages stand for.

Tolerances of decode, element by element.  P is rounded to bf16 (half a step 2^-8; f16 with E4M3
pages, 2^-11), which moves o by at most that share of A = sum p |v| / sum p; o is rounded to bf16
(2^-8 |o|).  Scores are sums of d products in 32 bits: with N(0,1) inputs and d = 128 they are off by
less than 2^-13, as are the 32-bit sums of P and O together, so 2^-12 A more.  lse: 2^-13 of score
error and a few roundings of a number below 32: 2e-4."""

import ctypes
import dataclasses

import numpy as np
import pytest
import torch

from oracle import cowa_oracle as orc
from oracle import fp8_kv as f8
from oracle import rope as orp
from structured_sparse_attention_cowa_b200 import cowa as cw
from structured_sparse_attention_cowa_b200 import synth
from tests.gpu_helpers import host_and_device, oracle_pattern, to64
from tests.test_gpu_rope import assert_rotated

pytestmark = pytest.mark.gpu
LSE_TOL = 2e-4


def assert_decoded(o, lse, q64, k, v, pos, pat, p_eps=2.0 ** -8, has=None):
    """o, lse (CUDA) against attention of q64 [B, Hq, d] over k, v [B, Hkv, T, d] (float64) at pos; `has`
    [B, Hkv, T]: positions that have a page."""
    B, Hq, d = q64.shape
    Hkv, Tc = k.shape[1], k.shape[2]
    op = oracle_pattern(pat)
    scale = pat.softmax_scale or 1 / np.sqrt(d)
    go, gl = to64(o), lse.double().cpu().numpy()
    for b in range(B):
        t = min(pos[b], Tc - 1)
        for g in range(Hkv):
            hs = slice(g * Hq // Hkv, (g + 1) * Hq // Hkv)
            see = orc.visible_mask(np.array([max(t, 0)]), Tc, op, g, Hkv)[0] if t >= 0 else np.zeros(Tc, bool)
            if has is not None:
                see = see & has[b, g]
            if not see.any():
                assert (go[b, hs] == 0).all() and (gl[b, hs] == -np.inf).all(), (b, g)
                continue
            s = q64[b, hs] @ k[b, g, see].T * scale
            m = s.max(1, keepdims=True)
            p = np.exp(s - m)
            want = p @ v[b, g, see] / p.sum(1, keepdims=True)
            A = p @ np.abs(v[b, g, see]) / p.sum(1, keepdims=True)
            err = np.abs(go[b, hs] - want)
            assert (err <= p_eps * A + 2.0 ** -8 * np.abs(want) + 2.0 ** -12 * A).all(), (b, g, err.max())
            lerr = np.abs(gl[b, hs] - (m[:, 0] + np.log(p.sum(1))))
            assert (lerr <= LSE_TOL).all(), (b, g, lerr.max())


def make_table(rng, B, n, spare=2, heads=None):
    """A table [B(, heads), n] of distinct pages in random order and the pool's size."""
    want = B * n * (heads or 1)
    t = rng.permutation(want + spare)[:want].astype(np.int32)
    return t.reshape((B, heads, n) if heads else (B, n)), want + spare


def widened(pat, tab, ps):
    """The pattern with a far longer declared span (head 0's interval then holds everything behind the
    sink) and the table with unmapped pages up to 25,000 positions: a call that could have long pairs,
    whose work is shared out over the whole list of tiles and joined by a second kernel; the small
    caches of these tests otherwise take the cluster form."""
    more = -(-25000 // ps) - tab.shape[-1]
    return dataclasses.replace(pat, T=pat.S + 400000), np.concatenate(
        [tab, np.full((*tab.shape[:-1], more), -1, np.int32)], axis=-1)


def ws_for(fn, pat, B, Hq, Hkv, d, n, ps, dev):
    size = getattr(cw.lib(), fn + "_workspace_size")(ctypes.byref(pat.c()), B, Hq, Hkv, d, n, ps)
    return torch.zeros(size, dtype=torch.uint8, device=dev)


DECODE = [
    # Hq, Hkv, d, pattern, page, pages, per head, layout, positions
    (8, 4, 128, cw.Pattern(64, 128, 1024, 4), 64, 16, False, "bhtd", [0, 63, 64, 200, 1023, 511, -1]),
    (10, 2, 128, cw.Pattern(20, 100, 900, 2), 16, 63, False, "bthd", [899, 17, 1000, 5, 5000]),   # past T, past the end
    (8, 8, 128, cw.Pattern(0, 1, 1024, 8), 8, 128, True, "bhtd", [1023, 0, 700]),                 # L = 1, no sink
    (16, 2, 64, cw.Pattern(4, 60, 4, 1), 24, 43, False, "bthd", [1023, 3, 64, -1, -7]),           # sinks and band only
    (7, 1, 64, cw.Pattern(33, 5000, 1024, 1), 48, 22, True, "bthd", [1000, 1]),                   # dense, group of 7
    (24, 4, 128, cw.Pattern(100, 7, 700, 2), 256, 4, False, "bhtd", [1023, 650, 0]),              # pages over a tile, D < H
    (6, 2, 128, cw.Pattern(30, 90, 1000, 4, kv_head_base=1, h_kv_global=4), 32, 32, False, "bthd", [999, 400]),
    (40, 8, 128, cw.Pattern(128, 500, 4096, 8), 128, 32, False, "bhtd", [4095] * 3 + [17]),
    (5, 1, 128, cw.Pattern(0, 1, 0, 1), 16, 4, False, "bthd", [40]),                              # one visible key
    (3, 3, 64, cw.Pattern(10**6, 1, 10**6, 1), 40, 20, False, "bthd", [777, 39, 40]),             # all sink
]


@pytest.mark.parametrize("Hq,Hkv,d,pat,ps,n,per_head,layout,pos", DECODE)
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("wide", [False, True])
def test_decode_matches_oracle(cuda_device, Hq, Hkv, d, pat, ps, n, per_head, layout, pos, e4m3, wide):
    if e4m3 and d != 128:
        pytest.skip("E4M3 pages need d = 128")
    B, rng = len(pos), np.random.default_rng(ps * n)
    tab, n_pages = make_table(rng, B, n, heads=Hkv if per_head else None)
    cap = n * ps
    if wide:
        pat, tab = widened(pat, tab, ps)
        pos = [min(p, cap - 1) for p in pos]
        n = tab.shape[-1]
    shape = (n_pages, ps, 1 if per_head else Hkv, d)
    if e4m3:
        kc, vc = (f8.f64_to_e4m3(rng.standard_normal(shape) * 3) for _ in range(2))
        kd, vd = torch.from_numpy(kc).to(cuda_device), torch.from_numpy(vc).to(cuda_device)
        k64, v64 = 0.4 * f8.e4m3_to_f64(kc), 0.25 * f8.e4m3_to_f64(vc)
    else:
        (k64, kd), (v64, vd) = (host_and_device(shape, x, cuda_device, 71) for x in ("k", "v"))
    if layout == "bhtd":
        kd, vd = kd.transpose(1, 2).contiguous(), vd.transpose(1, 2).contiguous()
    q64, q = host_and_device((B, Hq, d), "q", cuda_device, 72)
    fn = "cowa_decode_paged_fp8" if e4m3 else "cowa_decode_paged"
    ws = ws_for(fn, pat, B, Hq, Hkv, d, n, ps, cuda_device)
    o, lse = getattr(cw, fn)(q, kd, vd, torch.from_numpy(tab).to(cuda_device),
                             torch.tensor(pos, dtype=torch.int32, device=cuda_device), pat,
                             *((0.4, 0.25) if e4m3 else ()), layout=layout, workspace=ws)
    assert cw.workspace_status(ws) == 0
    k, _ = orp.gather_pages(k64, tab, cap)
    v, _ = orp.gather_pages(v64, tab, cap)
    assert_decoded(o, lse, q64, k, v, pos, pat, 2.0 ** -11 if e4m3 else 2.0 ** -8)


def test_decode_equals_the_contiguous_decode(cuda_device):
    """The same keys in one array per sequence: cowa_decode within both roundings."""
    B, Hq, Hkv, d, Tc, ps = 3, 10, 2, 128, 2048, 64
    pat = cw.Pattern(64, 300, 2048, 2)
    kc, vc = (synth.cuda_normal_bf16((B, Hkv, Tc, d), synth.seed_of(x, 73), cuda_device) for x in ("k", "v"))
    q = synth.cuda_normal_bf16((B, Hq, d), synth.seed_of("q", 73), cuda_device)
    pos = torch.tensor([2047, 1000, 3], dtype=torch.int32, device=cuda_device)
    pages = lambda x: x.view(B, Hkv, Tc // ps, ps, d).permute(0, 2, 1, 3, 4).reshape(-1, Hkv, ps, d).contiguous()
    tab = torch.arange(B * Tc // ps, dtype=torch.int32, device=cuda_device).view(B, -1)
    o, lse = cw.cowa_decode_paged(q, pages(kc), pages(vc), tab, pos, pat, layout="bhtd")
    wo, wl = cw.cowa_decode(q, kc, vc, pos, pat)
    assert (o.float() - wo.float()).abs().max() <= 2 * 2e-2
    assert (lse - wl).abs().max() <= 2 * LSE_TOL


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("ps,layout", [(16, "bthd"), (64, "bhtd"), (24, "bthd")])
@pytest.mark.parametrize("wide", [False, True])
def test_unseen_rows_may_hold_anything(cuda_device, e4m3, ps, layout, wide):
    """NaN and infinities in every row that no head sees, and pages of their own for each head, of which
    only the needed ones are mapped: the same result, to the bit, as over clean pages."""
    Hq, Hkv, d, n = 10, 2, 128, 512 // ps
    pat, pos = cw.Pattern(20, 70, 500, 2), [500, 130, 60, 21, 0]
    B, rng = len(pos), np.random.default_rng(74)
    tab, n_pages = make_table(rng, B, n, heads=Hkv)
    if wide:
        pat, tab = widened(pat, tab, ps)
        n = tab.shape[-1]
    clean = tab.copy()
    shape = (n_pages, ps, 1, d)
    if e4m3:
        pools = [torch.from_numpy(f8.f64_to_e4m3(rng.standard_normal(shape))).to(cuda_device) for _ in range(2)]
        junk = [0x7f, 0xff]
    else:
        pools = [host_and_device(shape, x, cuda_device, 74)[1] for x in ("k", "v")]
        junk = [float("nan"), float("inf")]
    dirty = [p.clone() for p in pools]
    for b in range(B):
        for g in range(Hkv):
            see = orc.visible_mask(np.array([pos[b]]), n * ps, oracle_pattern(pat), g, Hkv)[0]
            for s in np.flatnonzero(~see[:512 // ps * ps]):
                for i, p in enumerate(dirty):
                    p[int(tab[b, g, s // ps]), int(s % ps), 0] = junk[(i + int(s)) % 2]
            tab[b, g, ~see.reshape(n, ps).any(1)] = [-1, 2**31 - 1, n_pages][g + 0 if b % 2 else 2]
    for p in dirty:  # pages that no table names
        p[torch.tensor(sorted(set(range(n_pages)) - set(tab[tab >= 0].tolist()) - {n_pages}), device=cuda_device)] = junk[0]
    if layout == "bhtd":
        pools, dirty = ([x.transpose(1, 2).contiguous() for x in y] for y in (pools, dirty))
    q = synth.cuda_normal_bf16((B, Hq, d), synth.seed_of("q", 74), cuda_device)
    fn = "cowa_decode_paged_fp8" if e4m3 else "cowa_decode_paged"
    run = lambda pools, t, ws: getattr(cw, fn)(q, *pools, torch.from_numpy(t).to(cuda_device),
                                               torch.tensor(pos, dtype=torch.int32, device=cuda_device), pat,
                                               *((0.5, 0.5) if e4m3 else ()), layout=layout, workspace=ws)
    ws = ws_for(fn, pat, B, Hq, Hkv, d, n, ps, cuda_device)
    wo, wl = run(pools, clean, ws)
    o, lse = run(dirty, tab, ws)
    assert cw.workspace_status(ws) == 0
    assert torch.isfinite(wo.float()).all()
    assert torch.equal(o, wo) and torch.equal(lse, wl)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("wide", [False, True])
def test_bad_entries_are_left_out_and_reported(cuda_device, e4m3, wide):
    """Entries outside the pool on pages with visible keys: their keys are left out, the status says so
    once, and a sequence whose every page is bad gives zeros and -inf."""
    B, Hq, Hkv, d, ps, n = 4, 8, 2, 128, 16, 20
    pat, pos = cw.Pattern(20, 70, 300, 2), [300, 250, 319, 15]
    rng = np.random.default_rng(75)
    tab, n_pages = make_table(rng, B, n)
    tab[0, [1, 17]] = -1, n_pages
    tab[1, 15] = 2**31 - 1
    tab[3, :] = -2**31
    if wide:
        pat, tab = widened(pat, tab, ps)
        n = tab.shape[-1]
    shape = (n_pages, ps, Hkv, d)
    if e4m3:
        kc, vc = (f8.f64_to_e4m3(rng.standard_normal(shape) * 3) for _ in range(2))
        kd, vd = torch.from_numpy(kc).to(cuda_device), torch.from_numpy(vc).to(cuda_device)
        k64, v64 = f8.e4m3_to_f64(kc), f8.e4m3_to_f64(vc)
    else:
        (k64, kd), (v64, vd) = (host_and_device(shape, x, cuda_device, 75) for x in ("k", "v"))
    q64, q = host_and_device((B, Hq, d), "q", cuda_device, 75)
    fn = "cowa_decode_paged_fp8" if e4m3 else "cowa_decode_paged"
    ws = ws_for(fn, pat, B, Hq, Hkv, d, n, ps, cuda_device)
    o, lse = getattr(cw, fn)(q, kd, vd, torch.from_numpy(tab).to(cuda_device),
                             torch.tensor(pos, dtype=torch.int32, device=cuda_device), pat,
                             *((1.0, 1.0) if e4m3 else ()), workspace=ws)
    assert cw.workspace_status(ws) == 8
    assert cw.workspace_status(ws) == 0
    k, has = orp.gather_pages(k64, tab, 320)
    v, _ = orp.gather_pages(v64, tab, 320)
    assert_decoded(o, lse, q64, k, v, pos, pat, 2.0 ** -11 if e4m3 else 2.0 ** -8, has=has)


def test_growing_scores_rescale(cuda_device):
    """Keys that grow along the sequence push the running maximum past its threshold again and again."""
    B, Hq, Hkv, d, ps, n = 1, 8, 1, 128, 64, 32
    pat, pos = cw.Pattern(0, 5000, 0, 1), [n * ps - 1]
    _, k = host_and_device((n, ps, Hkv, d), "k", cuda_device, 76)
    k = (k.float() * torch.linspace(0.1, 6, n, device=cuda_device)[:, None, None, None]).bfloat16()
    k64 = to64(k)
    v64, v = host_and_device((n, ps, Hkv, d), "v", cuda_device, 76)
    q64, q = host_and_device((B, Hq, d), "q", cuda_device, 76)
    tab = torch.arange(n, dtype=torch.int32, device=cuda_device)[None]
    o, lse = cw.cowa_decode_paged(q, k, v, tab, torch.tensor(pos, dtype=torch.int32, device=cuda_device), pat)
    flat = lambda x: x.transpose(2, 0, 1, 3).reshape(1, Hkv, n * ps, d)
    # scores up to about 6 sqrt(d) / sqrt(d) * 5: their 32-bit sums are off by six times as much
    go, gl = to64(o), lse.double().cpu().numpy()
    s = q64[0] @ flat(k64)[0, 0].T / np.sqrt(d)
    p = np.exp(s - s.max(1, keepdims=True))
    want, A = p @ flat(v64)[0, 0] / p.sum(1, keepdims=True), p @ np.abs(flat(v64)[0, 0]) / p.sum(1, keepdims=True)
    assert (np.abs(go[0] - want) <= 2.0 ** -8 * (A + np.abs(want)) + 6 * 2.0 ** -12 * A).all()
    assert np.abs(gl[0] - (s.max(1) + np.log(p.sum(1)))).max() <= 6 * LSE_TOL


def test_many_sequences_and_one_long_one(cuda_device):
    """300 short sequences beside one of 40,000 positions: shares of the work that hold many pairs, and
    pairs that many CTAs share; the same bits twice."""
    B, Hq, Hkv, d, ps = 301, 2, 2, 64, 32
    pat = cw.Pattern(40, 20000, 40000, 2)
    pos = [int(x) for x in np.random.default_rng(77).integers(-1, 90, B)]
    pos[150] = 39999
    n = 40000 // ps
    rng = np.random.default_rng(78)
    n_pages = 3000
    tab = rng.integers(0, n_pages, (B, n)).astype(np.int32)  # sequences may share pages
    (k64, kd), (v64, vd) = (host_and_device((n_pages, ps, Hkv, d), x, cuda_device, 77) for x in ("k", "v"))
    q64, q = host_and_device((B, Hq, d), "q", cuda_device, 77)
    tabd, posd = torch.from_numpy(tab).to(cuda_device), torch.tensor(pos, dtype=torch.int32, device=cuda_device)
    o, lse = cw.cowa_decode_paged(q, kd, vd, tabd, posd, pat)
    o2, lse2 = cw.cowa_decode_paged(q, kd, vd, tabd, posd, pat)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    for b in list(range(0, 12)) + [149, 150, 151, 300]:
        k, _ = orp.gather_pages(k64, tab[b:b + 1], pos[b] + 1 if pos[b] >= 0 else 1)
        v, _ = orp.gather_pages(v64, tab[b:b + 1], pos[b] + 1 if pos[b] >= 0 else 1)
        assert_decoded(o[b:b + 1], lse[b:b + 1], q64[b:b + 1], k, v, [pos[b]], pat)


# ------------------------------------------------------------------------------------------ append
APPEND = [
    # Hq, Hkv, d, r, sections, interleaved, page, pages, per head, layout
    (8, 4, 64, 64, (32,), False, 16, 6, False, "bthd"),
    (5, 1, 128, 96, (20, 20, 8), False, 24, 5, False, "bhtd"),
    (8, 2, 128, 128, (64,), True, 64, 2, True, "bthd"),
    (4, 4, 64, 22, (6, 5), False, 8, 12, True, "bhtd"),
    (0, 3, 128, 128, (64,), False, 32, 4, False, "bthd"),   # no queries
    (6, 2, 128, 0, (), False, 16, 8, False, "bthd"),        # no rotation
]


@pytest.mark.parametrize("Hq,Hkv,d,r,sec,inter,ps,n,per_head,layout", APPEND)
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("chunks", [False, True])
def test_append_matches_oracle(cuda_device, Hq, Hkv, d, r, sec, inter, ps, n, per_head, layout, e4m3, chunks):
    """Rows of several sequences, some of them padding, past the capacity or without a page: pages hold
    exactly the rotated keys and the values (E4M3: the quantiser's codes, bit for bit), everything else
    of pools and q_out stays as it was."""
    if e4m3 and d != 128:
        pytest.skip("E4M3 pages need d = 128")
    rng = np.random.default_rng(81)
    n_seq, cap = 5, n * ps
    tab, n_pages = make_table(rng, n_seq, n, heads=Hkv if per_head else None)
    tab[(0, 0, 1) if per_head else (0, 1)] = -1
    tab[(2, Hkv - 1, 0) if per_head else (2, 0)] = n_pages
    if chunks:
        seq = np.repeat(np.arange(n_seq), [20, 1, cap, 3, 7])
        pos = np.concatenate([np.arange(s, s + c) for s, c in zip((5, 0, 0, cap - 2, 9), (20, 1, cap, 3, 7))])
        seq, pos = np.r_[seq, [-1, n_seq, 3, 3]], np.r_[pos, [0, 0, -1, -2**31]]
    else:
        seq, pos = None, np.array([0, cap - 1, cap // 2, -1, 2**31 - 1])
    total = len(pos)
    f, f64 = (cw.rope_frequencies(r, device=cuda_device), None) if r else (None, None)
    rope = cw.Rope(f, sec, interleaved=inter) if r else None
    rp = rng.integers(0, 5000, (max(1, len(sec)), total)).astype(np.int32)
    qkv64, qkv = host_and_device((total, Hq + 2 * Hkv, d), "q", cuda_device, 81)
    q, k, v = qkv.split([Hq, Hkv, Hkv], dim=1)
    q64, k64, v64 = np.split(qkv64, [Hq, Hq + Hkv], axis=1)
    shape = (n_pages, ps, 1 if per_head else Hkv, d)
    view = (lambda x: x.transpose(1, 2).contiguous()) if layout == "bhtd" else (lambda x: x)
    if e4m3:
        pools = [view(torch.from_numpy(rng.integers(0, 255, shape).astype(np.uint8)).to(cuda_device)) for _ in range(2)]
    else:
        pools = [view(host_and_device(shape, x, cuda_device, 82)[1]) for x in ("k", "v")]
    before = [p.clone() for p in pools]
    i32 = lambda x: None if x is None else torch.from_numpy(x.astype(np.int32)).to(cuda_device)
    q_out = torch.full((total, Hq, d), 7.0, dtype=torch.bfloat16, device=cuda_device) if Hq else None
    args = dict(rope=rope, seq=i32(seq), rope_pos=i32(rp) if r else None, q_out=q_out, layout=layout)
    if e4m3:
        got = cw.paged_append_fp8(q if Hq else None, k, v, i32(pos), *pools, i32(tab), 0.02, 0.03, **args)
    else:
        got = cw.paged_append(q if Hq else None, k, v, i32(pos), *pools, i32(tab), **args)
    assert got is q_out
    fr = f.cpu().numpy() if r else None
    turn = (lambda x: orp.rope(x, rp, fr, sec, inter)) if r else (lambda x: x)
    kr, qr = turn(k64), turn(q64)
    row_seq = seq if seq is not None else np.arange(total)
    live = (pos >= 0) & (row_seq >= 0) & (row_seq < n_seq)
    if Hq:
        g = to64(q_out)
        assert (g[~live] == 7.0).all()
        assert_rotated(g[live], q64[live], qr[live], r, inter) if r else np.testing.assert_array_equal(g[live], q64[live])
    back = (lambda x: x.transpose(1, 2)) if layout == "bhtd" else (lambda x: x)
    want_at = {}
    for i in np.flatnonzero(live):
        for h in range(Hkv):
            if pos[i] >= cap:
                continue
            page = (tab[row_seq[i], h] if per_head else tab[row_seq[i]])[pos[i] // ps]
            if 0 <= page < n_pages:
                want_at[(int(page), int(pos[i] % ps), 0 if per_head else h)] = (i, h)
    for pool, was, new, scale in zip(pools, before, (kr, v64), (0.02, 0.03)):
        now, old = back(pool).cpu(), back(was).cpu().clone()
        idx = np.array(list(want_at)).reshape(-1, 3).T
        src = np.array(list(want_at.values())).reshape(-1, 2).T
        rows = new[src[0], src[1]]
        if e4m3:
            codes = f8.quantize_e4m3_f32(rows.astype(np.float32), scale)
            np.testing.assert_array_equal(now.numpy()[tuple(idx)], codes)
            old.numpy()[tuple(idx)] = codes
            np.testing.assert_array_equal(now.numpy(), old.numpy())
        else:
            have = now[tuple(torch.from_numpy(idx))]
            if new is kr and r:
                assert_rotated(to64(have)[:, None], k64[src[0], src[1]][:, None], rows[:, None], r, inter)
            else:
                np.testing.assert_array_equal(to64(have), rows)
            old[tuple(torch.from_numpy(idx))] = have
            assert torch.equal(now, old)


def test_append_rotates_queries_in_place(cuda_device):
    f = cw.rope_frequencies(128, device=cuda_device)
    q, k, v = (synth.cuda_normal_bf16((9, h, 128), synth.seed_of(n, 83), cuda_device) for n, h in (("q", 4), ("k", 2), ("v", 2)))
    pos = torch.arange(9, dtype=torch.int32, device=cuda_device)
    tab = torch.zeros((9, 1), dtype=torch.int32, device=cuda_device) + torch.arange(9, device=cuda_device, dtype=torch.int32)[:, None]
    kp, vp = (torch.zeros((9, 16, 2, 128), dtype=torch.bfloat16, device=cuda_device) for _ in range(2))
    want = cw.paged_append(q, k, v, pos, kp, vp, tab, rope=cw.Rope(f))
    got = cw.paged_append(q, k, v, pos, kp, vp, tab, rope=cw.Rope(f), q_out=q)
    assert got is q and torch.equal(q, want)


# ------------------------------------------------------------------------------------------ together
@pytest.mark.parametrize("per_head,layout,ps", [(False, "bhtd", 32), (True, "bthd", 16)])
def test_prompt_then_decode_steps(cuda_device, per_head, layout, ps):
    """A prompt written to pages, then tokens appended and decoded one by one, heads giving back the pages
    they no longer need: every step against the fp64 row of the whole sequence's attention."""
    B, Hq, Hkv, d, N0, steps = 2, 8, 2, 128, 200, 60
    pat = cw.Pattern(20, 40, 300, 2)
    f = cw.rope_frequencies(d, device=cuda_device)
    rope, fr = cw.Rope(f), f.cpu().numpy()
    N = N0 + steps
    (q64, q), (k64, k), (v64, v) = (host_and_device((B, N, h, d), n, cuda_device, 84)
                                    for n, h in (("q", Hq), ("k", Hkv), ("v", Hkv)))
    n = -(-N // ps)
    tab, n_pages = make_table(np.random.default_rng(84), B, n, heads=Hkv if per_head else None)
    shape = (n_pages, ps, 1 if per_head else Hkv, d) if layout == "bthd" else (n_pages, 1 if per_head else Hkv, ps, d)
    kp, vp = (torch.full(shape, float("nan"), dtype=torch.bfloat16, device=cuda_device) for _ in range(2))
    tabd = torch.from_numpy(tab).to(cuda_device)
    flat = lambda x: x[:, :N0].reshape(B * N0, -1, d)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    cw.paged_append(flat(q), flat(k), flat(v), i32(list(range(N0)) * B), kp, vp, tabd, rope=rope,
                    seq=i32([b for b in range(B) for _ in range(N0)]), layout=layout)
    turn = lambda x: np.stack([orp.rope(x[b], np.arange(N)[None], fr) for b in range(B)])
    # the cache holds bf16 keys and the queries are bf16: what the attention is computed on
    bf = lambda x: orc.bf16_bits_to_f64(synth.f32_to_bf16_bits(x.astype(np.float32)))
    qr, kr = bf(turn(q64)), bf(turn(k64))
    ws = ws_for("cowa_decode_paged", pat, B, Hq, Hkv, d, n, ps, cuda_device)
    for t in range(N0, N):
        pos = i32([t] * B)
        qt = cw.paged_append(q[:, t], k[:, t], v[:, t], pos, kp, vp, tabd, rope=rope, layout=layout)
        o, lse = cw.cowa_decode_paged(qt, kp, vp, tabd, pos, pat, layout=layout, workspace=ws)
        if per_head and t % 7 == 0:  # give pages back, and let somebody write to them
            for g, keep in enumerate(cw.pages_needed(pat, Hkv, ps, n, t + 1)):
                gone = tabd[:, g, torch.from_numpy(~keep).to(cuda_device)].long().reshape(-1)
                kp[gone[gone >= 0]] = float("nan")
                vp[gone[gone >= 0]] = float("inf")
                tabd[:, g, torch.from_numpy(~keep).to(cuda_device)] = -1
        # a key or query next to a rounding border may differ by a bf16 step from the oracle's
        c = lambda x: x[:, :t + 1].transpose(0, 2, 1, 3)
        go, gl = to64(o), lse.double().cpu().numpy()
        wo, wl = orc.decode(qr[:, t], c(kr), c(v64), [t] * B, oracle_pattern(pat))
        assert np.abs(go - wo).max() <= 2e-2, t
        assert np.abs(gl - wl).max() <= 1e-3, t
    assert cw.workspace_status(ws) == 0


def test_step_in_two_graphs_that_share_a_workspace(cuda_device):
    """append + decode captured twice, over two caches, with one workspace: replayed in turn, each gives
    the bits of the direct calls; and on a stream of their own, next to each other with two workspaces."""
    B, Hq, Hkv, d, ps, n = 4, 10, 2, 128, 32, 64
    pat = cw.Pattern(64, 300, 2048, 2)
    rope = cw.Rope(cw.rope_frequencies(d, device=cuda_device))
    pos = torch.tensor([2047, 31, 1000, -1], dtype=torch.int32, device=cuda_device)
    tab = torch.randperm(B * n, device=cuda_device).int().view(B, n)
    size = 1 << 23
    sets = []
    for x in range(2):
        r = lambda *s, nm: synth.cuda_normal_bf16(s, synth.seed_of(nm, 90 + x), cuda_device)
        sets.append(dict(q=r(B, Hq, d, nm="q"), k=r(B, Hkv, d, nm="k"), v=r(B, Hkv, d, nm="v"),
                         kp=r(B * n, ps, Hkv, d, nm="k_cache"), vp=r(B * n, ps, Hkv, d, nm="v_cache"),
                         qo=torch.zeros((B, Hq, d), dtype=torch.bfloat16, device=cuda_device),
                         o=torch.zeros((B, Hq, d), dtype=torch.bfloat16, device=cuda_device),
                         lse=torch.zeros((B, Hq), device=cuda_device),
                         ws=torch.zeros(size, dtype=torch.uint8, device=cuda_device)))

    def step(s, ws, stream=None):
        cw.paged_append(s["q"], s["k"], s["v"], pos, s["kp"], s["vp"], tab, rope=rope, q_out=s["qo"], stream=stream)
        cw.cowa_decode_paged(s["qo"], s["kp"], s["vp"], tab, pos, pat, out=s["o"], lse=s["lse"], workspace=ws, stream=stream)

    want = []
    for s in sets:
        step(s, s["ws"])
        torch.cuda.synchronize()
        want.append((s["o"].clone(), s["lse"].clone()))
    graphs = []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(s, sets[0]["ws"])
        graphs.append(g)
    for _ in range(3):
        for s in sets:
            s["o"].zero_(), s["lse"].zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for s, (o, lse) in zip(sets, want):
            assert torch.equal(s["o"], o) and torch.equal(s["lse"], lse)
    streams = [torch.cuda.Stream() for _ in sets]
    for s in sets:
        s["o"].zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for s, st in zip(sets, streams):
            step(s, s["ws"], st)
    torch.cuda.synchronize()
    for s, (o, lse) in zip(sets, want):
        assert torch.equal(s["o"], o) and torch.equal(s["lse"], lse)
        assert cw.workspace_status(s["ws"]) == 0
    # a workspace that the call allocates belongs to the call's stream
    o, lse = cw.cowa_decode_paged(sets[0]["qo"], sets[0]["kp"], sets[0]["vp"], tab, pos, pat, stream=streams[1])
    streams[1].synchronize()
    assert torch.equal(o, want[0][0]) and torch.equal(lse, want[0][1])


def test_refusals_of_the_binding(cuda_device):
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device=cuda_device)
    k = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device=cuda_device)
    pool = torch.zeros((6, 16, 2, 64), dtype=torch.bfloat16, device=cuda_device)
    tab = torch.zeros((2, 3), dtype=torch.int32, device=cuda_device)
    pos = torch.zeros(2, dtype=torch.int32, device=cuda_device)
    pat = cw.Pattern(4, 8, 48, 2)
    dec = lambda **c: cw.cowa_decode_paged(**{**dict(q_t=q, k_pages=pool, v_pages=pool, page_table=tab, pos=pos,
                                                     pattern=pat), **c})
    app = lambda **c: cw.paged_append(**{**dict(q=q, k=k, v=k, pos=pos, k_pages=pool, v_pages=pool, page_table=tab), **c})
    for bad in (dict(page_table=tab[:1]), dict(pos=pos[:1]), dict(layout="thbd"), dict(v_pages=pool[:5]),
                dict(page_table=torch.zeros((2, 2, 3), dtype=torch.int32, device=cuda_device)),
                dict(page_table=tab.t().contiguous().t()), dict(out=q[:1]), dict(lse=torch.zeros(2, 4)),
                dict(q_t=q.transpose(0, 1)), dict(lse=torch.zeros((2, 4), dtype=torch.float64, device=cuda_device))):
        with pytest.raises(ValueError):
            dec(**bad)
    for bad in (dict(pos=pos.long()), dict(page_table=tab.long()), dict(k_pages=pool.float()), dict(out=q.half())):
        with pytest.raises(TypeError):
            dec(**bad)
    with pytest.raises(cw.CowaError):
        dec(workspace=torch.zeros(300, dtype=torch.uint8, device=cuda_device))
    with pytest.raises(cw.CowaError):  # pages of 12 positions
        dec(k_pages=pool[:, :12].contiguous(), v_pages=pool[:, :12].contiguous())
    with pytest.raises(cw.CowaError):  # E4M3 needs d = 128
        cw.cowa_decode_paged_fp8(q, pool.to(torch.uint8), pool.to(torch.uint8), tab, pos, pat, 1.0, 1.0)
    for bad in (dict(v=k[:1]), dict(q=q[:1]), dict(pos=pos[:1]), dict(seq=pos[:1]), dict(q_out=q[:, :2]),
                dict(rope_pos=pos), dict(k_pages=pool[:, :, :1], v_pages=pool[:, :, :1])):
        with pytest.raises(ValueError):
            app(**bad)
    with pytest.raises(cw.CowaError):  # more rows than sequences, and no seq
        app(page_table=tab[:1])
    with pytest.raises(TypeError):
        app(v_pages=pool.half())


# ------------------------------------------------------------------------------------------ chunks
def assert_chunk(o, lse, q64, k, v, start, pat, has=None):
    """One sequence's rows o [n, Hq, d], lse [Hq, n] (CUDA) at positions start.. against k, v [Hkv, T, d]."""
    n, Hq, d = q64.shape
    Hkv, Tc = k.shape[0], k.shape[1]
    op = oracle_pattern(pat)
    go, gl = to64(o), lse.double().cpu().numpy()
    for g in range(Hkv):
        see = orc.visible_mask(np.arange(start, start + n), Tc, op, g, Hkv)
        if has is not None:
            see = see & has[g]
        for h in range(g * Hq // Hkv, (g + 1) * Hq // Hkv):
            s = np.where(see, q64[:, h] @ k[g].T * (pat.softmax_scale or 1 / np.sqrt(d)), -np.inf)
            m = np.where(see.any(1), s.max(1), 0.0)
            p = np.exp(s - m[:, None])
            l = p.sum(1)
            none = l == 0
            assert (go[none, h] == 0).all() and (gl[h, none] == -np.inf).all()
            l = np.where(none, 1.0, l)[:, None]
            want, A = p @ v[g] / l, p @ np.abs(v[g]) / l
            err = np.abs(go[:, h] - want)
            assert (err <= 2.0 ** -8 * (A + np.abs(want)) + 2.0 ** -12 * A).all(), (h, err.max())
            assert (np.abs(gl[h] - (m + np.log(l[:, 0])))[~none] <= LSE_TOL).all(), h


CHUNK = [
    # Hq, Hkv, d, pattern, page, pages, per head, layout, (start, rows) of each sequence
    (8, 4, 64, cw.Pattern(64, 128, 1024, 4), 16, 64, False, "bthd", [(824, 200)]),
    (10, 2, 128, cw.Pattern(20, 100, 900, 2), 64, 16, False, "bhtd", [(0, 1), (1000, 24), (500, 0), (37, 300), (0, 128)]),
    (3, 3, 128, cw.Pattern(0, 1, 1024, 3), 8, 96, True, "bthd", [(767, 1), (13, 130)]),       # single heads, L = 1
    (7, 1, 64, cw.Pattern(33, 5000, 600, 1), 24, 30, False, "bhtd", [(100, 257), (719, 1)]),  # dense, odd group
    (8, 2, 128, cw.Pattern(4, 60, 4, 1), 128, 8, False, "bthd", [(896, 128), (1, 127)]),      # sinks and band only
    (4, 2, 128, cw.Pattern(100, 7, 700, 2), 256, 3, True, "bhtd", [(301, 400)]),
    (6, 2, 64, cw.Pattern(30, 90, 1000, 4, kv_head_base=1, h_kv_global=4), 32, 32, False, "bthd", [(600, 333), (5, 5)]),
    (40, 8, 128, cw.Pattern(128, 500, 2048, 8), 48, 43, False, "bthd", [(1500, 500)]),
]


@pytest.mark.parametrize("Hq,Hkv,d,pat,ps,n,per_head,layout,chunks", CHUNK)
def test_chunks_match_oracle(cuda_device, Hq, Hkv, d, pat, ps, n, per_head, layout, chunks):
    """Packed chunks against their pages; rows past each sequence's last key hold NaN, rows of q behind the
    last sequence are left as they were, heads of their own map only what some row of the chunk sees."""
    B, rng = len(chunks), np.random.default_rng(ps * n)
    tab, n_pages = make_table(rng, B, n, heads=Hkv if per_head else None)
    shape = (n_pages, ps, 1 if per_head else Hkv, d)
    (k64, kd), (v64, vd) = (host_and_device(shape, x, cuda_device, 91) for x in ("k", "v"))
    k, _ = orp.gather_pages(k64, tab, n * ps)
    v, _ = orp.gather_pages(v64, tab, n * ps)
    for b, (start, rows) in enumerate(chunks):
        for s in range(start + rows, n * ps):
            page = tab[b, ..., s // ps]
            kd[torch.from_numpy(np.atleast_1d(page)).long().to(cuda_device), s % ps] = float("nan")
            vd[torch.from_numpy(np.atleast_1d(page)).long().to(cuda_device), s % ps] = float("inf")
        if per_head:
            for g in range(Hkv):
                see = orc.visible_mask(np.arange(start, start + rows), n * ps, oracle_pattern(pat), g, Hkv).any(0)
                tab[b, g, ~see.reshape(n, ps).any(1)] = -1
    if layout == "bhtd":
        kd, vd = kd.transpose(1, 2).contiguous(), vd.transpose(1, 2).contiguous()
    lens = [r for _, r in chunks]
    total = sum(lens) + 3
    q64, q = host_and_device((total, Hq, d), "q", cuda_device, 92)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    cu = np.cumsum([0] + lens)
    ws = torch.zeros(cw.lib().cowa_fwd_paged_workspace_size(ctypes.byref(pat.c()), B, total, Hq, Hkv, d, n, ps),
                     dtype=torch.uint8, device=cuda_device)
    out = torch.full((total, Hq, d), 3.0, dtype=torch.bfloat16, device=cuda_device)
    lse = torch.full((Hq, total), 5.0, device=cuda_device)
    o, l = cw.cowa_fwd_paged(q, kd, vd, torch.from_numpy(tab).to(cuda_device), i32(cu.tolist()),
                             i32([s for s, _ in chunks]), pat, layout=layout, out=out, lse=lse, workspace=ws)
    assert cw.workspace_status(ws) == 0
    assert o is out and (out[cu[-1]:] == 3.0).all() and (lse[:, cu[-1]:] == 5.0).all()
    for b, (start, rows) in enumerate(chunks):
        r = slice(cu[b], cu[b + 1])
        assert_chunk(o[r], l[:, r], q64[r], k[b, :, :start + rows], v[b, :, :start + rows], start, pat)


def test_chunks_equal_the_contiguous_forward(cuda_device):
    """Over pages of 128 in order the tiles and their masks are those of cowa_fwd_chunk: the same bits
    (with enough heads that the key tiles are not cut into parts)."""
    N, Hq, Hkv, d, start = 1100, 40, 8, 128, 640
    pat = cw.Pattern(64, 300, 1100, 8)
    k, v = (synth.cuda_normal_bf16((1, 1152, Hkv, d), synth.seed_of(x, 93), cuda_device) for x in ("k", "v"))
    q = synth.cuda_normal_bf16((1, N - start, Hq, d), synth.seed_of("q", 93), cuda_device)
    wo, wl = cw.cowa_fwd_chunk(q, k, v, pat, start, n_k=N)
    pages = lambda x: x.view(9, 128, Hkv, d)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    o, lse = cw.cowa_fwd_paged(q[0], pages(k), pages(v), i32([list(range(9))]), i32([0, N - start]), i32([start]), pat)
    assert torch.equal(o, wo[0]) and torch.equal(lse, wl[0])


@pytest.mark.parametrize("Hq", [2, 3, 4])
@pytest.mark.parametrize("ps", [16, 64])
def test_chunk_bad_entries_and_overlong_sequences(cuda_device, Hq, ps):
    """A bad entry leaves the query tiles (128 rows) that see a key of its page empty and is reported; the
    other tiles are not touched by it.  A chunk longer than the cache starts at 0, and its rows past the
    capacity see what there is (none, if the band has passed it); a start past the end is moved back."""
    Hkv, d, n = 1, 64, 320 // ps
    cap = n * ps
    pat = cw.Pattern(0, 40, 0, 1)
    tab, n_pages = make_table(np.random.default_rng(94), 4, n)
    tab[0, [64 // ps, 300 // ps]] = -1, n_pages
    tab[1, :] = 2**31 - 1
    (k64, kd), (v64, vd) = (host_and_device((n_pages, ps, Hkv, d), x, cuda_device, 94) for x in ("k", "v"))
    chunks = [(20, 240), (50, 70), (-5, cap + 90), (10**9, 30)]
    real = [(20, 240), (50, 70), (0, cap + 90), (cap - 30, 30)]
    lens = [r for _, r in chunks]
    cu = np.cumsum([0] + lens)
    q64, q = host_and_device((int(cu[-1]), Hq, d), "q", cuda_device, 94)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    ws = torch.zeros(1 << 23, dtype=torch.uint8, device=cuda_device)
    o, lse = cw.cowa_fwd_paged(q, kd, vd, torch.from_numpy(tab).to(cuda_device), i32(cu.tolist()),
                               i32([s for s, _ in chunks]), pat, workspace=ws)
    assert cw.workspace_status(ws) == 8 and cw.workspace_status(ws) == 0
    k, has = orp.gather_pages(k64, tab, cap)
    v, _ = orp.gather_pages(v64, tab, cap)
    empty = []
    for b, (start, rows) in enumerate(real):
        for i in range(0, rows, 128):
            m = min(128, rows - i)
            r = slice(cu[b] + i, cu[b] + i + m)
            see = orc.visible_mask(np.arange(start + i, start + i + m), cap, oracle_pattern(pat), 0, 1).any(0)
            ok = np.full((1, cap), (see <= has[b, 0]).all())
            empty.append(not ok.all())
            assert_chunk(o[r], lse[:, r], q64[r], k[b], v[b], start + i, pat, ok)
    # (with pages of 64 the second tile of sequence 0 sees both bad entries' pages, with 16 neither)
    assert empty == [True, ps == 64, True] + [False] * (len(empty) - 3)


@pytest.mark.parametrize("n_seq", [33, 64, 65, 150])
def test_chunks_of_many_sequences(cuda_device, n_seq):
    """However many sequences a call has (their tiles are dealt out in other orders then), some of them
    empty, some a single row."""
    Hq, Hkv, d, ps, n = 3, 1, 64, 16, 40
    pat = cw.Pattern(30, 100, 640, 1)
    rng = np.random.default_rng(n_seq)
    lens = [int(x) for x in rng.choice([0, 0, 1, 2, 17, 128, 129, 300], n_seq)]
    starts = [int(rng.integers(0, n * ps - x + 1)) for x in lens]
    (k64, kp), (v64, vp) = (host_and_device((500, ps, Hkv, d), x, cuda_device, 96) for x in ("k", "v"))
    tabh = rng.integers(0, 500, (n_seq, n)).astype(np.int32)
    tab = torch.from_numpy(tabh).to(cuda_device)
    total = max(1, sum(lens))
    q64, q = host_and_device((total, Hq, d), "q", cuda_device, 96)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    cu = np.cumsum([0] + lens)
    ws = torch.zeros(1 << 23, dtype=torch.uint8, device=cuda_device)
    o, lse = cw.cowa_fwd_paged(q, kp, vp, tab, i32(cu.tolist()), i32(starts), pat, workspace=ws)
    assert cw.workspace_status(ws) == 0
    for s in range(n_seq):
        if lens[s] == 0:
            continue
        r = slice(cu[s], cu[s + 1])
        k, _ = orp.gather_pages(k64, tabh[s:s + 1], starts[s] + lens[s])
        v, _ = orp.gather_pages(v64, tabh[s:s + 1], starts[s] + lens[s])
        assert_chunk(o[r], lse[:, r], q64[r], k[0], v[0], starts[s], pat)


@pytest.mark.parametrize("Hq,Hkv,d,rows", [(5, 1, 128, 3), (4, 2, 64, 130), (8, 1, 128, 1)])
def test_short_chunks_behind_long_prefixes(cuda_device, Hq, Hkv, d, rows):
    """A few rows against thousands of keys: the key tiles are cut into parts that several CTAs take."""
    ps, n = 64, 100
    pat = cw.Pattern(100, 900, 6400, Hkv)
    rng = np.random.default_rng(98)
    tab, n_pages = make_table(rng, 2, n)
    (k64, kp), (v64, vp) = (host_and_device((n_pages, ps, Hkv, d), x, cuda_device, 98) for x in ("k", "v"))
    starts, lens = [6000, 77], [rows, 2 * rows]
    total = sum(lens) + 4
    q64, q = host_and_device((total, Hq, d), "q", cuda_device, 98)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    size = lambda pages: cw.lib().cowa_fwd_paged_workspace_size(ctypes.byref(pat.c()), 2, total, Hq, Hkv, d, pages, ps)
    assert size(n) > 256 + 8 * total * Hq * d > size(2)  # (the cut needs room for its parts)
    out, lse = torch.full_like(q, 3.0), torch.full((Hq, total), 5.0, device=cuda_device)
    ws = torch.zeros(size(n), dtype=torch.uint8, device=cuda_device)
    run = lambda: cw.cowa_fwd_paged(q, kp, vp, torch.from_numpy(tab).to(cuda_device), i32([2, 2 + rows, 2 + 3 * rows]),
                                    i32(starts), pat, out=out, lse=lse, workspace=ws)
    run()
    assert cw.workspace_status(ws) == 0
    first = out.clone(), lse.clone()
    run()
    assert torch.equal(first[0], out) and torch.equal(first[1], lse)
    for r in (slice(0, 2), slice(2 + 3 * rows, total)):  # rows of no sequence
        assert (out[r] == 3.0).all() and (lse[:, r] == 5.0).all()
    row = 2
    for b in range(2):
        k, _ = orp.gather_pages(k64, tab[b:b + 1], starts[b] + lens[b])
        v, _ = orp.gather_pages(v64, tab[b:b + 1], starts[b] + lens[b])
        r = slice(row, row + lens[b])
        assert_chunk(out[r], lse[:, r], q64[r], k[0], v[0], starts[b], pat)
        row += lens[b]


def test_chunk_offsets_are_clamped(cuda_device):
    """A malformed cu_seqlens: sequences in order, disjoint and inside the rows, as for cowa_fwd_varlen."""
    Hq, Hkv, d, ps, n = 2, 1, 64, 16, 20
    pat = cw.Pattern(8, 30, 320, 1)
    kp, vp = (synth.cuda_normal_bf16((60, ps, Hkv, d), synth.seed_of(x, 97), cuda_device) for x in ("k", "v"))
    q = synth.cuda_normal_bf16((100, Hq, d), synth.seed_of("q", 97), cuda_device)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    tab = torch.arange(80, device=cuda_device).int().view(4, n) % 60
    start = i32([10, 20, 30, 40])
    run = lambda cu: cw.cowa_fwd_paged(q, kp, vp, tab, i32(cu), start, pat, out=torch.zeros_like(q),
                                       lse=torch.zeros((Hq, 100), device=cuda_device))
    for bad, good in (([-5, 30, 20, 70, 500], [0, 30, 30, 70, 100]), ([200, 1, 2, 3, 4], [100] * 5)):
        (o, lse), (wo, wl) = run(bad), run(good)
        assert torch.equal(o, wo) and torch.equal(lse, wl)


def test_chunk_graph_stream_and_refusals(cuda_device):
    Hq, Hkv, d, ps, n = 4, 2, 64, 32, 16
    pat = cw.Pattern(16, 60, 512, 2)
    r = lambda s, nm: synth.cuda_normal_bf16(s, synth.seed_of(nm, 95), cuda_device)
    q, kp, vp = r((200, Hq, d), "q"), r((2 * n, ps, Hkv, d), "k"), r((2 * n, ps, Hkv, d), "v")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    tab, cu, start = torch.randperm(2 * n, device=cuda_device).int().view(2, n), i32([0, 150, 200]), i32([300, 0])
    wo, wl = cw.cowa_fwd_paged(q, kp, vp, tab, cu, start, pat)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, lse = cw.cowa_fwd_paged(q, kp, vp, tab, cu, start, pat, stream=side)
    side.synchronize()
    assert torch.equal(o, wo) and torch.equal(lse, wl)
    ws = torch.zeros(1 << 23, dtype=torch.uint8, device=cuda_device)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cw.cowa_fwd_paged(q, kp, vp, tab, cu, start, pat, out=o, lse=lse, workspace=ws)
    o.zero_(), lse.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, wo) and torch.equal(lse, wl)
    run = lambda **c: cw.cowa_fwd_paged(**{**dict(q=q, k_pages=kp, v_pages=vp, page_table=tab, cu_seqlens=cu,
                                                  q_start=start, pattern=pat), **c})
    for bad in (dict(cu_seqlens=cu[:2]), dict(q_start=cu), dict(out=o[:5]), dict(lse=lse[:, :5]), dict(layout="hd"),
                dict(v_pages=vp[:3]), dict(page_table=tab.view(2, 4, 4))):
        with pytest.raises(ValueError):
            run(**bad)
    for bad in (dict(q=q.half()), dict(q_start=start.long()), dict(k_pages=kp.to(torch.uint8))):
        with pytest.raises(TypeError):
            run(**bad)
    with pytest.raises(cw.CowaError):
        run(workspace=torch.zeros(128, dtype=torch.uint8, device=cuda_device))


# ------------------------------------------------------------------------------------------ large pools, debug build
@pytest.mark.parametrize("e4m3", [False, True])
def test_pools_past_32_bit_offsets(cuda_device, e4m3):
    """Pages whose elements (and bytes) lie past 2^32: written, decoded, and read by a chunk."""
    Hq, Hkv, d, ps = 4, 4, 128, 64
    n_pages = (1 << 32) // (ps * Hkv * d) + 40  # 8.6 GB of bf16, 4.3 GB of codes
    pat = cw.Pattern(8, 100, 200, 4)
    dt = torch.uint8 if e4m3 else torch.bfloat16
    kp, vp = (torch.empty((n_pages, ps, Hkv, d), dtype=dt, device=cuda_device) for _ in range(2))
    tab = torch.tensor([[n_pages - 1, 0, n_pages - 7, n_pages - 30]], dtype=torch.int32, device=cuda_device)
    N = 4 * ps
    (k64, k), (v64, v) = (host_and_device((N, Hkv, d), x, cuda_device, 99) for x in ("k", "v"))
    q64, q = host_and_device((1, Hq, d), "q", cuda_device, 99)
    pos = torch.arange(N, dtype=torch.int32, device=cuda_device)
    seq = torch.zeros(N, dtype=torch.int32, device=cuda_device)
    one = torch.tensor([N - 1], dtype=torch.int32, device=cuda_device)
    if e4m3:
        cw.paged_append_fp8(None, k, v, pos, kp, vp, tab, 1 / 64, 1 / 64, seq=seq)
        o, lse = cw.cowa_decode_paged_fp8(q, kp, vp, tab, one, pat, 1 / 64, 1 / 64)
        k64, v64 = (f8.e4m3_to_f64(f8.quantize_e4m3_f32(x.astype(np.float32), 1 / 64)) / 64 for x in (k64, v64))
    else:
        cw.paged_append(None, k, v, pos, kp, vp, tab, seq=seq)
        o, lse = cw.cowa_decode_paged(q, kp, vp, tab, one, pat)
    assert_decoded(o, lse, q64, k64.transpose(1, 0, 2)[None], v64.transpose(1, 0, 2)[None], [N - 1], pat,
                   2.0 ** -11 if e4m3 else 2.0 ** -8)
    if not e4m3:
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
        o, lse = cw.cowa_fwd_paged(q, kp, vp, tab, i32([0, 1]), i32([N - 1]), pat)
        assert_chunk(o, lse, q64, k64.transpose(1, 0, 2), v64.transpose(1, 0, 2), N - 1, pat)


def test_debug_build_gives_the_same_bits(cuda_device):
    from structured_sparse_attention_cowa_b200 import build as cbuild

    B, Hq, Hkv, d, ps, n = 3, 10, 2, 128, 24, 40
    pat = cw.Pattern(20, 100, 900, 2)
    rope = cw.Rope(cw.rope_frequencies(d, device=cuda_device))
    tab = torch.randperm(B * n, device=cuda_device).int().view(B, n)
    r = lambda s, nm: synth.cuda_normal_bf16(s, synth.seed_of(nm, 100), cuda_device)
    q, k, v = r((B, Hq, d), "q"), r((B, Hkv, d), "k"), r((B, Hkv, d), "v")
    pools = r((B * n, ps, Hkv, d), "k_cache"), r((B * n, ps, Hkv, d), "v_cache")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    pos = i32([900, 31, -1])

    def step():
        kp, vp = (p.clone() for p in pools)
        ws = torch.zeros(1 << 23, dtype=torch.uint8, device=cuda_device)
        qr = cw.paged_append(q, k, v, pos, kp, vp, tab, rope=rope, q_out=torch.zeros_like(q))
        out = [qr, kp, vp, *cw.cowa_decode_paged(qr, kp, vp, tab, pos, pat, workspace=ws),
               *cw.cowa_fwd_paged(qr, kp, vp, tab, i32([0, 1, 1, 3]), i32([900, 0, 5]), pat, workspace=ws)]
        assert cw.workspace_status(ws) == 0
        return out

    want = step()
    saved = cw._lib, cw.LIB_PATH
    cw._lib, cw.LIB_PATH = None, cbuild.build(debug=True)
    try:
        got = step()
    finally:
        cw._lib, cw.LIB_PATH = saved
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("wide", [False, True])
def test_chained_calls_without_waits(cuda_device, wide):
    """Each call reads what the one before it in the stream wrote, with nothing in between (the kernels are
    set up while the one before runs): the same bits as with the GPU waited for after every call."""
    B, Hq, Hkv, d, ps, n = 6, 4, 2, 128, 32, 20
    pat, rope = cw.Pattern(16, 100, 640, 2), cw.Rope(cw.rope_frequencies(d, device=cuda_device))
    tabh = np.random.default_rng(101).permutation(B * n).astype(np.int32).reshape(B, n)
    if wide:
        pat, tabh = widened(pat, tabh, ps)
    tab = torch.from_numpy(tabh).to(cuda_device)
    pools = [synth.cuda_normal_bf16((B * n, ps, Hkv, d), synth.seed_of(x, 101), cuda_device) for x in ("k_cache", "v_cache")]
    first = synth.cuda_normal_bf16((B, Hq, d), synth.seed_of("q", 101), cuda_device)
    steps = [torch.tensor([(37 * i + 101 * b) % 600 for b in range(B)], dtype=torch.int32, device=cuda_device)
             for i in range(40)]
    cu = torch.arange(B + 1, dtype=torch.int32, device=cuda_device)

    def run(wait):
        kp, vp = (p.clone() for p in pools)
        ws = torch.zeros(1 << 23, dtype=torch.uint8, device=cuda_device)
        x, qo, o = first.clone(), torch.empty_like(first), torch.empty_like(first)
        lse, lse2 = torch.empty((B, Hq), device=cuda_device), torch.empty((Hq, B), device=cuda_device)
        calls = (lambda p: cw.paged_append(x, x[:, :Hkv], x[:, Hkv:], p, kp, vp, tab, rope=rope, q_out=qo),
                 lambda p: cw.cowa_decode_paged(qo, kp, vp, tab, p, pat, out=o, lse=lse, workspace=ws),
                 lambda p: cw.cowa_fwd_paged(o, kp, vp, tab, cu, p, pat, out=qo, lse=lse2, workspace=ws),
                 lambda p: cw.cowa_rope(qo[None], None, rope, p[None], q_out=x[None]))
        torch.cuda.synchronize()
        for p in steps:
            for call in calls:
                call(p)
                if wait:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert cw.workspace_status(ws) == 0
        return x, o, lse, kp, vp

    for a, b in zip(run(True), run(False)):
        assert torch.isfinite(a.float()).all() and torch.equal(a, b)


def test_workspace_in_pieces_is_refused(cuda_device):
    """A workspace whose elements are not one piece of memory would be smaller, or in other places, than its
    element count says."""
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device=cuda_device)
    pool = torch.zeros((6, 16, 2, 64), dtype=torch.bfloat16, device=cuda_device)
    tab = torch.zeros((2, 3), dtype=torch.int32, device=cuda_device)
    pos = torch.zeros(2, dtype=torch.int32, device=cuda_device)
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device=cuda_device)
    pat = cw.Pattern(4, 8, 48, 2)
    one = torch.zeros(1, dtype=torch.uint8, device=cuda_device)
    for ws in (one.expand(1 << 24), torch.zeros(1 << 24, dtype=torch.uint8, device=cuda_device)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            cw.cowa_decode_paged(q, pool, pool, tab, pos, pat, workspace=ws)
        with pytest.raises(ValueError, match="workspace"):
            cw.cowa_fwd_paged(q, pool, pool, tab, cu, pos, pat, workspace=ws)


def test_status_of_workspaces_of_other_calls(cuda_device):
    """Only the status word had to be cleared before there were paged calls: whatever else the header of such
    a workspace holds is not a bad page."""
    ws = torch.full((256,), 0x5A, dtype=torch.uint8, device=cuda_device)
    ws[:4] = 0
    assert cw.workspace_status(ws) == 0
    ws[12:16] = torch.tensor([1, 0, 0, 0], dtype=torch.uint8, device=cuda_device)
    assert cw.workspace_status(ws) == 0


@pytest.mark.parametrize("Hq,Hkv,pat,chunks", [
    # up to 64 (head, sequence)s, odd groups, intervals that some rows see in part
    (24, 8, cw.Pattern(40, 200, 2500, 8), [(1900, 700), (0, 1), (130, 513), (2700, 90)]),
    # .. repeated intervals of other ranks' heads, one sequence
    (30, 6, cw.Pattern(0, 64, 2000, 4, kv_head_base=3, h_kv_global=12), [(700, 1300)]),
    # .. 64 of them, most empty; a band longer than the cache, no long-range region
    (24, 8, cw.Pattern(100, 2**31 - 1, 100, 1), [(0, 900), (1500, 0), (0, 0), (77, 300), (5, 2), (1, 0), (0, 0), (2000, 200)]),
    # more: sequences by their positions
    (24, 8, cw.Pattern(40, 200, 2500, 8), [(1200, 300), (0, 1), (130, 129), (2700, 90)] + [(3, 20)] * 5),
])
def test_chunks_of_more_work_than_the_gpu_holds(cuda_device, Hq, Hkv, pat, chunks):
    """Calls of more than 148 (query tile, pair of heads)s, which are dealt out by their weight: each is
    computed, once."""
    d, ps, n = 64, 64, 44
    lens, B = [r for _, r in chunks], len(chunks)
    rng = np.random.default_rng(98)
    (k64, kp), (v64, vp) = (host_and_device((120, ps, Hkv, d), x, cuda_device, 98) for x in ("k", "v"))
    tabh = rng.integers(0, 120, (B, n)).astype(np.int32)
    total = sum(lens)
    assert (total // 128 + B) * Hkv * ((Hq // Hkv + 1) // 2) > 148
    q64, q = host_and_device((total, Hq, d), "q", cuda_device, 98)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    cu = np.cumsum([0] + lens)
    ws = torch.zeros(1 << 24, dtype=torch.uint8, device=cuda_device)
    out = torch.full((total, Hq, d), float("nan"), dtype=torch.bfloat16, device=cuda_device)
    o, lse = cw.cowa_fwd_paged(q, kp, vp, torch.from_numpy(tabh).to(cuda_device), i32(cu.tolist()),
                               i32([s for s, _ in chunks]), pat, out=out, workspace=ws)
    assert cw.workspace_status(ws) == 0
    for s, (start, rows) in enumerate(chunks):
        if rows == 0:
            continue
        r = slice(cu[s], cu[s + 1])
        k, _ = orp.gather_pages(k64, tabh[s:s + 1], start + rows)
        v, _ = orp.gather_pages(v64, tabh[s:s + 1], start + rows)
        assert_chunk(o[r], lse[:, r], q64[r], k[0], v[0], start, pat)


@pytest.mark.parametrize("Hq,Hkv,d,T,parts,chunks", [
    (20, 4, 64, 1000, 1, [(1200, 500), (1900, 380)]),                             # single heads, taking turns
    (3, 1, 64, 1000, 6, [(2000, 200), (0, 1), (700, 0), (300, 140), (2600, 5)]),  # single heads, cut
    (8, 1, 128, 1000, 2, [(1500, 1279)]),                                         # single heads, cut, taking turns
    (20, 4, 64, 1000, 2, [(2600, 100), (0, 50), (9, 0), (9, 1), (1000, 27), (2222, 60), (40, 40)]),  # pairs, the same
])
def test_chunks_in_other_cuts(cuda_device, Hq, Hkv, d, T, parts, chunks):
    """Calls whose CTAs take single heads, or parts of the key tiles, or both, and where these take turns on the
    GPU; then with a bad page under the first sequence's sinks, which empties that sequence alone."""
    ps, n, pat = 64, 44, cw.Pattern(100, 2000, T, 1)
    lens, B = [r for _, r in chunks], len(chunks)
    rng = np.random.default_rng(99)
    (k64, kp), (v64, vp) = (host_and_device((120, ps, Hkv, d), x, cuda_device, 99) for x in ("k", "v"))
    tabh = rng.integers(0, 120, (B, n)).astype(np.int32)
    total = sum(lens)
    size = cw.lib().cowa_fwd_paged_workspace_size(ctypes.byref(pat.c()), B, total, Hq, Hkv, d, n, ps)
    per_part = Hq * total * (d + 2) * 4  # (and the alignment of what each part keeps)
    assert 0 <= size - 256 - (parts > 1) * parts * per_part < 256
    q64, q = host_and_device((total, Hq, d), "q", cuda_device, 99)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    cu = np.cumsum([0] + lens)
    ws = torch.zeros(size, dtype=torch.uint8, device=cuda_device)
    run = lambda tab: cw.cowa_fwd_paged(q, kp, vp, torch.from_numpy(tab).to(cuda_device), i32(cu.tolist()),
                                        i32([s for s, _ in chunks]), pat, workspace=ws)
    o, lse = run(tabh)
    assert cw.workspace_status(ws) == 0
    for s, (start, rows) in enumerate(chunks):
        if rows == 0:
            continue
        r = slice(cu[s], cu[s + 1])
        k, _ = orp.gather_pages(k64, tabh[s:s + 1], start + rows)
        v, _ = orp.gather_pages(v64, tabh[s:s + 1], start + rows)
        assert_chunk(o[r], lse[:, r], q64[r], k[0], v[0], start, pat)
    bad = tabh.copy()
    bad[0, 0] = 120
    ob, lb = run(bad)
    assert cw.workspace_status(ws) == 8
    assert (ob[:cu[1]] == 0).all() and (lb[:, :cu[1]] == -float("inf")).all()
    assert torch.equal(ob[cu[1]:], o[cu[1]:]) and torch.equal(lb[:, cu[1]:], lse[:, cu[1]:])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("total,Hq,Hkv", [(2400, 40, 8), (1822, 8, 1), (4003, 0, 2)])
def test_tokens_are_appended_alike_however_many(cuda_device, total, Hq, Hkv, e4m3):
    """How many tokens a block owns depends on the call's size: the same queries and pages as from calls of 100
    tokens."""
    d, ps = 128, 16
    n = (total + ps - 1) // ps
    rope = cw.Rope(cw.rope_frequencies(96, device=cuda_device))
    _, qkv = host_and_device((total, Hq + 2 * Hkv, d), "q", cuda_device, 83)
    q, k, v = qkv.split([Hq, Hkv, Hkv], dim=1)
    i32 = lambda x: torch.from_numpy(x.astype(np.int32)).to(cuda_device)
    rng = np.random.default_rng(84)
    tab, pos, seq = i32(rng.permutation(n)[None]), i32(rng.permutation(total)), i32(np.zeros(total))
    pools = [torch.zeros((n, ps, Hkv, d), dtype=torch.uint8 if e4m3 else torch.bfloat16, device=cuda_device) for _ in range(4)]
    fn, scales = (cw.paged_append_fp8, (0.02, 0.03)) if e4m3 else (cw.paged_append, ())
    put = lambda s, kp, vp: fn(q[s] if Hq else None, k[s], v[s], pos[s], kp, vp, tab, *scales, rope=rope, seq=seq[s])
    got = put(slice(0, total), *pools[:2])
    parts = [put(slice(i, i + 100), *pools[2:]) for i in range(0, total, 100)]
    assert got is None if Hq == 0 else torch.equal(got, torch.cat(parts))
    assert torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3]) and pools[0].any()
