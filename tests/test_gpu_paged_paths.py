"""GPU parity of the paged calls where a call takes another way through the code than the cases of
test_gpu_paged: rotary dimensions that are no whole units of 8 pairs (written as bf16 and as E4M3 codes), more KV
heads than travel with a kernel's arguments, more (sequence, head) pairs than the threads of a block keep at
hand; and the contiguous calls and whole serving steps held to the derived bounds of test_gpu_paged."""

import numpy as np
import pytest
import torch

import tests.test_gpu_paged as tp
from oracle import fp8_kv as f8
from oracle import rope as orp
from structured_sparse_attention_cowa_b200 import cowa as cw
from structured_sparse_attention_cowa_b200 import synth
from tests.gpu_helpers import host_and_device, to64
from tests.test_gpu_rope import assert_rotated

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv,r,sec,inter,ps,n,per_head,layout", [
    (8, 2, 22, (11,), False, 16, 6, False, "bthd"),      # halves of 11 pairs: pieces through shared memory
    (5, 1, 26, (6, 7), False, 24, 5, True, "bhtd"),
    (6, 2, 20, (7, 3), True, 8, 12, False, "bhtd"),      # neighbours, r = 4 mod 8
    (4, 4, 126, (63,), False, 16, 6, False, "bthd"),
    (8, 2, 40, (20,), True, 16, 6, False, "bthd"),       # neighbours, the last unit half rotated
    (3, 3, 72, (12, 12, 12), True, 32, 4, True, "bthd"),
    (0, 2, 8, (4,), True, 16, 6, False, "bhtd"),         # half a unit, no queries
    (2, 1, 2, (1,), False, 16, 6, False, "bthd"),        # one pair
])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("chunks", [False, True])
def test_append_of_odd_rotary_dimensions(cuda_device, Hq, Hkv, r, sec, inter, ps, n, per_head, layout, e4m3, chunks):
    tp.test_append_matches_oracle(cuda_device, Hq, Hkv, 128, r, sec, inter, ps, n, per_head, layout, e4m3, chunks)


MANY_HEADS = [
    # Hq, Hkv, d, pattern, page, pages, per head, layout
    (66, 66, 64, cw.Pattern(20, 50, 700, 6), 16, 48, False, "bthd"),
    (130, 65, 128, cw.Pattern(0, 9, 768, 65), 24, 32, True, "bhtd"),
    (140, 70, 128, cw.Pattern(33, 100, 500, 7, kv_head_base=10, h_kv_global=140), 32, 24, False, "bhtd"),
]


@pytest.mark.parametrize("Hq,Hkv,d,pat,ps,n,per_head,layout", MANY_HEADS)
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("wide", [False, True])
def test_decode_of_many_heads(cuda_device, Hq, Hkv, d, pat, ps, n, per_head, layout, e4m3, wide):
    """More than 64 KV heads, whose intervals are worked out on the device."""
    if e4m3 and d != 128:
        pytest.skip("E4M3 pages need d = 128")
    tp.test_decode_matches_oracle(cuda_device, Hq, Hkv, d, pat, ps, n, per_head, layout, [767, 300, -1], e4m3, wide)


@pytest.mark.parametrize("Hq,Hkv,d,pat,ps,n,per_head,layout", MANY_HEADS)
def test_chunks_of_many_heads(cuda_device, Hq, Hkv, d, pat, ps, n, per_head, layout):
    tp.test_chunks_match_oracle(cuda_device, Hq, Hkv, d, pat, ps, n, per_head, layout, [(500, 200), (0, 3), (766, 2)])


@pytest.mark.parametrize("B,Hq,Hkv,d,e4m3", [
    (100, 16, 8, 64, False),    # 800 pairs: five a thread
    (90, 24, 8, 128, True),     # groups of 3
    (128, 48, 8, 128, True),    # groups of 6
    (401, 2, 2, 128, False),    # 802
    (2000, 1, 1, 64, False),    # 13 a thread
    (81, 8, 8, 128, False),     # 648
])
def test_decode_of_many_pairs(cuda_device, B, Hq, Hkv, d, e4m3):
    """More than 640 (sequence, KV head)s: lengths from none to some hundreds, runs of empty slots at the start, in
    the middle and at the end, one long sequence that many blocks share; every row against the oracle, and the
    same bits again."""
    ps, n, n_pages = 16, 600, 700
    pat = cw.Pattern(10, 60, 9600, Hkv)
    rng = np.random.default_rng(B)
    pos = [int(x) for x in np.where(rng.random(B) < 0.2, -1, rng.integers(0, 300, B))]
    for i in (0, 1, 2, *range(B // 2, B // 2 + 7), B - 2, B - 1):
        pos[i] = -1
    pos[B // 3] = n * ps - 1
    pos[B // 3 + 1] = 0
    tab = rng.integers(0, n_pages, (B, n)).astype(np.int32)
    shape = (n_pages, ps, Hkv, d)
    if e4m3:
        kc, vc = (f8.f64_to_e4m3(rng.standard_normal(shape) * 3) for _ in range(2))
        kd, vd = torch.from_numpy(kc).to(cuda_device), torch.from_numpy(vc).to(cuda_device)
        k64, v64 = 0.4 * f8.e4m3_to_f64(kc), 0.25 * f8.e4m3_to_f64(vc)
    else:
        (k64, kd), (v64, vd) = (host_and_device(shape, x, cuda_device, 141) for x in ("k", "v"))
    q64, q = host_and_device((B, Hq, d), "q", cuda_device, 141)
    fn = "cowa_decode_paged_fp8" if e4m3 else "cowa_decode_paged"
    ws = tp.ws_for(fn, pat, B, Hq, Hkv, d, n, ps, cuda_device)
    run = lambda: getattr(cw, fn)(q, kd, vd, torch.from_numpy(tab).to(cuda_device),
                                  torch.tensor(pos, dtype=torch.int32, device=cuda_device), pat,
                                  *((0.4, 0.25) if e4m3 else ()), workspace=ws)
    assert B * Hkv > 640
    o, lse = run()
    o2, lse2 = run()
    assert cw.workspace_status(ws) == 0
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    for b in range(B):
        t = max(pos[b], 0) + 1
        k, v = (orp.gather_pages(x, tab[b:b + 1], t)[0] for x in (k64, v64))
        tp.assert_decoded(o[b:b + 1], lse[b:b + 1], q64[b:b + 1], k, v, [pos[b]], pat, 2.0 ** -11 if e4m3 else 2.0 ** -8)


def test_decode_and_the_contiguous_decode_within_the_derived_bound(cuda_device):
    """The same keys in pages and in one array per sequence: each within the bound of its roundings."""
    B, Hq, Hkv, d, Tc, ps = 3, 10, 2, 128, 2048, 64
    pat, pos = cw.Pattern(64, 300, 2048, 2), [2047, 1000, 3]
    (k64, kc), (v64, vc) = (host_and_device((B, Hkv, Tc, d), x, cuda_device, 142) for x in ("k", "v"))
    q64, q = host_and_device((B, Hq, d), "q", cuda_device, 142)
    posd = torch.tensor(pos, dtype=torch.int32, device=cuda_device)
    pages = lambda x: x.view(B, Hkv, Tc // ps, ps, d).permute(0, 2, 1, 3, 4).reshape(-1, Hkv, ps, d).contiguous()
    tab = torch.arange(B * Tc // ps, dtype=torch.int32, device=cuda_device).view(B, -1)
    for o, lse in (cw.cowa_decode_paged(q, pages(kc), pages(vc), tab, posd, pat, layout="bhtd"),
                   cw.cowa_decode(q, kc, vc, posd, pat)):
        tp.assert_decoded(o, lse, q64, k64, v64, pos, pat)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("per_head,layout,ps", [(False, "bhtd", 32), (True, "bthd", 16), (True, "bhtd", 24)])
def test_serving_steps_within_the_derived_bounds(cuda_device, per_head, layout, ps, e4m3):
    """A prompt written to pages in two chunks (bf16: the second's rows attend to both), then steps of append and
    decode, heads giving pages back to another sequence that overwrites them.  What the pages hold is the rotated
    keys and the values; what the attention gives is right for exactly what the pages and the queries hold."""
    B, Hq, Hkv, d, N0, steps = 2, 8, 2, 128, 200, 40
    pat = cw.Pattern(20, 40, 300, 2)
    f = cw.rope_frequencies(d, device=cuda_device)
    rope, fr = cw.Rope(f), f.cpu().numpy()
    N = N0 + steps
    (q64, q), (k64, k), (v64, v) = (host_and_device((B, N, h, d), x, cuda_device, 143)
                                    for x, h in (("q", Hq), ("k", Hkv), ("v", Hkv)))
    n = -(-N // ps)
    tab, n_pages = tp.make_table(np.random.default_rng(143), B, n, heads=Hkv if per_head else None)
    shape = (n_pages, ps, 1 if per_head else Hkv, d) if layout == "bthd" else (n_pages, 1 if per_head else Hkv, ps, d)
    ks, vs = 0.02, 0.03
    kp, vp = (torch.full(shape, 0x7f if e4m3 else float("nan"), dtype=torch.uint8 if e4m3 else torch.bfloat16,
                         device=cuda_device) for _ in range(2))
    tabd = torch.from_numpy(tab).to(cuda_device)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)

    def append(q, k, v, pos, seq=None):
        rest = dict(rope=rope, seq=None if seq is None else i32(seq), layout=layout)
        if e4m3:
            return cw.paged_append_fp8(q, k, v, i32(pos), kp, vp, tabd, ks, vs, **rest)
        return cw.paged_append(q, k, v, i32(pos), kp, vp, tabd, **rest)

    def held(t):  # keys, values 0 .. t as the pages hold them, and which have a page
        out = []
        for pool, scale in ((kp, ks), (vp, vs)):
            x = pool.transpose(1, 2) if layout == "bhtd" else pool
            x = scale * f8.e4m3_to_f64(x.cpu().numpy()) if e4m3 else to64(x)
            out.append(orp.gather_pages(x, tabd.cpu().numpy(), t + 1)[0])
        return out

    turned = lambda x, p: np.stack([orp.rope(x[b], np.asarray(p)[None], fr) for b in range(B)])
    first, last = 130, N0
    for lo, hi in ((0, first), (first, last)):
        flat = lambda x: x[:, lo:hi].reshape(B * (hi - lo), -1, d)
        qr = append(flat(q), flat(k), flat(v), list(range(lo, hi)) * B, [b for b in range(B) for _ in range(lo, hi)])
        assert_rotated(to64(qr).reshape(B * (hi - lo), Hq, d), q64[:, lo:hi].reshape(-1, Hq, d),
                       turned(q64[:, lo:hi], np.arange(lo, hi)).reshape(-1, Hq, d), d, False)
    hk, hv = held(N0 - 1)
    want_k = turned(k64[:, :N0], np.arange(N0)).transpose(0, 2, 1, 3)
    want_v = v64[:, :N0].transpose(0, 2, 1, 3)
    if e4m3:
        code = lambda x, s: s * f8.e4m3_to_f64(f8.quantize_e4m3_f32(x.astype(np.float32), s))
        np.testing.assert_array_equal(hk, code(want_k, ks))
        np.testing.assert_array_equal(hv, code(want_v, vs))
    else:
        flat = lambda x: x.reshape(-1, 1, d)
        assert_rotated(flat(hk), flat(k64[:, :N0].transpose(0, 2, 1, 3)), flat(want_k), d, False)
        np.testing.assert_array_equal(hv, want_v)
        o, lse = cw.cowa_fwd_paged(qr, kp, vp, tabd, i32([0, last - first, 2 * (last - first)]), i32([first] * B), pat,
                                   layout=layout)
        for b in range(B):
            r = slice(b * (last - first), (b + 1) * (last - first))
            tp.assert_chunk(o[r], lse[:, r], to64(qr[r]), hk[b], hv[b], first, pat)
    fn = "cowa_decode_paged_fp8" if e4m3 else "cowa_decode_paged"
    ws = tp.ws_for(fn, pat, B, Hq, Hkv, d, n, ps, cuda_device)
    for t in range(N0, N):
        qt = append(q[:, t], k[:, t], v[:, t], [t] * B)
        o, lse = getattr(cw, fn)(qt, kp, vp, tabd, i32([t] * B), pat, *((ks, vs) if e4m3 else ()), layout=layout,
                                 workspace=ws)
        tp.assert_decoded(o, lse, to64(qt), *held(t), [t] * B, pat, 2.0 ** -11 if e4m3 else 2.0 ** -8)
        if per_head and t % 5 == 0:  # pages go back, and somebody else writes to them
            for g, keep in enumerate(cw.pages_needed(pat, Hkv, ps, n, t + 1)):
                gone = tabd[:, g, torch.from_numpy(~keep).to(cuda_device)].long().reshape(-1)
                gone = gone[gone >= 0]
                kp[gone], vp[gone] = (0x7f, 0xff) if e4m3 else (float("nan"), float("inf"))
                tabd[:, g, torch.from_numpy(~keep).to(cuda_device)] = -1
    assert cw.workspace_status(ws) == 0
    if per_head:
        assert (tabd < 0).any()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("layout", ["bthd", "bhtd"])
def test_decode_of_strided_pools_and_tables(cuda_device, e4m3, wide, layout):
    """Keys and values of a page side by side in one pool, which holds more heads than the call's; a table that is a
    slice of a larger one; no lse; a scale of the scores."""
    B, Hq, Hkv, d, ps, n = 5, 6, 3, 128, 24, 30
    pat, pos = cw.Pattern(9, 70, 600, 3, softmax_scale=0.05), [719, 0, -1, 23, 400]
    rng = np.random.default_rng(144)
    tab, n_pages = tp.make_table(rng, B, n)
    if wide:
        pat, tab = tp.widened(pat, tab, ps)
    shape = (n_pages, 2, ps, Hkv + 2, d) if layout == "bthd" else (n_pages, 2, Hkv + 2, ps, d)
    if e4m3:
        codes = f8.f64_to_e4m3(rng.standard_normal(shape) * 3)
        pool, p64 = torch.from_numpy(codes).to(cuda_device), 0.25 * f8.e4m3_to_f64(codes)
    else:
        p64, pool = host_and_device(shape, "k", cuda_device, 144)
    cut = (lambda x: (x[:, 0, :, 1:1 + Hkv], x[:, 1, :, 2:])) if layout == "bthd" else \
        (lambda x: (x[:, 0, 1:1 + Hkv], x[:, 1, 2:]))
    large = torch.full((2 * B, tab.shape[1] + 9), -7, dtype=torch.int32, device=cuda_device)
    large[::2, 5:5 + tab.shape[1]] = torch.from_numpy(tab).to(cuda_device)
    q64, q = host_and_device((B, Hq, d), "q", cuda_device, 144)
    fn = cw.cowa_decode_paged_fp8 if e4m3 else cw.cowa_decode_paged
    run = lambda **c: fn(q, *cut(pool), large[::2, 5:5 + tab.shape[1]], torch.tensor(pos, dtype=torch.int32, device=cuda_device),
                         pat, *((0.25, 0.25) if e4m3 else ()), layout=layout, **c)
    o, lse = run()
    k, v = (orp.gather_pages(x.transpose(0, 2, 1, 3) if layout == "bhtd" else x, tab, n * ps)[0] for x in cut(p64))
    tp.assert_decoded(o, lse, q64, k, v, pos, pat, 2.0 ** -11 if e4m3 else 2.0 ** -8)
    o2, none = run(want_lse=False)
    assert none is None and torch.equal(o, o2)


@pytest.mark.parametrize("Hq,Hkv,d,ps,n,pat,chunks", [
    (6, 3, 128, 24, 30, cw.Pattern(9, 70, 600, 3, softmax_scale=0.05), [(300, 200), (0, 7)]),
    (10, 2, 64, 16, 64, cw.Pattern(0, 2**31 - 1, 2**31 - 1, 2), [(1000, 24), (0, 130)]),           # all in the band
    (10, 2, 64, 1024, 1, cw.Pattern(2**31 - 1, 1, 2**31 - 1, 2), [(1023, 1), (100, 300)]),         # all sinks, one page
    (4, 4, 64, 512, 2, cw.Pattern(5, 3, 2**31 - 1, 4), [(0, 1024)]),                               # intervals far away
    (16, 2, 128, 40, 25, cw.Pattern(1, 1, 1000, 1, softmax_scale=0.3), [(999, 1), (0, 1), (500, 129)]),
])
def test_chunks_of_strided_tensors_and_extreme_patterns(cuda_device, Hq, Hkv, d, ps, n, pat, chunks):
    """Queries that are a slice of a packed projection, outputs that are a slice of a wider array, keys and values
    side by side in one pool; windows up to INT_MAX, pages of many tiles."""
    B, rng = len(chunks), np.random.default_rng(ps * n)
    tab, n_pages = tp.make_table(rng, B, n)
    p64, pool = host_and_device((n_pages, ps, 2 * Hkv, d), "k", cuda_device, 145)
    lens = [r for _, r in chunks]
    total, cu = sum(lens), np.cumsum([0] + lens)
    x64, x = host_and_device((total, Hq + 3, d), "q", cuda_device, 145)
    wide = torch.full((total, 2, Hq, d), 3.0, dtype=torch.bfloat16, device=cuda_device)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=cuda_device)
    o, lse = cw.cowa_fwd_paged(x[:, 2:2 + Hq], pool[:, :, :Hkv], pool[:, :, Hkv:], torch.from_numpy(tab).to(cuda_device),
                               i32(cu.tolist()), i32([s for s, _ in chunks]), pat, out=wide[:, 1])
    assert (wide[:, 0] == 3.0).all()
    k, v = (orp.gather_pages(y, tab, n * ps)[0] for y in (p64[:, :, :Hkv], p64[:, :, Hkv:]))
    for b, (start, rows) in enumerate(chunks):
        r, e = slice(cu[b], cu[b + 1]), start + rows
        tp.assert_chunk(wide[r, 1], lse[:, r], x64[r, 2:2 + Hq], k[b, :, :e], v[b, :, :e], start, pat)


@pytest.mark.parametrize("pat", [
    cw.Pattern(0, 2**31 - 1, 2**31 - 1, 2), cw.Pattern(2**31 - 1, 1, 2**31 - 1, 2), cw.Pattern(5, 3, 2**31 - 1, 1),
    cw.Pattern(0, 1, 0, 1), cw.Pattern(2**31 - 1, 2**31 - 1, 2**31 - 1, 1),
])
@pytest.mark.parametrize("ps,n", [(8, 1), (1024, 2), (4096, 5)])
def test_decode_of_extreme_patterns(cuda_device, pat, ps, n):
    Hq, Hkv, d, B = 6, 2, 64, 4
    cap = ps * n
    pos = [cap - 1, 0, cap // 2, 2**31 - 1]
    tab, n_pages = tp.make_table(np.random.default_rng(ps), B, n)
    (k64, kd), (v64, vd) = (host_and_device((n_pages, ps, Hkv, d), x, cuda_device, 146) for x in ("k", "v"))
    q64, q = host_and_device((B, Hq, d), "q", cuda_device, 146)
    o, lse = cw.cowa_decode_paged(q, kd, vd, torch.from_numpy(tab).to(cuda_device),
                                  torch.tensor(pos, dtype=torch.int32, device=cuda_device), pat)
    k, v = (orp.gather_pages(x, tab, cap)[0] for x in (k64, v64))
    tp.assert_decoded(o, lse, q64, k, v, pos, pat)


@pytest.mark.parametrize("e4m3", [False, True])
def test_paged_calls_side_by_side(cuda_device, e4m3):
    """Appends, chunks and decodes of four caches on four streams at once, each with a workspace of its own, over
    and over: the bits of the calls made one after the other."""
    Hq, Hkv, d, ps, n, rows = 8, 2, 128, 32, 40, 300
    pat, rope = cw.Pattern(16, 200, 1280, 2), cw.Rope(cw.rope_frequencies(d, device=cuda_device))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=cuda_device)
    r = lambda s, nm, x: synth.cuda_normal_bf16(s, synth.seed_of(nm, 147 + x), cuda_device)
    sets = []
    for x in range(4):
        pools = [r((2 * n, ps, Hkv, d), nm, x) for nm in ("k", "v")]
        if e4m3:
            pools = [cw.quantize_e4m3(p, 1 / 64) for p in pools]
        sets.append(dict(qkv=r((rows, Hq + 2 * Hkv, d), "q", x), pools=pools, first=[p.clone() for p in pools],
                         tab=torch.randperm(2 * n, device=cuda_device).int().view(2, n),
                         ws=torch.zeros(1 << 24, dtype=torch.uint8, device=cuda_device), stream=torch.cuda.Stream()))
    pos = i32([900 + i for i in range(200)] + [17 + i for i in range(rows - 200)])
    seq, cu, start, last = i32([0] * 200 + [1] * (rows - 200)), i32([0, 200, rows]), i32([900, 17]), i32([1099, 16 + rows - 200])

    def step(s, stream):
        q, k, v = s["qkv"].split([Hq, Hkv, Hkv], dim=1)
        kp, vp = s["pools"]
        rest = dict(rope=rope, seq=seq, stream=stream)
        if e4m3:
            qr = cw.paged_append_fp8(q, k, v, pos, kp, vp, s["tab"], 1 / 64, 1 / 64, **rest)
            return qr, *cw.cowa_decode_paged_fp8(qr[:2], kp, vp, s["tab"], last, pat, 1 / 64, 1 / 64, workspace=s["ws"],
                                                 stream=stream)
        qr = cw.paged_append(q, k, v, pos, kp, vp, s["tab"], **rest)
        return qr, *cw.cowa_fwd_paged(qr, kp, vp, s["tab"], cu, start, pat, workspace=s["ws"], stream=stream), \
            *cw.cowa_decode_paged(qr[:2], kp, vp, s["tab"], last, pat, workspace=s["ws"], stream=stream)

    want = []
    for s in sets:
        want.append([x.clone() for x in (*step(s, None), *s["pools"])])
        torch.cuda.synchronize()
        for p, f in zip(s["pools"], s["first"]):
            p.copy_(f)
    torch.cuda.synchronize()
    for _ in range(10):
        got = [step(s, s["stream"]) for s in sets]
    torch.cuda.synchronize()
    for s, g, w in zip(sets, got, want):
        assert cw.workspace_status(s["ws"]) == 0
        for a, b in zip((*g, *s["pools"]), w):
            assert torch.equal(a, b)


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("Hkv,T", [(1, 0), (2, 2**30)])
def test_the_last_positions_of_the_largest_capacity(cuda_device, per_head, Hkv, T):
    """2^30 positions in pages of 8: append, decode and a chunk at the end, the sinks and the band mapped (and, with
    an interval of 2^29 positions for each head, nothing of it: left out and reported)."""
    ps, n, d, Hq, S, L = 8, 1 << 27, 64, 4, 10, 100
    cap, pat = ps * n, cw.Pattern(S, L, max(S, T), Hkv)
    last = cap - 1
    near = np.arange(last - L - 60, cap)  # positions that the rows see through the band, and some
    pages_at = np.unique(np.r_[np.arange(S), near] // ps)
    shape = (1, Hkv, n) if per_head else (1, n)
    tab = torch.full(shape, -1, dtype=torch.int32, device=cuda_device)
    heads = Hkv if per_head else 1
    ids = np.random.default_rng(160).permutation(len(pages_at) * heads + 3)[:len(pages_at) * heads].reshape(heads, -1)
    where = torch.from_numpy(pages_at).to(cuda_device)
    for g in range(heads):
        (tab[0, g] if per_head else tab[0])[where] = torch.from_numpy(ids[g].astype(np.int32)).to(cuda_device)
    kp, vp = (torch.full((len(pages_at) * heads + 3, ps, 1 if per_head else Hkv, d), float("nan"), dtype=torch.bfloat16,
                         device=cuda_device) for _ in range(2))
    rows = (pages_at[:, None] * ps + np.arange(ps)).reshape(-1)  # every position of the mapped pages
    edge = [S + i * (max(S, T) - S) // Hkv for i in range(Hkv + 1)]
    (k64, k), (v64, v) = (host_and_device((len(rows), Hkv, d), x, cuda_device, 160) for x in ("k", "v"))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    cw.paged_append(None, k, v, i32(rows.tolist()), kp, vp, tab, seq=i32([0] * len(rows)))
    q64, q = host_and_device((50, Hq, d), "q", cuda_device, 160)
    ws = torch.zeros(1 << 24, dtype=torch.uint8, device=cuda_device)

    def want(t, row):
        out = []
        for h in range(Hq):
            g = h * Hkv // Hq
            see = (rows <= t) & ((rows < S) | (rows > t - L) | ((rows >= edge[g]) & (rows < edge[g + 1])))
            s = k64[see, g] @ q64[row, h] / np.sqrt(d)
            p = np.exp(s - s.max())
            out.append((p @ v64[see, g] / p.sum(), p @ np.abs(v64[see, g]) / p.sum(), s.max() + np.log(p.sum())))
        return [np.array(x) for x in zip(*out)]

    def check(o, lse, t, row):
        w, A, wl = want(t, row)
        assert (np.abs(to64(o) - w) <= 2.0 ** -8 * (A + np.abs(w)) + 2.0 ** -12 * A).all()
        assert np.abs(lse.double().cpu().numpy() - wl).max() <= tp.LSE_TOL

    for pos in (last, last - 3, 2**31 - 1):
        o, lse = cw.cowa_decode_paged(q[:1], kp, vp, tab, i32([pos]), pat, workspace=ws)
        assert cw.workspace_status(ws) == (8 if T else 0)
        check(o[0], lse[0], min(pos, last), 0)
    if T == 0:
        o, lse = cw.cowa_fwd_paged(q, kp, vp, tab, i32([0, 50]), i32([cap - 50]), pat, workspace=ws)
        assert cw.workspace_status(ws) == 0
        for row in range(50):
            check(o[row], lse[:, row], cap - 50 + row, row)


@pytest.mark.parametrize("odd", [0, 1, 7])
def test_strides_of_dimensions_of_one_element(cuda_device, odd):
    """What a tensor says of the stride of a dimension with a single element means nothing (another framework's
    tensor, or a view, may say anything): the same bits as with the usual strides."""
    def as_odd(x):
        return x.as_strided(x.shape, [s if n > 1 else odd for s, n in zip(x.stride(), x.shape[:-1])] + [1])

    d, ps, n = 64, 16, 1
    rand = lambda s, nm: synth.cuda_normal_bf16(s, synth.seed_of(nm, 161), cuda_device)
    rope, pat = cw.Rope(cw.rope_frequencies(d, device=cuda_device)), cw.Pattern(2, 9, 16, 1)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    one, cu, start = i32([5]), i32([0, 1]), i32([5])
    for layout, per_head in (("bthd", False), ("bhtd", True)):
        x4, q, k = rand((1, 1, 1, d), "q"), rand((1, 1, d), "q"), rand((1, 1, d), "k")
        pool = rand((1, ps, 1, d) if layout == "bthd" else (1, 1, ps, d), "v")
        tab = torch.zeros((1, 1, n) if per_head else (1, n), dtype=torch.int32, device=cuda_device)

        def run(f):
            kp, vp = pool.clone(), pool.clone()
            fk, fv, ft = f(kp), f(vp), tab if f is not as_odd else tab.as_strided(tab.shape, [odd] * (tab.dim() - 1) + [1])
            out = [*cw.cowa_rope(f(x4), f(x4), rope, i32([[3]])), *cw.cowa_rope_bwd(f(x4), None, rope, i32([[3]]))[:1]]
            out.append(cw.paged_append(f(q), f(k), f(k), one, fk, fv, ft, rope=rope, layout=layout))
            out += cw.cowa_decode_paged(q, fk, fv, ft, one, pat, layout=layout)
            out += cw.cowa_fwd_paged(f(q), fk, fv, ft, cu, start, pat, layout=layout, out=f(torch.zeros_like(q)))
            return [*out, kp, vp]

        for a, b in zip(run(as_odd), run(lambda x: x)):
            assert torch.equal(a, b)
