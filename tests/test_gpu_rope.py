"""GPU parity: rotary positions (cowa_rope, cowa_rope_bwd) against the fp64 oracle.

Tolerance, element by element: the result is rounded once to bf16 (half a step: 2^-8 of the value);
before that, the angle in half turns is rounded to fp32 (2^-25 of a half turn, 2^-23 radians), sine
and cosine are within 2 units (2^-23) and two products and a sum are rounded (2^-24 each), which
together stays below 2^-21 scale (|a| + |b|) for a pair (a, b)."""

import numpy as np
import pytest
import torch

from oracle import cowa_oracle as orc
from oracle import rope as orp
from structured_sparse_attention_cowa_b200 import cowa as cw
from structured_sparse_attention_cowa_b200 import synth
from tests.gpu_helpers import host_and_device, to64

pytestmark = pytest.mark.gpu


def partner(x, r, inter):
    """Each rotated element's pair partner (0 for those that pass through)."""
    y, i = np.zeros_like(x), np.arange(r // 2)
    ia, ib = (2 * i, 2 * i + 1) if inter else (i, i + r // 2)
    y[..., ia], y[..., ib] = x[..., ib], x[..., ia]
    return y


def assert_rotated(got, x, want, r, inter, scale=1.0):
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -21 * scale * (np.abs(x) + np.abs(partner(x, r, inter)))
    tol[..., r:] = 0.0  # passed through
    bad = np.abs(got - want) > tol
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5], np.abs(got - want).max())


def freq_of(r, dev):
    f = cw.rope_frequencies(r, device=dev)
    return f, f.cpu().numpy()


CASES = [
    # B, N, Hq, Hkv, d, r, sections, interleaved, scale
    (1, 1, 1, 1, 64, 64, (32,), False, 1.0),            # one token
    (1, 37, 8, 4, 64, 64, (32,), False, 1.0),
    (2, 129, 5, 1, 128, 128, (22, 21, 21), False, 1.0),  # time, height, width
    (3, 50, 8, 2, 128, 96, (48,), False, 1.0),          # part of the head
    (1, 70, 8, 2, 128, 128, (16, 16, 16, 16), True, 1.3),  # neighbouring pairs, four axes, a scale
    (2, 33, 4, 4, 64, 40, (20,), True, 1.0),
    (2, 33, 4, 4, 64, 20, (7, 3), True, 1.0),           # r not a multiple of 8
    (2, 65, 7, 1, 128, 26, (13,), False, 0.5),          # r/2 odd
    (1, 9, 3, 2, 128, 2, (1,), False, 1.0),             # one pair
    (1, 9, 3, 2, 64, 62, (0, 31), True, 1.0),           # an axis without pairs
    (5, 11, 40, 8, 128, 128, (64,), False, 1.0),        # a block's tokens cross batch elements
    (1, 4000, 1, 1, 64, 64, (32,), False, 1.0),
]


@pytest.mark.parametrize("B,N,Hq,Hkv,d,r,sec,inter,scale", CASES)
@pytest.mark.parametrize("bwd", [False, True])
def test_rope_matches_oracle(cuda_device, B, N, Hq, Hkv, d, r, sec, inter, scale, bwd):
    f, f64 = freq_of(r, cuda_device)
    q64, q = host_and_device((B, N, Hq, d), "q", cuda_device, 61)
    k64, k = host_and_device((B, N, Hkv, d), "k", cuda_device, 61)
    pos = np.random.default_rng(N).integers(-1000, 200000, (len(sec), B, N)).astype(np.int32)
    rope = cw.Rope(f, sec, interleaved=inter, scale=scale)
    fn = cw.cowa_rope_bwd if bwd else cw.cowa_rope
    gq, gk = fn(q, k, rope, torch.from_numpy(pos).to(cuda_device))
    for got, x in ((gq, q64), (gk, k64)):
        x = x.reshape(B * N, *x.shape[2:])
        want = orp.rope(x, pos.reshape(len(sec), -1), f64, sec, inter, scale, transpose=bwd)
        assert_rotated(to64(got).reshape(x.shape), x, want, r, inter, scale)


def test_default_positions_and_single_tensors(cuda_device):
    f, f64 = freq_of(128, cuda_device)
    q64, q = host_and_device((2, 300, 3, 128), "q", cuda_device, 62)
    want = orp.rope(q64.reshape(600, 3, 128), np.tile(np.arange(300), 2)[None], f64)
    gq, gk = cw.cowa_rope(q, None, cw.Rope(f))
    assert gk is None
    assert_rotated(to64(gq).reshape(600, 3, 128), q64.reshape(600, 3, 128), want, 128, False)
    gq2, gk = cw.cowa_rope(None, q, cw.Rope(f))
    assert gq2 is None and torch.equal(gk, gq)


@pytest.mark.parametrize("pos", [2**31 - 1, -2**31, 131071, 1 << 24])
def test_far_positions(cuda_device, pos):
    """An fp32 angle would be off by far more than the tolerance from about 2^14 on."""
    f, f64 = freq_of(128, cuda_device)
    q64, q = host_and_device((1, 4, 2, 128), "q", cuda_device, 63)
    p = torch.full((1, 4), pos, dtype=torch.int32, device=cuda_device)
    gq, _ = cw.cowa_rope(q, None, cw.Rope(f), p)
    # 2^31 turns carry 2^-22 of a turn in 64 bits (2^-19 radians), on top of the usual error
    want = orp.rope(q64[0], np.full((1, 4), pos), f64)
    x = q64[0]
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -21 + 2.0 ** -18) * (np.abs(x) + np.abs(partner(x, 128, False)))
    assert (np.abs(to64(gq)[0] - want) <= tol).all()


@pytest.mark.parametrize("r,inter", [(128, False), (96, True), (50, False)])
def test_in_place_strided_and_packed(cuda_device, r, inter):
    """q and k as slices of one packed projection, rotated in place: same bits as out of place, and
    nothing else of the buffer changes; positions broadcast over the batch."""
    B, N, Hq, Hkv, d = 2, 77, 10, 2, 128
    f, _ = freq_of(r, cuda_device)
    rope = cw.Rope(f, interleaved=inter)
    buf = synth.cuda_normal_bf16((B, N, Hq + 2 * Hkv + 1, d), synth.seed_of("q", 64), cuda_device)
    keep = buf.clone()
    q, k = buf[:, :, :Hq], buf[:, :, Hq:Hq + Hkv]
    pos = torch.arange(5, 5 + N, dtype=torch.int32, device=cuda_device)[None].expand(B, N)
    wq, wk = cw.cowa_rope(q.contiguous(), k.contiguous(), rope, pos.contiguous())
    oq, ok = cw.cowa_rope(q, k, rope, pos, q_out=q, k_out=k)
    assert oq.data_ptr() == q.data_ptr()
    assert torch.equal(q, wq) and torch.equal(k, wk)
    assert torch.equal(buf[:, :, Hq + Hkv:], keep[:, :, Hq + Hkv:])
    # [B, H, N, d] storage
    bh = keep[:, :, :Hq].transpose(1, 2).contiguous().transpose(1, 2)
    out = torch.empty((B, Hq, N, d), dtype=torch.bfloat16, device=cuda_device).transpose(1, 2)
    cw.cowa_rope(bh, None, rope, pos, q_out=out)
    assert torch.equal(out, wq)


def test_backward_is_the_gradient(cuda_device):
    """<rope(x), dy> = <x, rope_bwd(dy)>, against sums in 64 bits of the bf16 results: each side is off by
    at most half a bf16 step (2^-8) of every term."""
    f, _ = freq_of(128, cuda_device)
    x64, x = host_and_device((1, 200, 4, 128), "q", cuda_device, 65)
    y64, y = host_and_device((1, 200, 4, 128), "do", cuda_device, 66)
    rope = cw.Rope(f, (22, 21, 21))
    pos = torch.randint(0, 9999, (3, 1, 200), dtype=torch.int32, device=cuda_device)
    a, b = to64(cw.cowa_rope(x, None, rope, pos)[0]), to64(cw.cowa_rope_bwd(y, None, rope, pos)[0])
    lhs, rhs = (a * y64).sum(), (x64 * b).sum()
    assert abs(lhs - rhs) <= 2.0 ** -8 * (np.abs(a * y64).sum() + np.abs(x64 * b).sum()) + 1e-6
    # and far below that bound, since the roundings are independent: five deviations of their sum
    dev = np.sqrt(((2.0 ** -8 * a * y64) ** 2).sum() + ((2.0 ** -8 * x64 * b) ** 2).sum())
    assert abs(lhs - rhs) <= 5 * dev


def test_gradient_of_rotated_attention(cuda_device):
    """q, k rotated, CoWA forward, backward, rotated back: dq and dk against the fp64 chain."""
    B, N, Hq, Hkv, d = 1, 260, 4, 2, 64
    pat = cw.Pattern(16, 40, 260, 2)
    f, f64 = freq_of(64, cuda_device)
    (q64, q), (k64, k), (v64, v), (do64, do) = (host_and_device((B, N, h, d), n, cuda_device, 67)
                                               for n, h in (("q", Hq), ("k", Hkv), ("v", Hkv), ("do", Hq)))
    rope = cw.Rope(f)
    qr, kr = cw.cowa_rope(q, k, rope)
    o, lse = cw.cowa_fwd(qr, kr, v, pat)
    dqr, dkr, dv = cw.cowa_bwd(qr, kr, v, o, lse, do, pat)
    dq, dk = cw.cowa_rope_bwd(dqr, dkr, rope)
    p = np.arange(N)[None]
    rot = lambda x, **kw: orp.rope(x[0], p, f64, **kw)[None]
    op = orc.Pattern(S=16, L=40, T=260, D=2)
    wq, wk, wv = orc.attention_bwd(rot(q64), rot(k64), v64, do64, op)
    for got, want in ((dq, rot(wq, transpose=True)), (dk, rot(wk, transpose=True)), (dv, wv)):
        # the library's gradient tolerance, and one bf16 rounding of q, k and of the result each
        assert np.linalg.norm(to64(got) - want) <= (1e-2 + 3 * 2.0 ** -8) * np.linalg.norm(want)


def test_other_stream_and_graph(cuda_device):
    f, _ = freq_of(128, cuda_device)
    rope = cw.Rope(f)
    q = synth.cuda_normal_bf16((1, 500, 4, 128), synth.seed_of("q", 68), cuda_device)
    k = synth.cuda_normal_bf16((1, 500, 2, 128), synth.seed_of("k", 68), cuda_device)
    wq, wk = cw.cowa_rope(q, k, rope)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    gq, gk = cw.cowa_rope(q, k, rope, stream=side)
    side.synchronize()
    assert torch.equal(gq, wq) and torch.equal(gk, wk)
    oq, ok = torch.zeros_like(q), torch.zeros_like(k)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cw.cowa_rope(q, k, rope, q_out=oq, k_out=ok)
    oq.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(oq, wq) and torch.equal(ok, wk)


def test_refusals_of_the_binding(cuda_device):
    f, _ = freq_of(64, cuda_device)
    q = torch.zeros((2, 8, 4, 64), dtype=torch.bfloat16, device=cuda_device)
    pos = torch.zeros((2, 8), dtype=torch.int32, device=cuda_device)
    rope = cw.Rope(f)
    with pytest.raises(TypeError):
        cw.cowa_rope(q.float(), None, rope)
    with pytest.raises(ValueError):
        cw.cowa_rope(q, q[:1], rope)
    with pytest.raises(ValueError):
        cw.cowa_rope(q, None, rope, pos[:, :7])
    with pytest.raises(TypeError):
        cw.cowa_rope(q, None, rope, pos.long())
    with pytest.raises(ValueError):
        cw.cowa_rope(q, None, rope, pos.t().contiguous().t())
    with pytest.raises(ValueError):
        cw.cowa_rope(q, None, cw.Rope(f, (16, 16)), pos)
    with pytest.raises(ValueError):
        cw.cowa_rope(q, None, rope, q_out=q[:, :4])
    with pytest.raises(ValueError):
        cw.Rope(f, (16, 15))
    with pytest.raises(TypeError):
        cw.Rope(f.double())
    with pytest.raises(cw.CowaError):  # more pairs than the head has
        cw.cowa_rope(q, None, cw.Rope(torch.ones(40, device=cuda_device)))
    with pytest.raises(cw.CowaError):  # a broadcast head
        cw.cowa_rope(q[:, :, :1].expand(2, 8, 4, 64), None, rope)


def test_no_memory_for_an_output(cuda_device):
    """An output that does not fit raises what torch raises for it (2^30 tokens of 64 heads of 128: 16 TiB)."""
    f, _ = freq_of(128, cuda_device)
    q = torch.zeros((1, 1, 1, 128), dtype=torch.bfloat16, device=cuda_device).expand(1, 1 << 30, 64, 128)
    with pytest.raises(torch.OutOfMemoryError):
        cw.cowa_rope(q, None, cw.Rope(f))


@pytest.mark.parametrize("B,N,Hq,Hkv,d,r,inter", [
    (4, 1025, 32, 8, 128, 128, False), (2, 1000, 40, 8, 128, 96, True), (3, 500, 5, 1, 64, 30, False), (1, 868, 1, 1, 128, 64, True),
])
def test_tokens_are_rotated_alike_however_many(cuda_device, B, N, Hq, Hkv, d, r, inter):
    """How many tokens a block owns depends on the call's size, what a token becomes does not: the same bits as
    from calls of 100 tokens."""
    f, _ = freq_of(r, cuda_device)
    rope = cw.Rope(f, (r // 2 - 3, 3), interleaved=inter)
    _, q = host_and_device((B, N, Hq, d), "q", cuda_device, 67)
    _, k = host_and_device((B, N, Hkv, d), "k", cuda_device, 67)
    pos = torch.from_numpy(np.random.default_rng(N).integers(-9, 99999, (2, B, N)).astype(np.int32)).to(cuda_device)
    gq, gk = cw.cowa_rope(q, k, rope, pos)
    for b in range(B):
        for t in range(0, N, 100):
            s = slice(t, t + 100)
            wq, wk = cw.cowa_rope(q[b:b + 1, s], k[b:b + 1, s], rope, pos[:, b:b + 1, s])
            assert torch.equal(gq[b:b + 1, s], wq) and torch.equal(gk[b:b + 1, s], wk)
