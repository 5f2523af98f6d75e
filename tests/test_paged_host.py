"""Host side of the rotary positions and the paged cache: every refusal returns its status before any
launch, the binding refuses what does not fit, and pages_needed matches the mask.  No GPU is touched."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import cowa_oracle as orc
from structured_sparse_attention_cowa_b200 import cowa as cw

T = lambda ptr=0x10000, sb=1 << 20, st=1024, sh=128: cw.c_tensor(ptr, sb, st, sh)


def rotary(freq=0x7000, r=128, axes=1, sec=(64, 0, 0, 0), inter=0, scale=1.0):
    return cw.c_rotary(freq, r, axes, (ctypes.c_int32 * 4)(*sec), inter, scale)


def table(ptr=0x8000, sb=64, sh=0, max_pages=64, page=16, n_pages=100, per_head=0):
    return cw.c_page_table(ptr, sb, sh, max_pages, page, n_pages, per_head)


@pytest.mark.parametrize("fn", ["cowa_rope", "cowa_rope_bwd"])
@pytest.mark.parametrize("status,change", [
    (1, dict(rot=None)), (1, dict(rot=rotary(freq=None))), (3, dict(rot=rotary(freq=0x7002))),
    (1, dict(rot=rotary(r=0))), (1, dict(rot=rotary(r=127))), (1, dict(rot=rotary(r=130))),
    (1, dict(rot=rotary(axes=0))), (1, dict(rot=rotary(axes=5))), (1, dict(rot=rotary(scale=float("nan")))),
    (1, dict(rot=rotary(axes=2, sec=(32, 31, 0, 0)))), (1, dict(rot=rotary(axes=2, sec=(65, -1, 0, 0)))),
    (1, dict(rot=rotary(axes=3, sec=(2**31 - 1, 2**31 - 1, 66, 0)))),
    (1, dict(B=0)), (1, dict(N=0)), (1, dict(Hq=-1)), (1, dict(Hq=0, Hkv=0)), (2, dict(d=96)), (2, dict(d=256)),
    (1, dict(q=T(None))), (3, dict(q=T(0x10008))), (3, dict(ko=T(st=1020))), (3, dict(k=T(sh=0))),
    (1, dict(sa=-1)), (1, dict(sb=-1)), (3, dict(pos=0x9002)),
])
def test_rope_refusals(fn, status, change):
    a = dict(rot=rotary(), B=1, N=16, Hq=8, Hkv=4, d=128, q=T(), k=T(), qo=T(), ko=T(), pos=0x9000, sa=16, sb=16)
    a.update(change)
    rot = ctypes.byref(a["rot"]) if a["rot"] is not None else None
    assert getattr(cw.lib(), fn)(rot, a["B"], a["N"], a["Hq"], a["Hkv"], a["d"], a["q"], a["k"], a["qo"], a["ko"],
                                 a["pos"], a["sa"], a["sb"], None) == status


@pytest.mark.parametrize("status,change", [
    (1, dict(total=0)), (1, dict(total=9)), (1, dict(n_seq=0)), (1, dict(Hkv=0)), (1, dict(Hq=-1)), (1, dict(pos=None)),
    (2, dict(d=96)), (2, dict(Hkv=1025)), (1, dict(rot=rotary(r=129))), (1, dict(k=T(None))), (3, dict(v=T(0x10004))),
    (3, dict(kp=T(st=4))), (1, dict(vp=T(None))), (1, dict(tab=table(ptr=None))), (3, dict(tab=table(ptr=0x8002))),
    (1, dict(tab=table(sb=-1))), (1, dict(tab=table(page=12))), (1, dict(tab=table(page=0))),
    (1, dict(tab=table(max_pages=0))), (1, dict(tab=table(n_pages=0))), (1, dict(tab=table(per_head=1))),
    (1, dict(tab=table(max_pages=1 << 26, page=32))), (3, dict(pos=0x9001)), (3, dict(seq=0x9003)),
    (3, dict(rp=0x9002)), (1, dict(rs=-1)),
    (1, dict(ks=0.0)), (1, dict(vs=float("inf"))), (1, dict(ks=float("nan"))), (2, dict(d=64)),
])
def test_append_refusals(status, change):
    base = dict(rot=rotary(), total=8, n_seq=8, Hq=8, Hkv=4, d=128, q=T(), k=T(), v=T(), qo=T(), pos=0x9000, seq=None,
                rp=0x9000, rs=8, kp=T(), vp=T(), ks=1.0, vs=1.0, tab=table())
    a, L = {**base, **change}, cw.lib()
    args = (ctypes.byref(a["rot"]), a["total"], a["n_seq"], a["Hq"], a["Hkv"], a["d"], a["q"], a["k"], a["v"], a["qo"],
            a["pos"], a["seq"], a["rp"], a["rs"], a["kp"], a["vp"])
    assert L.cowa_paged_append_fp8(*args, a["ks"], a["vs"], a["tab"], None) == status
    if not {"ks", "vs"} & set(change) and change != dict(d=64):
        assert L.cowa_paged_append(*args, a["tab"], None) == status


@pytest.mark.parametrize("status,change", [
    (1, dict(B=0)), (1, dict(Hq=7)), (2, dict(Hq=36)), (2, dict(d=96)), (1, dict(q=None)), (1, dict(pos=None)),
    (1, dict(o=None)), (3, dict(q=0x10004)), (3, dict(o=0x10008)), (3, dict(lse=0x10002)), (3, dict(pos=0x9002)),
    (1, dict(kp=T(None))), (3, dict(vp=T(sb=12))), (1, dict(tab=table(page=20))), (1, dict(tab=table(n_pages=0))),
    (1, dict(tab=table(ptr=None))), (1, dict(tab=table(per_head=1, sh=0))), (4, dict(ws=None)), (4, dict(ws=0x40080)),
    (4, dict(less=1)), (1, dict(pat=cw.Pattern(10, 4, 5, 1))), (1, dict(ks=-1.0)), (2, dict(B=2**30)),
])
def test_decode_refusals(status, change):
    a = dict(pat=cw.Pattern(64, 100, 1024, 4), B=3, Hq=8, Hkv=4, d=128, q=0x10000, kp=T(), vp=T(), tab=table(),
             pos=0x9000, o=0x20000, lse=0x30000, ws=0x40000, less=0, ks=1.0, vs=1.0)
    a.update(change)
    L, pat = cw.lib(), a["pat"].c()
    size = lambda f: f(ctypes.byref(cw.Pattern(64, 100, 1024, 4).c()), 3, 8, 4, 128, 64, 16)
    for fn, scales in (("cowa_decode_paged", ()), ("cowa_decode_paged_fp8", (a["ks"], a["vs"]))):
        if "ks" in change and not scales:
            continue
        n = size(getattr(L, fn + "_workspace_size"))
        assert n > 256
        got = getattr(L, fn)(ctypes.byref(pat), a["B"], a["Hq"], a["Hkv"], a["d"], a["q"], a["kp"], a["vp"], *scales,
                             a["tab"], a["pos"], a["o"], a["lse"], a["ws"], n - a["less"], None)
        assert got == status, fn
    assert L.cowa_decode_paged_fp8_workspace_size(ctypes.byref(cw.Pattern(64, 100, 1024, 4).c()), 3, 8, 4, 64, 64, 16) == 0


@pytest.mark.parametrize("status,change", [
    (1, dict(n_seq=0)), (1, dict(total=0)), (1, dict(Hq=7)), (2, dict(Hq=36)), (2, dict(d=96)), (1, dict(cu=None)),
    (1, dict(start=None)), (1, dict(lse=None)), (3, dict(cu=0x9002)), (3, dict(start=0x9001)), (3, dict(lse=0x9003)),
    (1, dict(q=T(None))), (3, dict(o=T(0x10004))), (3, dict(kp=T(sb=4))), (1, dict(vp=T(None))),
    (1, dict(tab=table(page=4))), (1, dict(tab=table(ptr=None))), (4, dict(less=1)), (4, dict(ws=0x40010)),
    (1, dict(pat=cw.Pattern(10, 4, 5, 1))),
])
def test_chunk_refusals(status, change):
    a = dict(pat=cw.Pattern(64, 100, 1024, 4), n_seq=3, total=500, Hq=8, Hkv=4, d=128, cu=0x9000, start=0x9100, q=T(),
             kp=T(), vp=T(), tab=table(), o=T(), lse=0x30000, ws=0x40000, less=0)
    a.update(change)
    L = cw.lib()
    n = L.cowa_fwd_paged_workspace_size(ctypes.byref(cw.Pattern(64, 100, 1024, 4).c()), 3, 500, 8, 4, 128, 64, 16)
    assert L.cowa_fwd_paged(ctypes.byref(a["pat"].c()), a["n_seq"], a["total"], a["Hq"], a["Hkv"], a["d"], a["cu"],
                            a["start"], a["q"], a["kp"], a["vp"], a["tab"], a["o"], a["lse"], a["ws"], n - a["less"],
                            None) == status


def test_workspace_is_bounded_and_grows_with_the_group():
    """At most two partials per CTA, and no more CTAs than the GPU holds: the size stops growing."""
    L, pat = cw.lib(), cw.Pattern(128, 4096, 131072, 8).c()
    ws = lambda B, Hq, pages: L.cowa_decode_paged_workspace_size(ctypes.byref(pat), B, Hq, 8, 128, pages, 64)
    assert ws(16, 40, 2048) == ws(512, 40, 2048) >= 256 + 16 * 296 + 2 * 296 * 5 * 130 * 4
    assert ws(1, 8, 1) < ws(1, 64, 1) < ws(16, 64, 2048)


@pytest.mark.parametrize("pat,h,ps,n,pos", [
    (cw.Pattern(20, 30, 300, 4), 4, 8, 50, 150), (cw.Pattern(0, 1, 300, 2), 4, 16, 25, 299),
    (cw.Pattern(64, 2**31 - 1, 300, 1), 2, 16, 25, 10), (cw.Pattern(4, 60, 4, 1), 1, 24, 20, 400),
    (cw.Pattern(3, 9, 257, 2, kv_head_base=2, h_kv_global=4), 2, 8, 40, 0),
])
def test_pages_needed_matches_the_mask(pat, h, ps, n, pos):
    got = cw.pages_needed(pat, h, ps, n, pos)
    N = n * ps
    op = orc.Pattern(S=pat.S, L=pat.L, T=pat.T, D=pat.D, kv_head_base=pat.kv_head_base,
                     h_kv_global=pat.h_kv_global or None)
    for g in range(h):
        # a position is still needed if some t >= pos sees it: now, in the band, sink or interval, or later
        seen = orc.visible_mask(np.arange(pos, max(N, pos + 1)), N, op, g, h).any(0)
        seen[min(pos + 1, N):] = True
        assert np.array_equal(got[g], seen.reshape(n, ps).any(1)), g


def test_pages_needed_refusals():
    pat = cw.Pattern(20, 30, 300, 4)
    for args in ((0, 8, 5, 1), (4, 0, 5, 1), (4, 8, 0, 1), (4, 8, 5, -1), (4, 1 << 20, 1 << 20, 1)):
        with pytest.raises((cw.CowaError, ValueError)):
            if args[0] == 0 or args[2] == 0 or args[1:3] == (1 << 20, 1 << 20):
                st = cw.lib().cowa_pages_needed(ctypes.byref(pat.c()), *args, ctypes.c_void_p(0x10000))
                raise cw.CowaError("cowa_pages_needed", st, "") if st == 1 else AssertionError(st)
            cw.pages_needed(pat, *args)


def test_status_of_a_bad_page_has_a_name():
    assert b"page" in cw.lib().cowa_status_string(8)


def test_binding_refuses_cpu_tensors_and_wrong_types():
    q = torch.zeros((2, 4, 8, 64), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        cw.Rope(torch.ones(32))
    fake = object.__new__(cw.Rope)
    fake.inv_freq, fake._c = torch.ones(32), rotary(r=64)
    fake._address = ctypes.addressof(fake._c)
    with pytest.raises(TypeError):
        cw.cowa_rope(q, None, fake)
    with pytest.raises(ValueError):
        cw.cowa_rope(None, None, fake)
    pos = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        cw.paged_append(None, q[:, 0], q[:, 0], pos, q, q, pos)
    with pytest.raises(TypeError):
        cw.cowa_decode_paged(q[:, 0], q, q, pos, pos, cw.Pattern(1, 1, 1, 1))
    with pytest.raises(TypeError):
        cw.cowa_decode_paged_fp8(q[:, 0], q, q, pos, pos, cw.Pattern(1, 1, 1, 1), 1.0, 1.0)


def test_missing_compiled_binding_raises(monkeypatch):
    import sys

    import structured_sparse_attention_cowa_b200 as pkg

    monkeypatch.setattr(cw, "_binding_of", None)
    monkeypatch.delattr(pkg, "_binding", raising=False)
    monkeypatch.setitem(sys.modules, pkg.__name__ + "._binding", None)
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(RuntimeError, match="_binding.so"):
        cw.paged_append(None, q, q, q, q, q, q)


def test_rope_cannot_be_changed():
    """A call reads the address that the Rope was made with: other frequencies need another Rope."""
    rope = object.__new__(cw.Rope)
    rope.inv_freq = torch.ones(32)
    with pytest.raises(AttributeError, match="Rope"):
        rope.inv_freq = torch.ones(32)


@pytest.mark.parametrize("rotary_dim,base", [(0, 1e4), (-2, 1e4), (7, 1e4), (64, 0.0), (64, -1e4)])
def test_rope_frequencies_refusals(rotary_dim, base):
    with pytest.raises(ValueError):
        cw.rope_frequencies(rotary_dim, base, device="cpu")


def test_rope_frequencies_match_their_formula():
    got = cw.rope_frequencies(96, 5e5, device="cpu")
    want = np.array([5e5 ** (-2 * i / 96) for i in range(48)])
    assert got.dtype == torch.float32 and (np.abs(got.double().numpy() - want) <= 2.0 ** -23 * want).all()


def test_rope_of_nothing_on_a_stream_is_refused():
    fake = object.__new__(cw.Rope)
    fake.inv_freq, fake._c = torch.ones(32), rotary(r=64)
    fake._address = ctypes.addressof(fake._c)
    with pytest.raises(ValueError, match="q or k"):
        cw.cowa_rope(None, None, fake, stream=object())
