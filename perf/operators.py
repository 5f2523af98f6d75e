"""Cases of the paged serving path and of rotary positions: what they compute, in elementary torch operations.

Four operators, as a serving or training program around CoWindow Attention calls them:

  rope    rotary positions of one to four axes on the queries and keys of a layer, forward and backward
  append  the tokens of a step (one per sequence, or the chunks of several prompts): queries and keys rotated, keys and
          values written to the pages of a paged cache, in bf16 or as E4M3 codes
  decode  one new token per sequence against a paged cache (bf16 or E4M3, pages shared by the heads or one table a head)
  chunk   the query rows of prompt chunks against a paged cache that already holds their keys

`run` computes them plainly where `own` is false and calls structured_sparse_attention_cowa_b200 where it is true.
"""

import math
import random

import numpy as np
import torch

own = False

F8 = torch.float8_e4m3fn


# ---------------------------------------------------------------------------------------------- the cases
def listed():
    layer = {"Hq": 40, "Hkv": 8, "d": 128}
    pat32 = {"S": 128, "L": 2048, "T": 32768, "D": 8}
    pat128 = {"S": 128, "L": 4096, "T": 131072, "D": 8}
    return [
        # the smallest training layer: 1024 tokens, d = 64; latency counts
        {"name": "rope_1k_d64", "op": "rope", "B": 1, "N": 1024, "Hq": 8, "Hkv": 4, "d": 64, "rd": 64, "axes": 1,
         "inter": False, "bwd": False, "mix": 1},
        # one 32K sequence of video and text tokens (time, height, width), the training layer's heads
        {"name": "rope_32k_video", "op": "rope", "B": 1, "N": 32768, **layer, "rd": 128, "axes": 3, "inter": False,
         "bwd": False, "mix": 2},
        # gradients of a layer that rotates part of each head (96 of 128), neighbouring pairs, two axes, an odd length
        {"name": "rope_bwd_8k_partial", "op": "rope", "B": 2, "N": 8191, "Hq": 32, "Hkv": 8, "d": 128, "rd": 96,
         "axes": 2, "inter": True, "bwd": True, "mix": 3},
        # a decode step of 16 long sequences: one token each, bf16 pages
        {"name": "append_step_b16", "op": "append", "total": 16, "n_seq": 16, "chunks": False, **layer, "rd": 128,
         "axes": 1, "inter": False, "page": 64, "cap": 32768, "per_head": False, "fp8": False, "layout": "bhtd",
         "idle": 0, "mix": 4},
        # prompt chunks of five sequences, 8K tokens in all, written as E4M3 codes into small pages
        {"name": "append_8k_e4m3", "op": "append", "total": 8192, "n_seq": 5, "chunks": True, **layer, "rd": 128,
         "axes": 3, "inter": False, "page": 16, "cap": 16384, "per_head": False, "fp8": True, "layout": "bthd",
         "idle": 7, "mix": 5},
        # one long prompt written in one go, bf16 pages of 128 tokens
        {"name": "append_32k_bf16", "op": "append", "total": 32768, "n_seq": 1, "chunks": True, **layer, "rd": 128,
         "axes": 1, "inter": False, "page": 128, "cap": 32768, "per_head": False, "fp8": False, "layout": "bhtd",
         "idle": 0, "mix": 6},
        # one user, 8K tokens: the smallest decode, latency counts
        {"name": "decode_b1_8k", "op": "decode", "B": 1, "Hq": 32, "Hkv": 8, "d": 128, "S": 128, "L": 1024, "T": 8192,
         "D": 8, "page": 64, "cap": 8192, "per_head": False, "fp8": False, "layout": "bhtd", "full": True, "idle": 0,
         "mix": 7},
        # the 128K decode configuration: 16 sequences at the last position
        {"name": "decode_b16_128k", "op": "decode", "B": 16, **layer, **pat128, "page": 64, "cap": 131072,
         "per_head": False, "fp8": False, "layout": "bhtd", "full": True, "idle": 0, "mix": 8},
        # a ragged batch with idle slots: lengths from 1 to 32K, E4M3 codes, every head with its own pages
        {"name": "decode_b37_e4m3", "op": "decode", "B": 37, **layer, **pat32, "page": 16, "cap": 32768,
         "per_head": True, "fp8": True, "layout": "bthd", "full": False, "idle": 3, "mix": 9},
        # a short chunk behind a cached prefix, d = 64
        {"name": "chunk_200_d64", "op": "chunk", "n_seq": 1, "total": 200, "Hq": 8, "Hkv": 4, "d": 64, "S": 64,
         "L": 128, "T": 1024, "D": 4, "page": 32, "cap": 2048, "per_head": False, "layout": "bthd", "mix": 10},
        # chunks of six sequences of different prefixes in one batch
        {"name": "chunk_6x_ragged", "op": "chunk", "n_seq": 6, "total": 2500, **layer, **pat32, "page": 16,
         "cap": 16384, "per_head": False, "layout": "bhtd", "mix": 11},
        # a 4K chunk at the end of a 32K prompt
        {"name": "chunk_4k_of_32k", "op": "chunk", "n_seq": 1, "total": 4096, **layer, **pat32, "page": 64,
         "cap": 32768, "per_head": False, "layout": "bhtd", "mix": 12},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    d = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    heads = {"Hq": Hkv * rng.choice([1, 2, 3, 4, 5, 6, 7, 8]), "Hkv": Hkv, "d": d}
    rd = rng.choice([d, d, d // 2, d - 16 * rng.randint(0, d // 16 - 1), 2 * rng.randint(4, d // 2)])
    axes = rng.choice([1, 2, 3, 4])
    turn = {"rd": rd, "axes": axes, "inter": rng.random() < 0.4}
    page = rng.choice([8, 16, 16, 24, 32, 48, 64, 128, 256])
    mix = rng.randrange(1 << 20)
    op = rng.choice(["rope", "append", "decode", "chunk"])
    if op == "rope":
        B = _log(rng, 1, 8)
        return {"op": op, "B": B, "N": _log(rng, 1, 16384 // B), **heads, **turn, "bwd": rng.random() < 0.5, "mix": mix}
    layout = rng.choice(["bthd", "bhtd"])
    per_head = rng.random() < 0.3
    if op == "append":
        chunks = rng.random() < 0.5
        n_seq = _log(rng, 1, 16) if chunks else _log(rng, 1, 256)
        total = _log(rng, n_seq, 16384) if chunks else n_seq
        cap = _up(max(total, _log(rng, 256, 16384)), page)
        if not chunks:
            cap = _up(_log(rng, 64, max(64, min(4096, (1 << 18) // n_seq))), page)
        return {"op": op, "total": total, "n_seq": n_seq, "chunks": chunks, **heads, **turn, "page": page, "cap": cap,
                "per_head": per_head, "fp8": d == 128 and rng.random() < 0.5, "layout": layout,
                "idle": rng.randint(0, min(3, total - 1)), "mix": mix}
    D = rng.choice([x for x in (1, 2, 4, 8) if Hkv % x == 0])
    if op == "decode":
        B = _log(rng, 1, 64)
        cap = _up(_log(rng, 64, max(64, min(131072, (1 << 19) // B))), page)
        pat = {"S": rng.choice([0, 4, 100, 128]), "L": _log(rng, 1, 8192), "D": D}
        pat["T"] = pat["S"] + rng.choice([0, _log(rng, 1, cap), cap])
        return {"op": op, "B": B, **heads, **pat, "page": page, "cap": cap, "per_head": per_head,
                "fp8": d == 128 and rng.random() < 0.5, "layout": layout, "full": rng.random() < 0.3,
                "idle": rng.randint(0, min(3, B - 1)), "mix": mix}
    n_seq = _log(rng, 1, 8)
    total = _log(rng, n_seq, 2048)
    cap = _up(max(total, _log(rng, 128, max(128, 32768 // n_seq))), page)
    pat = {"S": rng.choice([0, 4, 100, 128]), "L": _log(rng, 1, 4096), "D": D}
    pat["T"] = pat["S"] + rng.choice([0, _log(rng, 1, cap), cap])
    return {"op": op, "n_seq": n_seq, "total": total, **heads, **pat, "page": page, "cap": cap, "per_head": per_head,
            "layout": layout, "mix": mix}


def _up(x, m):
    return (x + m - 1) // m * m


def _sections(c):
    """Pairs of each axis: the first takes what an even split leaves over (rd/2 = 64, three axes: 22, 21, 21)."""
    h, n = c["rd"] // 2, min(c["axes"], c["rd"] // 2)
    return [h // n + (h % n if a == 0 else 0) for a in range(n)]


def _parts(rng, total, n):
    """n positive numbers that add up to total."""
    cut = sorted(rng.sample(range(1, total), n - 1)) if n > 1 else []
    return [b - a for a, b in zip([0] + cut, cut + [total])]


def _positions(c):
    """Decode: the position of each sequence's new token; -1 for a slot without a sequence."""
    rng = random.Random(c["mix"])
    pos = [c["cap"] - 1 if c["full"] else _log(rng, 1, c["cap"]) - 1 for _ in range(c["B"])]
    for i in rng.sample(range(c["B"]), c["idle"]):
        pos[i] = -1
    return pos


def _chunks(c):
    """(start, rows) of each sequence's chunk: rows of the call at positions start .. start + rows - 1."""
    rng = random.Random(c["mix"])
    rows = _parts(rng, c["total"], c["n_seq"])
    if c["n_seq"] == 1:  # the end of a prompt
        return [(c["cap"] - rows[0], rows[0])]
    return [(rng.randint(0, c["cap"] - r), r) for r in rows]


def _append_rows(c):
    """(sequence, position) of each row of an append; position -1: a row of padding."""
    rng = random.Random(c["mix"])
    if c["chunks"]:
        rows = [(s, p0 + i) for s, (p0, n) in enumerate(_chunks(c)) for i in range(n)]
    else:
        rows = [(s, rng.randrange(c["cap"])) for s in range(c["n_seq"])]
    for i in range(c["idle"]):  # the padding stands at the end, as a packed batch has it
        rows[len(rows) - 1 - i] = (0, -1)
    return rows


def _intervals(c):
    """Long-range interval [lo, hi) of each KV head: b_i = S + floor(i (T - S) / H), slot (g mod D) H / D."""
    H, S, T, D = c["Hkv"], c["S"], c["T"], c["D"]
    b = [S + i * (T - S) // H for i in range(H + 1)]
    slot = [(g % D) * (H // D) for g in range(H)]
    return [b[s] for s in slot], [b[s + 1] for s in slot]


def _seen(c, t):
    """Keys that position t (an int64 array) sees, per head: [H, len(t)]."""
    lo, hi = (np.array(x)[:, None] for x in _intervals(c))
    n0 = np.minimum(c["S"], t + 1)
    band = np.maximum(t - c["L"] + 1, n0)
    n1 = np.maximum(np.minimum(hi, band) - lo, 0)
    return np.where(t < 0, 0, n0 + n1 + t + 1 - band)


def work(c):
    """Bytes that are read and written once, and the products of the attention (or the rotation's)."""
    op = c["op"]
    if op == "rope":
        x = c["B"] * c["N"] * (c["Hq"] + c["Hkv"])
        return {"bytes": 4 * x * c["d"] + 4 * c["B"] * c["N"] * len(_sections(c)), "flops": 3 * x * c["rd"]}
    if op == "append":
        n, d = sum(p >= 0 for _, p in _append_rows(c)), c["d"]
        kv = 2 * c["Hkv"] * d
        return {"bytes": n * (4 * c["Hq"] * d + kv * (2 + (1 if c["fp8"] else 2)) + 4 * (2 + len(_sections(c)))),
                "flops": 3 * n * (c["Hq"] + c["Hkv"]) * c["rd"]}
    grp, d = c["Hq"] // c["Hkv"], c["d"]
    if op == "decode":
        t = np.array(_positions(c), dtype=np.int64)
        n = int(_seen(c, t).sum())
        return {"bytes": 2 * n * d * (1 if c["fp8"] else 2) + c["B"] * c["Hq"] * (4 * d + 4),
                "flops": 4 * n * d * grp}
    pairs = rows = 0
    lo, hi = _intervals(c)
    for p0, n in _chunks(c):
        pairs += int(_seen(c, np.arange(p0, p0 + n, dtype=np.int64)).sum())
        s = np.arange(p0 + n)
        for g in range(c["Hkv"]):
            rows += int(((s < c["S"]) | (s > p0 - c["L"]) | ((s >= lo[g]) & (s < hi[g]))).sum())
    return {"bytes": 4 * rows * d + c["total"] * c["Hq"] * (4 * d + 4), "flops": 4 * pairs * d * grp}


# ---------------------------------------------------------------------------------------------- their inputs
def _device():
    return torch.device("cuda", torch.cuda.current_device())


def _normal(shape, gen):
    return torch.randn(shape, generator=gen, device=gen.device, dtype=torch.bfloat16)


def _ints(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def _turn(c, n, first, gen, dev):
    """What a program keeps for its rotary positions, and the n positions of each axis."""
    rd = c["rd"]
    freq = (10000.0 ** (-torch.arange(0, rd, 2, dtype=torch.float64) / rd)).float().to(dev)
    sec = _sections(c)
    axis = torch.repeat_interleave(torch.arange(len(sec)), torch.tensor(sec)).to(dev)
    pos = torch.as_tensor(first, dtype=torch.int32, device=dev).reshape(1, -1).repeat(len(sec), 1)
    if len(sec) > 1:  # the other axes are places in an image
        pos[1:] = torch.randint(0, 64, (len(sec) - 1, n), generator=gen, device=dev, dtype=torch.int32)
    return {"freq": freq, "axis": axis, "sections": tuple(sec), "pos": pos}


def _table(c, last, gen, dev):
    """Page table for sequences whose last position is last[b] (-1: none), pages in random order, and the pool's
    page count.  One table a head maps only what the head can still see: its sink, its interval and the band."""
    n, ps = c["cap"] // c["page"], c["page"]
    first = torch.arange(n, device=dev) * ps
    have = first[None, None] <= torch.tensor(last, device=dev)[:, None, None]
    if c["per_head"]:
        have = have.expand(-1, c["Hkv"], -1)
        if "S" in c:
            lo, hi = (torch.tensor(x, device=dev)[None, :, None] for x in _intervals(c))
            t = torch.tensor(last if c["op"] == "decode" else [p for p, _ in _chunks(c)], device=dev)[:, None, None]
            have = have & ((first < c["S"]) | (first + ps > t - c["L"] + 1) | ((first < hi) & (first + ps > lo)))
    want = int(have.sum())
    order = torch.randperm(want + 3, generator=gen, device=dev).int()
    rank = torch.cumsum(have.reshape(-1).int(), 0).reshape(have.shape) - 1
    table = torch.where(have, order[rank.clamp(min=0)], -1).contiguous()
    return (table if c["per_head"] else table[:, 0].contiguous()), want + 3


def _pool(c, pages, gen, fp8):
    """Pages in the case's layout, one more than the table knows (where the plain form puts what has no page)."""
    H = 1 if c["per_head"] else c["Hkv"]
    shape = (pages + 1, c["page"], H, c["d"]) if c["layout"] == "bthd" else (pages + 1, H, c["page"], c["d"])
    if not fp8:
        return _normal(shape, gen)
    out = torch.empty(shape, dtype=torch.uint8, device=gen.device)
    step = max(1, (1 << 28) // math.prod(shape[1:]))
    for i in range(0, shape[0], step):
        out[i:i + step] = (_normal((min(step, shape[0] - i), *shape[1:]), gen).float() * 64).to(F8).view(torch.uint8)
    return out


def prepare(c, seed):
    dev = _device()
    gen = torch.Generator(device=dev).manual_seed(seed)
    st = {"case": c, "ws": torch.zeros(1 << 24, dtype=torch.uint8, device=dev)}
    op = c["op"]
    if op == "rope":
        n = c["B"] * c["N"]
        st["turn"] = _turn(c, n, torch.arange(c["N"]).repeat(c["B"]), gen, dev)
        st["turn"]["pos"] = st["turn"]["pos"].reshape(-1, c["B"], c["N"])
        st["q"] = _normal((c["B"], c["N"], c["Hq"], c["d"]), gen)
        st["k"] = _normal((c["B"], c["N"], c["Hkv"], c["d"]), gen)
        return st
    if op == "append":
        rows = _append_rows(c)
        last = [max((p for s, p in rows if s == b), default=-1) for b in range(c["n_seq"])] if not c["chunks"] else \
            [p0 + n - 1 for p0, n in _chunks(c)]
        st["table"], pages = _table(c, last, gen, dev)
        st["pos"] = _ints([p for _, p in rows], dev)
        st["seq"] = _ints([s for s, _ in rows], dev) if c["chunks"] else None
        st["turn"] = _turn(c, c["total"], st["pos"], gen, dev)
        qkv = _normal((c["total"], c["Hq"] + 2 * c["Hkv"], c["d"]), gen)  # one projection's output
        st["q"], st["k"], st["v"] = qkv.split([c["Hq"], c["Hkv"], c["Hkv"]], dim=1)
        st["q_out"] = torch.zeros((c["total"], c["Hq"], c["d"]), dtype=torch.bfloat16, device=dev)
        st["kp"], st["vp"] = _pool(c, pages, gen, c["fp8"]), _pool(c, pages, gen, c["fp8"])
        return st
    lo, hi = _intervals(c)
    st["lo"], st["hi"] = torch.tensor(lo, device=dev), torch.tensor(hi, device=dev)
    if op == "decode":
        pos = _positions(c)
        st["table"], pages = _table(c, pos, gen, dev)
        st["pos"] = _ints(pos, dev)
        st["q"] = _normal((c["B"], c["Hq"], c["d"]), gen)
        st["kp"], st["vp"] = _pool(c, pages, gen, c["fp8"]), _pool(c, pages, gen, c["fp8"])
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty((c["B"], c["Hq"]), device=dev)
        return st
    ch = _chunks(c)
    st["table"], pages = _table(c, [p0 + n - 1 for p0, n in ch], gen, dev)
    st["rows"] = (max(n for _, n in ch), max(p0 + n for p0, n in ch))
    st["start"] = _ints([p0 for p0, _ in ch], dev)
    st["cu"] = _ints(np.cumsum([0] + [n for _, n in ch]).tolist(), dev)
    st["q"] = _normal((c["total"], c["Hq"], c["d"]), gen)
    st["kp"], st["vp"] = _pool(c, pages, gen, False), _pool(c, pages, gen, False)
    st["out"] = torch.empty_like(st["q"])
    st["lse"] = torch.empty((c["Hq"], c["total"]), device=dev)
    return st


# ---------------------------------------------------------------------------------------------- one pass
def run(st):
    if own:
        return _own(st)
    return {"rope": _rope, "append": _append, "decode": _decode, "chunk": _chunk}[st["case"]["op"]](st)


def _own(st):
    from structured_sparse_attention_cowa_b200 import cowa as cw

    c, op = st["case"], st["case"]["op"]
    if "handle" not in st:  # what a program makes once
        t = st.get("turn")
        st["handle"] = (cw.Rope(t["freq"], t["sections"], interleaved=c["inter"]) if t else
                        cw.Pattern(c["S"], c["L"], c["T"], c["D"]))
    h = st["handle"]
    if op == "rope":
        return (cw.cowa_rope_bwd if c["bwd"] else cw.cowa_rope)(st["q"], st["k"], h, st["turn"]["pos"])
    kp, vp = st["kp"][:-1], st["vp"][:-1]
    if op == "append":
        rest = {"rope": h, "rope_pos": st["turn"]["pos"], "seq": st["seq"], "q_out": st["q_out"], "layout": c["layout"]}
        if c["fp8"]:
            q = cw.paged_append_fp8(st["q"], st["k"], st["v"], st["pos"], kp, vp, st["table"], 1 / 64, 1 / 64, **rest)
            return q, kp.view(F8), vp.view(F8)
        return cw.paged_append(st["q"], st["k"], st["v"], st["pos"], kp, vp, st["table"], **rest), kp, vp
    rest = {"layout": c["layout"], "out": st["out"], "lse": st["lse"], "workspace": st["ws"]}
    if op == "chunk":
        return cw.cowa_fwd_paged(st["q"], kp, vp, st["table"], st["cu"], st["start"], h, **rest)
    if c["fp8"]:
        return cw.cowa_decode_paged_fp8(st["q"], kp, vp, st["table"], st["pos"], h, 1 / 64, 1 / 64, **rest)
    return cw.cowa_decode_paged(st["q"], kp, vp, st["table"], st["pos"], h, **rest)


def _cos_sin(turn):
    """cos and sin of p * freq, [tokens, rd / 2]; the angle in 64 bits, as far positions need it."""
    p = turn["pos"].reshape(turn["pos"].shape[0], -1)
    a = p.double()[turn["axis"]].T * turn["freq"].double()
    return a.cos(), a.sin()


def _rotated(x, cos, sin, inter):
    """x [tokens, H, d] in cos's precision, its first rd elements rotated in pairs (i, i + rd/2) or (2i, 2i + 1)."""
    x = x.to(cos.dtype)
    h = cos.shape[1]
    cos, sin = cos[:, None], sin[:, None]
    a, b = (x[..., 0:2 * h:2], x[..., 1:2 * h:2]) if inter else (x[..., :h], x[..., h:2 * h])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((a, b), -1).flatten(-2) if inter else torch.cat((a, b), -1)
    return torch.cat((turned, x[..., 2 * h:]), -1)


def _rope(st):
    c = st["case"]
    cos, sin = (x.float() for x in _cos_sin(st["turn"]))
    if c["bwd"]:
        sin = -sin
    return tuple(_rotated(x.flatten(0, 1), cos, sin, c["inter"]).bfloat16().reshape(x.shape) for x in (st["q"], st["k"]))


def _rows_of(c, table, seq, pos, pages):
    """Page and slot of (sequence, position) for every head, [rows, H]; what has no page goes to the spare one."""
    p = pos.long().clamp(0, c["cap"] - 1)[:, None]
    page = table[seq, :, p[:, 0] // c["page"]] if c["per_head"] else table[seq[:, None], p // c["page"]]
    ok = (pos >= 0)[:, None] & (pos < c["cap"])[:, None] & (page >= 0) & (page < pages)
    return torch.where(ok, page.long(), pages).expand(-1, c["Hkv"]), (p % c["page"]).expand(-1, c["Hkv"])


def _append(st):
    c = st["case"]
    cos, sin = _cos_sin(st["turn"])
    live = (st["pos"] >= 0)[:, None, None]
    q = _rotated(st["q"], cos.float(), sin.float(), c["inter"]).bfloat16()
    q = torch.where(live, q, st["q_out"])
    if c["fp8"]:  # a value next to the border of two codes: the rotation in 64 bits
        new = (_rotated(st["k"], cos, sin, c["inter"]).float(), st["v"].float())
        new = [(x * torch.tensor(64.0)).clamp(-448, 448).to(F8).view(torch.uint8) for x in new]
    else:
        new = (_rotated(st["k"], cos.float(), sin.float(), c["inter"]).bfloat16(), st["v"])
    seq = st["seq"] if st["seq"] is not None else torch.arange(c["total"], device=st["pos"].device)
    page, slot = _rows_of(c, st["table"], seq.long(), st["pos"], st["kp"].shape[0] - 1)
    head = torch.zeros_like(page) if c["per_head"] else torch.arange(c["Hkv"], device=page.device).expand_as(page)
    at = (page, slot, head) if c["layout"] == "bthd" else (page, head, slot)
    st["kp"][at], st["vp"][at] = new
    kp, vp = st["kp"][:-1], st["vp"][:-1]
    return (q, kp.view(F8), vp.view(F8)) if c["fp8"] else (q, kp, vp)


def _values(c, pool, page, slot, head):
    x = pool[page, slot, head] if c["layout"] == "bthd" else pool[page, head, slot]
    return x.view(F8).float() / 64 if x.dtype == torch.uint8 else x.float()


def _softmax(s, see, v):
    """Rows of softmax(s) v over the keys that `see` admits, and the log of the sum; rows that see nothing: 0, -inf."""
    s = s.masked_fill_(~see, -math.inf)
    m = s.amax(-1, keepdim=True)
    m0 = m.masked_fill(m == -math.inf, 0.0)
    p = s.sub_(m0).exp_()
    total = p.sum(-1, keepdim=True)
    return (p @ v) / total.clamp(min=1e-30), (m0 + total.log())[..., 0]


def _decode(st):
    c, dev = st["case"], st["pos"].device
    B, H, cap, d = c["B"], c["Hkv"], c["cap"], c["d"]
    lo, hi = _intervals(c)
    most = min(cap, min(c["S"], cap) + min(c["L"], cap) + min(cap, max(b - a for a, b in zip(lo, hi))))
    t = st["pos"].long().clamp(max=cap - 1)[:, None, None]
    n0 = (t + 1).clamp(max=c["S"])
    band = torch.maximum(t - c["L"] + 1, n0)
    n1 = (torch.minimum(st["hi"][None, :, None], band) - st["lo"][None, :, None]).clamp(min=0)
    j = torch.arange(most, device=dev)[None, None]
    at = torch.where(j < n0, j, torch.where(j < n0 + n1, st["lo"][None, :, None] + j - n0, band + j - n0 - n1))
    see = (j < n0 + n1 + t + 1 - band) & (t >= 0)
    at = torch.where(see, at, 0)
    b, g = torch.arange(B, device=dev)[:, None, None], torch.arange(H, device=dev)[None, :, None]
    page = (st["table"][b, g, at // c["page"]] if c["per_head"] else st["table"][b, at // c["page"]]).long().clamp(min=0)
    head = torch.zeros_like(at) if c["per_head"] else g.expand_as(at)
    k, v = (_values(c, st[x], page, at % c["page"], head) for x in ("kp", "vp"))
    q = st["q"].float().reshape(B, H, -1, d)
    o, lse = _softmax(q @ k.transpose(-1, -2) * d ** -0.5, see[:, :, None], v)
    return o.reshape(B, -1, d).bfloat16(), lse.reshape(B, -1)


def _chunk(st):
    c, dev = st["case"], st["q"].device
    H, d, (mq, mk) = c["Hkv"], c["d"], st["rows"]
    grp, n = c["Hq"] // c["Hkv"], c["n_seq"]
    cu, start = st["cu"].long(), st["start"].long()
    i = torch.arange(mq, device=dev)[None]
    live = i < (cu[1:] - cu[:-1])[:, None]
    row = torch.where(live, cu[:-1, None] + i, 0)
    t = torch.where(live, start[:, None] + i, -1)[:, None, :, None]  # [n, 1, mq, 1]
    s = torch.arange(mk, device=dev)
    page = st["table"][..., s // c["page"]].long().clamp(min=0)
    page = page if c["per_head"] else page[:, None].expand(-1, H, -1)
    head = torch.zeros_like(page) if c["per_head"] else torch.arange(H, device=dev)[None, :, None].expand_as(page)
    k, v = (_values(c, st[x], page, (s % c["page"]).expand_as(page), head) for x in ("kp", "vp"))  # [n, H, mk, d]
    q = st["q"][row].float().reshape(n, mq, H, grp, d).permute(0, 2, 3, 1, 4)
    lo, hi = st["lo"][None, :, None, None], st["hi"][None, :, None, None]
    see = (s <= t) & ((s < c["S"]) | (s > t - c["L"]) | ((s >= lo) & (s < hi)))  # [n, H, mq, mk]
    score = (q.reshape(n, H, grp * mq, d) @ k.transpose(-1, -2)).mul_(d ** -0.5).reshape(n, H, grp, mq, mk)
    o, lse = _softmax(score, see[:, :, None], v[:, :, None])
    where = (torch.arange(c["total"], device=dev)[:, None] >= cu[None, 1:]).sum(1)
    i = torch.arange(c["total"], device=dev) - cu[where]
    o = o.permute(0, 3, 1, 2, 4).reshape(n, mq, c["Hq"], d)[where, i].bfloat16()
    return o, lse.reshape(n, c["Hq"], mq).transpose(1, 2)[where, i].T.contiguous()


# ---------------------------------------------------------------------------------------------- in 64 bits
def exact(c, seed):
    st = prepare(c, seed)
    return {"rope": _exact_rope, "append": _exact_append, "decode": _exact_decode, "chunk": _exact_chunk}[c["op"]](c, st)


def _by_complex(c, x, turn, sign=1.0):
    """Rotation as a product of complex numbers: (a + ib) e^(i angle)."""
    p = turn["pos"].reshape(turn["pos"].shape[0], -1).double()
    h = turn["freq"].numel()
    angle = torch.empty((p.shape[1], h), dtype=torch.float64, device=p.device)
    first = 0
    for a, n in enumerate(turn["sections"]):
        angle[:, first:first + n] = p[a, :, None] * turn["freq"][first:first + n].double()
        first += n
    e = torch.polar(torch.ones_like(angle), sign * angle)[:, None]
    y = x.double().clone()
    if c["inter"]:
        z = torch.view_as_complex(y[..., :2 * h].reshape(*y.shape[:-1], h, 2)) * e
        y[..., :2 * h] = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(y[..., :h], y[..., h:2 * h]) * e
        y[..., :h], y[..., h:2 * h] = z.real, z.imag
    return y


def _exact_rope(c, st):
    return tuple(_by_complex(c, x.flatten(0, 1), st["turn"], -1.0 if c["bwd"] else 1.0).reshape(x.shape)
                 for x in (st["q"], st["k"]))


def _e4m3(x):
    """The nearest E4M3 value (ties to even): steps of 2^(e - 3) in [2^e, 2^(e + 1)), 2^-9 below 2^-6, at most 448."""
    e = torch.frexp(x.abs().clamp(min=2.0 ** -6))[1].double() - 1
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_append(c, st):
    q, k = _by_complex(c, st["q"], st["turn"]), _by_complex(c, st["k"], st["turn"])
    v = st["v"].double()
    value = (lambda x: x.view(F8).double()) if c["fp8"] else (lambda x: x.double())
    kp, vp = value(st["kp"]), value(st["vp"])
    if c["fp8"]:
        k, v = _e4m3(64 * k), _e4m3(64 * v)
    rows = torch.tensor(_append_rows(c), device=q.device)
    ok = rows[:, 1] >= 0
    i = torch.nonzero(ok)[:, 0]
    s, p = rows[i, 0], rows[i, 1]
    for g in range(c["Hkv"]):
        page = (st["table"][s, g, p // c["page"]] if c["per_head"] else st["table"][s, p // c["page"]]).long()
        held = page >= 0
        page, slot, src = page[held], (p % c["page"])[held], i[held]
        h = 0 if c["per_head"] else g
        for pool, new in ((kp, k), (vp, v)):
            if c["layout"] == "bthd":
                pool[page, slot, h] = new[src, g]
            else:
                pool[page, h, slot] = new[src, g]
    return torch.where(ok[:, None, None], q, 0.0), kp[:-1], vp[:-1]


def _exact_rows(c, st, b, n):
    """Keys and values 0 .. n-1 of sequence b in 64 bits, [H, n, d]; zeros where a head has no page."""
    s = torch.arange(n, device=st["table"].device)
    out = []
    for pool in (st["kp"], st["vp"]):
        heads = []
        for g in range(c["Hkv"]):
            page = (st["table"][b, g] if c["per_head"] else st["table"][b])[s // c["page"]].long()
            h, at = (0 if c["per_head"] else g), page.clamp(min=0)
            x = pool[at, s % c["page"], h] if c["layout"] == "bthd" else pool[at, h, s % c["page"]]
            x = x.view(F8).double() / 64 if x.dtype == torch.uint8 else x.double()
            heads.append(torch.where((page >= 0)[:, None], x, 0.0))
        out.append(torch.stack(heads))
    return out


def _exact_attention(c, q, k, v, t, g):
    """Query rows q [rows, d] of head group g at positions t against keys 0 .. n-1."""
    lo, hi = _intervals(c)
    s = torch.arange(k.shape[0], device=k.device)[None]
    t = t[:, None]
    see = (s <= t) & ((s < c["S"]) | (s > t - c["L"]) | ((s >= lo[g]) & (s < hi[g])))
    x = torch.where(see, (q.double() @ k.T) / math.sqrt(c["d"]), -math.inf)
    lse = torch.logsumexp(x, 1)
    return torch.exp(x - lse[:, None]) @ v, lse


def _exact_decode(c, st):
    B, grp = c["B"], c["Hq"] // c["Hkv"]
    o = torch.zeros((B, c["Hq"], c["d"]), dtype=torch.float64, device=st["q"].device)
    lse = torch.full((B, c["Hq"]), -math.inf, dtype=torch.float64, device=o.device)
    for b, t in enumerate(_positions(c)):
        if t < 0:
            continue
        k, v = _exact_rows(c, st, b, t + 1)
        for g in range(c["Hkv"]):
            hs = slice(g * grp, (g + 1) * grp)
            at = torch.full((grp,), t, device=o.device)
            o[b, hs], lse[b, hs] = _exact_attention(c, st["q"][b, hs], k[g], v[g], at, g)
    return o, lse


def _exact_chunk(c, st):
    grp = c["Hq"] // c["Hkv"]
    o = torch.zeros((c["total"], c["Hq"], c["d"]), dtype=torch.float64, device=st["q"].device)
    lse = torch.zeros((c["Hq"], c["total"]), dtype=torch.float64, device=o.device)
    first = 0
    for b, (p0, n) in enumerate(_chunks(c)):
        k, v = _exact_rows(c, st, b, p0 + n)
        for h in range(c["Hq"]):
            at = torch.arange(p0, p0 + n, device=o.device)
            r = slice(first, first + n)
            o[r, h], lse[h, r] = _exact_attention(c, st["q"][r, h], k[h // grp], v[h // grp], at, h // grp)
        first += n
    return o, lse
