"""Timed cases of a decode step's way through an 8-bit cache: positions rotated in, rows written, attention.

Each case is one pass as a serving program makes it.  `own` chooses between the
plain torch form and the library's calls (transformer_layer_decode_gb300.kv
and .rope).

The cache is the paged one of perf/operators.py.  An 8-bit ("q8") page holds,
first for K and then for V, [kv head][row][head_dim] bytes, each a code + 128,
and behind them [kv head][row / 16] fp32 scales, powers of two, filled up to a
multiple of 64 bytes.  A block is 16 rows of one head: its scale is the least
power of two s with |x| <= 127 s for all its rows, the codes are x / s rounded
to the nearest, ties to even.  A call that writes rows of a block keeps those
before the first that it writes: the scale does not fall below the old one then,
and where it rises the kept codes are divided and rounded to the new steps.

Rotary positions turn pairs of the first `rot` dimensions of a head by position *
frequency: dimensions i and i + rot / 2 ("half") or 2 i and 2 i + 1
("interleaved"), frequency i being theta^(-2 i / rot), changed by `scaling`.
"""
import math
import random

import numpy as np
import torch

own = False


# ---- the cases -----------------------------------------------------------------

def listed():
    return [
        # one decode step of the hidden-512 layer: latency alone
        dict(name="attend_one_token", op="attend", fmt="q8", io="fp32", batch=1, heads=8, kv_heads=2, head_dim=64,
             page=128, layers=2, longest=127, window=0, sinks=0, padded=0, mix=1),
        # one stream of the 9B shape (grouped heads)
        dict(name="attend_stream", op="attend", fmt="q8", io="fp32", batch=1, heads=32, kv_heads=8, head_dim=128,
             page=64, layers=2, longest=4095, window=0, sinks=0, padded=0, mix=2),
        # a ragged batch of the 1B shape, fp32 in and out
        dict(name="attend_grouped", op="attend", fmt="q8", io="fp32", batch=16, heads=32, kv_heads=8, head_dim=64,
             page=128, layers=1, longest=8192, window=0, sinks=0, padded=0, mix=3),
        # a ragged batch of the 7B shape with a sliding window and first tokens that stay
        dict(name="attend_window", op="attend", fmt="q8", io="bf16", batch=48, heads=32, kv_heads=32, head_dim=128,
             page=64, layers=1, longest=8190, window=2048, sinks=16, padded=2, mix=4),
        # long contexts of the 7B shape, what eight bits are for
        dict(name="attend_batch", op="attend", fmt="q8", io="bf16", batch=24, heads=32, kv_heads=32, head_dim=128,
             page=64, layers=1, longest=24001, window=0, sinks=0, padded=0, mix=5),
        # the rows of one decode step of a batch, one behind each sequence, and their blocks read back
        dict(name="rows_decode", op="rows", fmt="q8", io="fp32", tokens=32, seqs=32, kv_heads=8, head_dim=128,
             page=64, layers=2, order="last", padded=0, mix=6),
        # the rows of a prefill
        dict(name="rows_prefill", op="rows", fmt="q8", io="bf16", tokens=8185, seqs=5, kv_heads=32, head_dim=128,
             page=64, layers=1, order="runs", padded=0, mix=7),
        # the queries of one decode step of the hidden-512 layer: latency alone
        dict(name="rotate_one_token", op="rotate", io="fp32", tokens=1, heads=8, head_dim=64, rot=64, layout="half",
             scaling="none", theta=1e4, factor=1.0, context=2048, longest=128, back=False, packed=0, padded=0, mix=8),
        # the queries of a prefill of the 7B shape, trained on a shorter context, cut from the projection's rows
        dict(name="rotate_prefill", op="rotate", io="bf16", tokens=8185, heads=32, head_dim=128, rot=128, layout="half",
             scaling="yarn", theta=1e4, factor=8.0, context=2048, longest=16384, back=False, packed=64, padded=0, mix=9),
        # the gradient of rotated queries: part of the head, neighbouring pairs, far positions
        dict(name="rotate_back", op="rotate", io="fp32", tokens=2049, heads=32, head_dim=128, rot=64,
             layout="interleaved", scaling="linear", theta=5e5, factor=4.0, context=8192, longest=1000000, back=True,
             packed=0, padded=0, mix=10),
        # a decode step of a batch: queries and keys rotated, the rows written in 8 bits, their blocks read back
        dict(name="step_decode", op="step", fmt="q8", io="bf16", tokens=32, seqs=32, heads=32, kv_heads=8, head_dim=128,
             page=64, layers=2, order="last", rot=128, layout="half", scaling="none", theta=1e4, factor=1.0,
             context=2048, padded=0, mix=11),
        # the same of a prompt's rows
        dict(name="step_prefill", op="step", fmt="q8", io="bf16", tokens=4093, seqs=3, heads=32, kv_heads=8,
             head_dim=128, page=64, layers=1, order="runs", rot=128, layout="half", scaling="yarn", theta=1e4,
             factor=4.0, context=2048, padded=0, mix=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _rotation(rng, head_dim):
    return dict(rot=rng.choice([head_dim, head_dim, head_dim // 2, head_dim // 4, 2 * rng.randint(2, head_dim // 2)]),
                layout=rng.choice(["half", "interleaved"]), scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                theta=rng.choice([1e4, 5e5]), factor=rng.choice([2.0, 4.0, 8.0, 2.5]),
                context=rng.choice([2048, 4096, 8192]))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "rows", "rotate", "rotate", "step", "step"])
    mix, io = rng.randrange(1 << 30), rng.choice(["fp32", "bf16"])
    hd, page = rng.choice([64, 128]), rng.choice([16, 32, 48, 64, 128])
    if op == "attend":
        kvh, group = rng.choice([1, 2, 3, 4, 8, 16, 32]), rng.choice([1, 1, 2, 3, 4, 5, 8, 12])
        batch = _log(rng, 1, 64)
        most = 2_200_000_000 // (batch * kvh * hd * 2)
        window = rng.choice([0, max(1, min(most, _log(rng, 1, 16384)))])
        longest = _log(rng, 1, 65536 if window else min(65536, max(1, most)))
        return dict(op=op, fmt="q8", io=io, batch=batch, heads=kvh * group, kv_heads=kvh, head_dim=hd, page=page,
                    layers=rng.choice([1, 2]), longest=longest, window=window,
                    sinks=rng.choice([0, 1, 4, rng.randrange(1, 200)]) if window else 0,
                    padded=rng.choice([0, 0, 1, 3]) if batch > 3 else 0, mix=mix)
    if op == "rotate":
        hd = rng.choice([64, 128, 80, 96, 256])
        return dict(op=op, io=io, tokens=_log(rng, 1, 8000), heads=rng.choice([1, 2, 5, 8, 32]), head_dim=hd,
                    longest=_log(rng, 1, 1 << 20), back=rng.random() < 0.4, packed=rng.choice([0, 0, 2, 8]),
                    padded=rng.choice([0, 0, 1, 5]), mix=mix, **_rotation(rng, hd))
    seqs = _log(rng, 1, 64)
    order = rng.choice(["last", "runs", "runs", "mixed"])
    case = dict(op=op, fmt="q8", io=io, tokens=seqs if order == "last" else max(seqs, _log(rng, 1, 6000)), seqs=seqs,
                kv_heads=rng.choice([1, 2, 3, 8, 16]), head_dim=hd, page=page, layers=rng.choice([1, 2]), order=order,
                padded=rng.choice([0, 1, 5]), mix=mix)
    if op == "step":
        case.update(fmt=rng.choice(["q8", "q8", "q4", "bf16"]), heads=case["kv_heads"] * rng.choice([1, 2, 4, 5]),
                    **_rotation(rng, hd))
    return case


def lengths(case):
    """The sequences' lengths: the longest, an empty one where there are many, others between."""
    n, rng = case["batch"], random.Random(case["mix"])
    longest = case["longest"]
    out = [longest] + [rng.randint(longest // 8, longest) for _ in range(n - 1)]
    if n > 3:
        out[n // 2] = 0
    return out


def visible(n, window, sinks):
    """(first rows, start of the window) that a query behind n rows sees."""
    lo = max(n - window, 0) if window else 0
    return min(sinks, lo), lo


def token_plan(case):
    """Which sequence and position each row goes to, the sequences' lengths after it, and the rows to read back:
    what blocks of 16 that are written to hold, the rows written and those before the first of them."""
    rng = random.Random(case["mix"])
    n, s = case["tokens"], case["seqs"]
    cuts = sorted(rng.randint(0, n) for _ in range(s - 1)) if n > s else list(range(1, s))
    counts = [b - a for a, b in zip([0] + cuts, cuts + [n])]
    before = [rng.randint(0, 500) for _ in range(s)]
    plan = [(i, before[i] + j) for i, c in enumerate(counts) for j in range(c)]
    if case["order"] == "mixed":
        rng.shuffle(plan)
    for i in range(min(case["padded"], n - 1)):
        plan[n - 1 - i] = (-1, 0)
    rows = {}
    for i, p in plan:
        if i >= 0:
            rows.setdefault((i, p // 16), set()).add(p % 16)
    back = [(i, 16 * b + r) for (i, b), new in sorted(rows.items()) for r in sorted(new | set(range(min(new))))]
    return plan, [b + c for b, c in zip(before, counts)], back if case["fmt"] == "q8" else [x for x in plan if x[0] >= 0]


def row_bytes(case):
    """K and V of one position of one kv head."""
    d = case["head_dim"]
    return {"bf16": 4 * d, "q4": d + d // 8, "q8": 2 * d + 0.5}[case["fmt"]]


def half_bytes(case):
    """K, or V, of a page."""
    d, rows = case["head_dim"], case["kv_heads"] * case["page"]
    if case["fmt"] == "q8":
        return -(-(rows * d + rows // 4) // 64) * 64
    return rows * (2 * d if case["fmt"] == "bf16" else d // 2 + d // 16)


def work(case):
    io, d = 4 if case["io"] == "fp32" else 2, case["head_dim"]
    if case["op"] == "attend":
        n = case["batch"] - case["padded"]
        rows = sum(first + length - lo for length in lengths(case)[:n]
                   for first, lo in [visible(length, case["window"], case["sinks"])])
        return {"bytes": rows * case["kv_heads"] * row_bytes(case) + io * 2 * n * case["heads"] * d,
                "flops": 4 * rows * case["heads"] * d}
    n = case["tokens"] - min(case["padded"], case["tokens"] - 1)
    if case["op"] == "rotate":
        return {"bytes": 2 * io * n * case["heads"] * d, "flops": 3 * n * case["heads"] * case["rot"]}
    back, values = len(token_plan(case)[2]), case["kv_heads"] * d
    w = {"bytes": 2 * n * values * io + (n + back) * case["kv_heads"] * row_bytes(case) + 2 * back * values * io,
         "flops": 2 * (n + back) * values}
    if case["op"] == "step":
        w["bytes"] += 2 * io * n * case["heads"] * d + 2 * back * values * (2 - io)  # (read back in bf16)
        w["flops"] += 3 * n * (case["heads"] + case["kv_heads"]) * case["rot"]
    return w


# ---- inputs ---------------------------------------------------------------------

def _parts8(pool, case):
    """codes [layers][pages][K, V][kv head][row][dim] and scales [layers][pages][K, V][kv head][block] of 8-bit pages"""
    R, kvh, d = case["page"], case["kv_heads"], case["head_dim"]
    halves = pool.unflatten(-1, (2, half_bytes(case)))
    codes, rest = halves[..., :kvh * R * d], halves[..., kvh * R * d:kvh * R * d + kvh * R // 4]
    return codes.unflatten(-1, (kvh, R, d)), rest.view(torch.float32).unflatten(-1, (kvh, R // 16))


def _parts4(pool, case):
    """codes [...][row][bytes] and scales [...][row][block of 32 dimensions] (fp16) of 4-bit pages"""
    R, d = case["page"], case["head_dim"]
    heads = pool.unflatten(-1, (2, case["kv_heads"], R * (d // 2 + d // 16)))
    codes = heads[..., :R * d // 2].unflatten(-1, (R, d // 2))
    return codes, heads[..., R * d // 2:].view(torch.float16).unflatten(-1, (R, d // 32))


def _parts16(pool, case):
    """bf16 values [layers][pages][K, V][kv head][row][dim]"""
    return pool.view(torch.bfloat16).unflatten(-1, (2, case["kv_heads"], case["page"], case["head_dim"]))


def _pool(case, pages, gen, low=(-7, -7)):
    """A pool of random rows; of 8 bits with scales 2^low to 2^(low + 1) for K and for V."""
    shape = (case["layers"], pages, 2 * half_bytes(case))
    if case["fmt"] == "bf16":
        return torch.randn(shape[:2] + (shape[2] // 2,), device="cuda", dtype=torch.bfloat16, generator=gen).view(torch.uint8)
    pool = torch.randint(1, 256, shape, device="cuda", dtype=torch.uint8, generator=gen)
    if case["fmt"] == "q4":
        scales = _parts4(pool, case)[1]
        scales.copy_(torch.rand(scales.shape, device="cuda", generator=gen).mul_(0.2).add_(0.1))
        return pool
    scales = _parts8(pool, case)[1]
    e = torch.randint(0, 2, scales.shape, device="cuda", generator=gen)
    scales.copy_(torch.exp2((e + torch.tensor(low, device="cuda")[:, None, None]).float()))
    return pool


def _int(a):
    return torch.tensor(np.asarray(a, np.int32), device="cuda")


def _tables(case, lens, wanted, spare, rng):
    """table, refs: a page at random for each (sequence, page of it) wanted."""
    order = rng.permutation(len(wanted) + spare)
    table = np.full((len(lens), max(1, max(-(-n // case["page"]) for n in lens))), -1, np.int32)
    for (s, i), p in zip(wanted, order):
        table[s, i] = p
    refs = np.zeros(len(order), np.int32)
    refs[order[:len(wanted)]] = 1
    return dict(table=_int(table), lens=_int(lens), refs=_int(refs)), len(order)


def frequencies(case):
    """Radians per position of each pair, and what the rotated values are multiplied by."""
    rot, f = case["rot"], case["factor"]
    theta = case["theta"] * (f ** (rot / (rot - 2)) if case["scaling"] == "ntk" else 1)
    w = theta ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    if case["scaling"] == "linear":
        w = w / f
    if case["scaling"] == "yarn":  # by how often a pair turns over the context: 32 times, kept; once, divided
        keep = np.clip((case["context"] * w / (2 * math.pi) - 1) / 31, 0, 1)
        w = w * keep + w / f * (1 - keep)
    return w, 0.1 * math.log(f) + 1 if case["scaling"] == "yarn" else 1.0


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.RandomState(seed % (1 << 31))
    st, d = {"case": dict(case)}, case["head_dim"]
    io = torch.float32 if case["io"] == "fp32" else torch.bfloat16
    if "rot" in case:
        w, st["magnitude"] = frequencies(case)
        st["turns"] = torch.tensor(w, device="cuda")
    if case["op"] == "rotate":
        n, pad = case["tokens"], min(case["padded"], case["tokens"] - 1)
        rows = torch.randn((n, case["heads"] + case["packed"], d), device="cuda", generator=gen).to(io)
        pos = rng.randint(0, case["longest"], n)
        pos[n - pad:] = -1
        st.update(x=rows[:, :case["heads"]], positions=_int(pos),
                  out=torch.zeros((n, case["heads"], d), device="cuda", dtype=io))
        return st
    R = case["page"]
    if case["op"] == "attend":
        lens = lengths(case)
        first = [visible(n, case["window"], case["sinks"]) for n in lens]
        wanted = [(s, i) for s, n in enumerate(lens) for i in range(-(-n // R))
                  if i * R < first[s][0] or (i + 1) * R > first[s][1]]
        tables, pages = _tables(case, lens, wanted, 1, rng)
        seqs = [s if s < case["batch"] - case["padded"] else -1 for s in range(case["batch"])]
        shape = (case["batch"], case["heads"], d)
        st.update(tables, pool=_pool(case, pages, gen), seqs=_int(seqs),
                  q=torch.randn(shape, device="cuda", generator=gen).to(io),
                  out=torch.zeros(shape, device="cuda", dtype=io),
                  span=max(1, max(a + n - lo for n, (a, lo) in zip(lens, first))))
        return st
    plan, lens, back = token_plan(case)
    wanted = [(s, i) for s, n in enumerate(lens) for i in range(-(-n // R))]
    tables, pages = _tables(case, lens, wanted, 1, rng)
    shape = (case["tokens"], case["kv_heads"], d)
    # keys as they come: a few dimensions much larger than the rest; the kept rows' blocks now and then get new scales
    big = 1 + 7 * (torch.rand(d, device="cuda", generator=gen) < 0.05)
    k, v = (torch.randn(shape, device="cuda", generator=gen) for _ in range(2))
    st.update(tables, pool=_pool(case, pages, gen, (-4, -6)), seqs=_int([i for i, _ in plan]),
              positions=_int([p for _, p in plan]), k=(k * big).to(io), v=v.to(io),
              back_seqs=_int([i for i, _ in back]), back_positions=_int([p for _, p in back]))
    # of a step the rotated values' last bits are not fixed, and then neither are the codes of a few: read as bf16
    to = torch.bfloat16 if case["op"] == "step" else io
    st.update(k_out=torch.zeros((len(back),) + shape[1:], device="cuda", dtype=to),
              v_out=torch.zeros((len(back),) + shape[1:], device="cuda", dtype=to))
    if case["op"] == "step":
        q = torch.randn((case["tokens"], case["heads"], d), device="cuda", generator=gen).to(io)
        st.update(q=q, q_out=torch.zeros_like(q))
    return st


# ---- one pass -------------------------------------------------------------------

def run(st):
    if own:
        return _run_own(st)
    return {"attend": _attend, "rows": _rows, "rotate": _rotate, "step": _step}[st["case"]["op"]](st)


def _cache(st):
    """The library's view of the state's tensors: made once, as a serving program keeps it."""
    if "cache" not in st:
        from transformer_layer_decode_gb300 import kv
        c = st["case"]
        st["cache"] = kv.KVCache(n_layers=c["layers"], n_kv_heads=c["kv_heads"], head_dim=c["head_dim"],
                                 page_rows=c["page"], fmt=c["fmt"], pool=st["pool"], table=st["table"],
                                 lens=st["lens"], refs=st["refs"])
    return st["cache"]


def _rotary(st):
    """The model's rotation: made once."""
    if "rotary" not in st:
        from transformer_layer_decode_gb300 import rope
        c = st["case"]
        st["rotary"] = rope.Rotary(c["head_dim"], rot_dim=c["rot"], layout=c["layout"], theta=c["theta"],
                                   scaling=None if c["scaling"] == "none" else c["scaling"], factor=c["factor"],
                                   context=c["context"])
    return st["rotary"]


def _run_own(st):
    case = st["case"]
    if case["op"] == "rotate":
        return _rotary(st).rotate(st["x"], st["positions"], out=st["out"], backward=case["back"])
    cache, layer = _cache(st), case["layers"] - 1
    if case["op"] == "attend":
        return cache.attention(layer, st["q"], seqs=st["seqs"], window=case["window"], sinks=case["sinks"],
                               out=st["out"])
    positions = None if case["order"] == "last" else st["positions"]
    if case["op"] == "step":
        cache.append_rotated(layer, _rotary(st), st["q"], st["k"], st["v"], seqs=st["seqs"], positions=positions,
                             q_out=st["q_out"])
    else:
        cache.append(layer, st["k"], st["v"], seqs=st["seqs"], positions=positions)
    back = cache.read(layer, st["back_seqs"], st["back_positions"], k_out=st["k_out"], v_out=st["v_out"])
    return (st["q_out"],) + back if case["op"] == "step" else back


def _gather(st, which, page, row):
    """Rows of K (0) or V (1) of the last layer as fp32 [..., kv head, dim], by page and row of the page."""
    case, pool = st["case"], st["pool"][st["case"]["layers"] - 1]
    if case["fmt"] == "bf16":
        return _parts16(pool, case)[:, which][page, :, row].float()
    if case["fmt"] == "q8":
        codes, scales = _parts8(pool, case)
        x = codes[:, which][page, :, row].float().sub_(128)
        return x.mul_(scales[:, which][page, :, row // 16][..., None])
    codes, scales = _parts4(pool, case)
    b, s = codes[:, which][page, :, row], scales[:, which][page, :, row]
    n = torch.stack((b & 15, b >> 4), -1).flatten(-2)
    n = n.unflatten(-1, (8, case["head_dim"] // 32, 4)).transpose(-3, -2).flatten(-2)
    return ((n.float() - 8) * s.float()[..., None]).flatten(-2)


def _attend(st):
    case, table = st["case"], st["table"]
    R, kvh = case["page"], case["kv_heads"]
    seq = st["seqs"].long().clamp(min=0)
    n = torch.where(st["seqs"] >= 0, st["lens"][seq], 0)[:, None]
    lo = (n - case["window"]).clamp(min=0) if case["window"] else torch.zeros_like(n)
    first = lo.clamp(max=case["sinks"])
    j = torch.arange(st["span"], device=n.device)[None]
    seen = j < first + n - lo
    pos = torch.where(seen, torch.where(j < first, j, lo + j - first), 0)
    page = table[seq[:, None], pos // R].long().clamp(min=0)
    q = st["q"].float().unflatten(1, (kvh, case["heads"] // kvh))
    s = torch.matmul(q, _gather(st, 0, page, pos % R).permute(0, 2, 3, 1)) / math.sqrt(case["head_dim"])
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    w = torch.exp(s - torch.where(top == -math.inf, 0, top))
    o = torch.matmul(w, _gather(st, 1, page, pos % R).permute(0, 2, 1, 3))
    total = w.sum(-1, keepdim=True)
    return torch.where(total > 0, o / total, 0).flatten(1, 2).to(st["out"].dtype)


def _turn(st, x, positions, back=False):
    """x [n, heads, head_dim] rotated, in fp32: angles in 64 bits."""
    case, rot = st["case"], st["case"]["rot"]
    angle = positions.double()[:, None, None] * st["turns"]
    c, s = ((f(angle) * st["magnitude"]).float() for f in (torch.cos, torch.sin))
    s = -s if back else s
    x = x.float()
    if case["layout"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        return torch.cat((a * c - b * s, b * c + a * s, x[..., rot:]), -1)
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    return torch.cat((torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2), x[..., rot:]), -1)


def _rotate(st):
    y = _turn(st, st["x"], st["positions"], st["case"]["back"])
    return torch.where((st["positions"] >= 0)[:, None, None], y, 0).to(st["out"].dtype)


def _store8(codes, scales, block, row, x):
    """Rows x [n][K, V][kv head][dim] written into codes [blocks][16][K, V][kv head][dim] with scales
    [blocks][K, V][kv head]: both as they are then."""
    m, e = torch.frexp(x.abs().amax(-1))  # |x| = m 2^e, 1/2 <= m < 1: within 127 2^(e - 7) if m <= 127 / 128
    need = torch.where(m > 0, e - 7 + (m > 127 / 128).int(), -126).clamp(-126, 121)
    first = torch.full((len(codes),), 16, device=x.device).scatter_reduce(0, block, row, "amin")
    old = torch.frexp(scales).exponent - 1
    top = torch.full_like(old, -126).scatter_reduce(0, block[:, None, None].expand_as(need), need, "amax")
    touched, keeps = (first < 16)[:, None, None], (first > 0)[:, None, None]
    new = torch.where(touched, torch.where(keeps, torch.maximum(top, old), top), old)
    kept = torch.arange(16, device=x.device)[None] < torch.where(first < 16, first, 0)[:, None]
    fewer = (codes.float() - 128) * torch.exp2((old - new).float())[:, None, :, :, None]
    codes = torch.where(kept[:, :, None, None, None], fewer.round().add(128).to(torch.uint8), codes)
    step = torch.exp2(new.double())
    codes[block, row] = (x / step[block][..., None]).round().clamp(-127, 127).add(128).to(torch.uint8)
    return codes, torch.where(touched, step.float(), scales)


def _store(st, k, v):
    """Writes rows k and v (fp32) of the listed tokens into the last layer's pages."""
    case, pool = st["case"], st["pool"][st["case"]["layers"] - 1]
    R, d, real = case["page"], case["head_dim"], st["seqs"] >= 0
    seq, pos = st["seqs"][real].long(), st["positions"][real].long()
    page, row = st["table"][seq, pos // R].long(), pos % R
    x = torch.stack((k[real], v[real]), 1)
    if case["fmt"] == "bf16":
        _parts16(pool, case)[page, :, :, row] = x.to(torch.bfloat16)
    elif case["fmt"] == "q4":
        x = x.unflatten(-1, (d // 32, 32))
        s = (x.abs().amax(-1) / 7).clamp(max=65504).half()
        step = s.double()[..., None]
        n = torch.where(step > 0, x.double() / step, 0).round().clamp(-8, 7).int() + 8
        n = n.unflatten(-1, (8, 4)).transpose(-3, -2).flatten(-3)
        codes, scales = _parts4(pool, case)
        codes[page, :, :, row] = (n[..., 0::2] | (n[..., 1::2] << 4)).to(torch.uint8)
        scales[page, :, :, row] = s
    else:
        codes, scales = _parts8(pool, case)
        rows, steps = _store8(codes.permute(0, 3, 1, 2, 4).unflatten(1, (R // 16, 16)).flatten(0, 1),
                              scales.permute(0, 3, 1, 2).flatten(0, 1), page * (R // 16) + row // 16, row % 16, x)
        codes.copy_(rows.unflatten(0, (-1, R // 16)).flatten(1, 2).permute(0, 2, 3, 1, 4))
        scales.copy_(steps.unflatten(0, (-1, R // 16)).permute(0, 2, 3, 1))


def _read(st):
    R, seq, pos = st["case"]["page"], st["back_seqs"].long(), st["back_positions"].long()
    page = st["table"][seq, pos // R].long()
    return tuple(_gather(st, which, page, pos % R).to(st["k_out"].dtype) for which in (0, 1))


def _rows(st):
    _store(st, st["k"].float(), st["v"].float())
    return _read(st)


def _step(st):
    real = (st["seqs"] >= 0)[:, None, None]
    q = torch.where(real, _turn(st, st["q"], st["positions"]), 0).to(st["q"].dtype)
    _store(st, _turn(st, st["k"], st["positions"]), st["v"].float())
    return (q,) + _read(st)


# ---- the definition in 64 bits ----------------------------------------------------

def _exact_turn(case, x, positions, back):
    """As complex numbers."""
    w, m = frequencies(case)
    rot, x = case["rot"], x.double().cpu().numpy()
    z = m * np.exp((-1j if back else 1j) * positions.cpu().numpy().astype(np.float64)[:, None, None] * w)
    y = x.copy()
    at = [(i, i + rot // 2) if case["layout"] == "half" else (2 * i, 2 * i + 1) for i in range(rot // 2)]
    a, b = [i for i, _ in at], [j for _, j in at]
    t = (x[..., a] + 1j * x[..., b]) * z
    y[..., a], y[..., b] = t.real, t.imag
    return y


def _exact_blocks(case, st, x, which, plan, back):
    """Rows x (fp64 [token][kv head][dim]) written, block after block, and the rows `back` of what is then there."""
    R, d, kvh = case["page"], case["head_dim"], case["kv_heads"]
    pool, table = st["pool"][case["layers"] - 1].cpu().numpy(), st["table"].cpu().numpy()
    half = half_bytes(case)
    of, out = {}, {}
    for t, (s, p) in enumerate(plan):
        if s >= 0:
            of.setdefault((s, p // 16), {})[p % 16] = t
    for (s, b), rows in of.items():
        page, at = pool[table[s, b * 16 // R]][which * half:(which + 1) * half], b * 16 % R
        codes = page[:kvh * R * d].reshape(kvh, R, d)[:, at:at + 16].astype(np.float64) - 128
        scale = page[kvh * R * d:kvh * R * d + kvh * R // 4].view(np.float32).reshape(kvh, R // 16)[:, at // 16]
        first, values = min(rows), np.zeros((16, kvh, d))
        new = x[list(rows.values())]
        top = np.abs(new).max((0, 2))
        e = np.full(kvh, -126)
        for h in range(kvh):
            while top[h] > 127 * 2.0 ** e[h] and e[h] < 121:
                e[h] += 1
        s_new = 2.0 ** e
        if first:
            s_new = np.maximum(s_new, scale.astype(np.float64))
            for r in range(first):
                values[r] = np.rint(codes[:, r] * (scale / s_new)[:, None]) * s_new[:, None]
        for r, t in rows.items():
            values[r] = np.clip(np.rint(x[t] / s_new[:, None]), -127, 127) * s_new[:, None]
        out[s, b] = values
    return np.stack([out[s, p // 16][p % 16] for s, p in back])


def _exact_rows(case, st, x, which, plan, back):
    if case["fmt"] == "q8":
        return _exact_blocks(case, st, x, which, plan, back)
    x = x[[t for t, (s, _) in enumerate(plan) if s >= 0]]
    if case["fmt"] == "bf16":
        return torch.from_numpy(x).to(torch.bfloat16).double().numpy()
    b = x.reshape(*x.shape[:-1], -1, 32)
    s = np.minimum(np.abs(b).max(-1, keepdims=True) / 7, 65504).astype(np.float16).astype(np.float64)
    with np.errstate(all="ignore"):
        return (np.where(s > 0, np.clip(np.rint(b / s), -8, 7), 0) * s).reshape(x.shape)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rotate":
        y = _exact_turn(case, st["x"], st["positions"], case["back"])
        y[st["positions"].cpu().numpy() < 0] = 0
        return torch.from_numpy(y)
    if case["op"] != "attend":
        plan, _, back = token_plan(case)
        k, v, pad = st["k"].double().cpu().numpy(), st["v"].double().cpu().numpy(), [s < 0 for s, _ in plan]
        outs = []
        if case["op"] == "step":
            q, k = (_exact_turn(case, st[name], st["positions"], False) for name in ("q", "k"))
            q[pad] = 0
            outs.append(torch.from_numpy(q))
        outs += [torch.from_numpy(_exact_rows(case, st, x, i, plan, back)) for i, x in enumerate((k, v))]
        return tuple(outs)
    R, d, kvh, heads = case["page"], case["head_dim"], case["kv_heads"], case["heads"]
    table, lens, pool = st["table"].cpu().numpy(), st["lens"].cpu().numpy(), st["pool"][case["layers"] - 1]
    out = torch.zeros(case["batch"], heads, d, dtype=torch.float64, device="cuda")
    for b in range(case["batch"] - case["padded"]):
        n = int(lens[b])
        pos = np.array([p for p in range(n) if not case["window"] or p >= n - case["window"] or p < case["sinks"]], np.int64)
        if not len(pos):
            continue
        pages, which = np.unique(table[b][pos // R], return_inverse=True)
        raw = pool[torch.tensor(pages, device="cuda").long()].reshape(len(pages), 2, half_bytes(case))
        at, row = torch.tensor(which.reshape(-1), device="cuda"), torch.tensor(pos % R, device="cuda")
        codes = raw[:, :, :kvh * R * d].reshape(len(pages), 2, kvh, R, d)
        scales = raw[:, :, kvh * R * d:kvh * R * d + kvh * R // 4].contiguous().view(torch.float32)
        scales = scales.reshape(len(pages), 2, kvh, R // 16)
        for h in range(kvh):
            k, v = ((codes[:, i, h][at, row].double() - 128) * scales[:, i, h][at, row // 16].double()[:, None]
                    for i in (0, 1))
            group = slice(h * heads // kvh, (h + 1) * heads // kvh)
            out[b, group] = torch.softmax(k @ st["q"][b, group].double().T / math.sqrt(d), 0).T @ v
    return out
