"""Timed cases of the paged key/value cache: attention over it, its rows, its pages.

Each case is one pass as a serving program makes it.  `own` chooses between the
plain torch form and the library's calls (transformer_layer_decode_gb300.kv).

The cache: a pool of pages, uint8 [layers][pages][page_bytes].  A page holds
`page` positions, K first and V after it, each [kv head][positions][head_dim]:
bf16, or ("q4") per kv head the 4-bit codes of all positions (head_dim / 2
bytes each) and after them the fp16 scales (head_dim / 32 each).  Dimension
32 b + 4 g + i of a row (block b, g < 8, i < 4) is nibble (g * blocks + b) * 4 + i,
low nibble first, stored as code + 8.  table[s][i] is the page of positions
[i * page, (i + 1) * page) of sequence s or -1, lens[s] its length, refs[p]
how many tables name page p.
"""
import math
import random

import numpy as np
import torch

own = False


# ---- the cases -----------------------------------------------------------------

def listed():
    return [
        # one decode step of the hidden-512 layer with a short window: latency alone
        dict(name="window_one_token", op="attend", fmt="bf16", io="fp32", batch=1, heads=8, kv_heads=2,
             head_dim=64, page=128, layers=2, longest=128, window=64, sinks=4, padded=0, mix=1),
        # one long stream at the largest context: a window of it and the first tokens
        dict(name="window_long_stream", op="attend", fmt="bf16", io="fp32", batch=1, heads=32, kv_heads=8,
             head_dim=128, page=64, layers=2, longest=65536, window=8192, sinks=4, padded=0, mix=2),
        # a ragged batch of the 7B shape, bf16 in and out, windowed
        dict(name="window_batch", op="attend", fmt="bf16", io="bf16", batch=48, heads=32, kv_heads=32,
             head_dim=128, page=64, layers=1, longest=8190, window=2048, sinks=16, padded=2, mix=3),
        # one decode step of the hidden-512 layer over 4 bits
        dict(name="q4_one_token", op="attend", fmt="q4", io="fp32", batch=1, heads=8, kv_heads=2,
             head_dim=64, page=128, layers=2, longest=127, window=0, sinks=0, padded=0, mix=4),
        # one stream of the 9B shape (grouped heads) over 4 bits
        dict(name="q4_stream", op="attend", fmt="q4", io="fp32", batch=1, heads=32, kv_heads=8,
             head_dim=128, page=64, layers=2, longest=4095, window=0, sinks=0, padded=0, mix=5),
        # a ragged batch of long contexts, what four bits are for
        dict(name="q4_batch", op="attend", fmt="q4", io="bf16", batch=24, heads=32, kv_heads=32,
             head_dim=128, page=64, layers=1, longest=24001, window=0, sinks=0, padded=0, mix=6),
        # the rows of one decode step of a batch: quantized into the pool and read back
        dict(name="rows_decode", op="rows", fmt="q4", io="fp32", tokens=32, seqs=32, kv_heads=8,
             head_dim=128, page=64, layers=2, padded=1, mix=7),
        # the rows of a prefill
        dict(name="rows_prefill", op="rows", fmt="q4", io="bf16", tokens=8185, seqs=5, kv_heads=32,
             head_dim=128, page=64, layers=1, padded=0, mix=8),
        # a beam step of one layer: losers freed, winners forked into their slots, all one token on
        dict(name="beams_small", op="beams", seqs=8, forks=3, longest=300, kv_heads=2, head_dim=64,
             page=128, layers=1, window=0, sinks=0, spare=12, mix=9),
        # the same over the 16 layers of the 1B shape, with a window's pages freed
        dict(name="beams_layers", op="beams", seqs=64, forks=24, longest=1087, kv_heads=8, head_dim=64,
             page=128, layers=16, window=512, sinks=4, spare=90, mix=10),
        # a pool with holes made dense: small
        dict(name="compact_small", op="compact", seqs=8, longest=500, kv_heads=2, head_dim=64, page=128,
             layers=1, pages=48, mix=11),
        # and four layers of the 7B shape
        dict(name="compact_layers", op="compact", seqs=24, longest=1500, kv_heads=32, head_dim=128, page=64,
             layers=4, pages=512, mix=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "attend", "rows", "beams", "compact"])
    mix = rng.randrange(1 << 30)
    if op == "attend":
        hd, page = rng.choice([64, 128]), rng.choice([16, 32, 48, 64, 128])
        kvh, group = rng.choice([1, 2, 3, 4, 8, 16, 32]), rng.choice([1, 1, 2, 3, 4, 5, 8, 12])
        fmt, batch = rng.choice(["bf16", "q4"]), _log(rng, 1, 64)
        most = 1_400_000_000 // (batch * kvh * hd * (4 if fmt == "bf16" else 1))
        window = rng.choice([0, max(1, min(most, _log(rng, 1, 16384)))])
        longest = _log(rng, 1, 65536 if window else min(65536, max(1, most)))
        return dict(op=op, fmt=fmt, io=rng.choice(["fp32", "bf16"]), batch=batch,
                    heads=kvh * group, kv_heads=kvh, head_dim=hd, page=page, layers=rng.choice([1, 2]),
                    longest=longest, window=window, sinks=rng.choice([0, 1, 4, rng.randrange(1, 200)]) if window else 0,
                    padded=rng.choice([0, 0, 1, 3]) if batch > 3 else 0, mix=mix)
    if op == "rows":
        seqs = _log(rng, 1, 64)
        return dict(op=op, fmt=rng.choice(["bf16", "q4", "q4"]), io=rng.choice(["fp32", "bf16"]),
                    tokens=max(seqs, _log(rng, 1, 8000)), seqs=seqs, kv_heads=rng.choice([1, 2, 3, 8, 32]),
                    head_dim=rng.choice([64, 128]), page=rng.choice([16, 32, 48, 64, 128]),
                    layers=rng.choice([1, 2]), padded=rng.choice([0, 1, 5]), mix=mix)
    seqs = _log(rng, 4, 48)
    shape = dict(seqs=seqs, longest=_log(rng, 40, 1200), kv_heads=rng.choice([1, 2, 8]),
                 head_dim=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]), layers=rng.choice([1, 3, 8]),
                 mix=mix)
    if op == "beams":
        return dict(op=op, forks=rng.randint(1, seqs // 2), window=rng.choice([0, rng.randint(1, 600)]),
                    sinks=rng.choice([0, 4]), spare=2 * seqs + rng.randrange(8), **shape)
    most = sum(-(-n // shape["page"]) for n in lengths(shape))
    return dict(op=op, pages=most + rng.randint(1, most + 8), **shape)


def lengths(case):
    """The sequences' lengths: the longest, an empty one where there are many, others between."""
    n, rng = case.get("batch", case.get("seqs")), random.Random(case["mix"])
    longest = case["longest"]
    out = [longest] + [rng.randint(longest // 8, longest) for _ in range(n - 1)]
    if n > 3:
        out[n // 2] = 0
    return out


def visible(n, window, sinks):
    """(first rows, start of the window) that a query behind n rows sees."""
    lo = max(n - window, 0) if window else 0
    return min(sinks, lo), lo


def row_bytes(case):
    """K and V of one position of one kv head."""
    d = case["head_dim"]
    return 4 * d if case.get("fmt", "bf16") == "bf16" else d + d // 8


def token_plan(case):
    """Which sequence and position each token of a "rows" case goes to, and the sequences' lengths after it."""
    rng = random.Random(case["mix"])
    n, s = case["tokens"], case["seqs"]
    cuts = sorted(rng.randint(0, n) for _ in range(s - 1)) if n > s else list(range(1, s))
    counts = [b - a for a, b in zip([0] + cuts, cuts + [n])]
    before = [rng.randint(0, 500) for _ in range(s)]
    seq = [i for i, c in enumerate(counts) for _ in range(c)]
    pos = [before[i] + j for i, c in enumerate(counts) for j in range(c)]
    for i in range(min(case["padded"], n - 1)):
        seq[n - 1 - i] = -1
    return seq, pos, [b + c for b, c in zip(before, counts)]


def beam_plan(case):
    """(sequences freed, parents, children, sequences that go on) of a "beams" case."""
    rng = random.Random(case["mix"] + 1)
    ids = list(range(case["seqs"]))
    rng.shuffle(ids)
    freed, live = ids[:case["forks"]], ids[case["forks"]:]
    parents = [rng.choice(live) for _ in freed]
    return freed, parents, list(freed), sorted(ids)


def page_bytes(case):
    return row_bytes(case) * case["kv_heads"] * case["page"]


def work(case):
    if case["op"] == "attend":
        n_in = case["batch"] - case["padded"]
        rows = 0
        for n in lengths(case)[:n_in]:
            first, lo = visible(n, case["window"], case["sinks"])
            rows += first + n - lo
        io = (4 if case["io"] == "fp32" else 2) * 2 * n_in * case["heads"] * case["head_dim"]
        return {"bytes": rows * case["kv_heads"] * row_bytes(case) + io,
                "flops": 4 * rows * case["heads"] * case["head_dim"]}
    if case["op"] == "rows":
        n = case["tokens"] - min(case["padded"], case["tokens"] - 1)
        values = 2 * n * case["kv_heads"] * case["head_dim"]
        return {"bytes": 2 * values * (4 if case["io"] == "fp32" else 2) + 2 * n * case["kv_heads"] * row_bytes(case),
                "flops": 2 * values}
    tables = 4 * case["seqs"] * (case["longest"] // case["page"] + 3)
    if case["op"] == "beams":
        _, parents, _, _ = beam_plan(case)
        n = lengths(case)
        moved = sum(1 for p in parents if n[p] % case["page"])
    else:
        taken = _taken(case, case["mix"])
        moved = int((taken >= len(taken)).sum())
    return {"bytes": 2 * moved * page_bytes(case) * case["layers"] + tables, "flops": 0}


def _taken(case, mix):
    """The pages that a "compact" case's sequences hold, in table order."""
    used = sum(-(-n // case["page"]) for n in lengths(case))
    return np.random.RandomState(mix % (1 << 31)).permutation(case["pages"])[:used]


# ---- inputs ---------------------------------------------------------------------

def _pool(case, pages, gen):
    """A pool of random rows."""
    L, pb = case["layers"], page_bytes(case)
    if case.get("fmt", "bf16") == "bf16":
        rows = torch.randn(L * pages * pb // 2, device="cuda", dtype=torch.bfloat16, generator=gen)
        return rows.view(torch.uint8).view(L, pages, pb)
    pool = torch.randint(0, 256, (L, pages, pb), device="cuda", dtype=torch.uint8, generator=gen)
    _, scales = _q4_parts(pool, case)
    scales.copy_(torch.rand(scales.shape, device="cuda", generator=gen).mul_(0.2).add_(0.1))
    return pool


def _tables(case, lens, pages, order, width, window=0, sinks=0):
    """The table of sequences of these lengths, pages taken from `order`; a page that the window
    no longer sees has none."""
    R = case["page"]
    table = np.full((len(lens), width), -1, np.int32)
    at = 0
    for s, n in enumerate(lens):
        first, lo = visible(n, window, sinks)
        for i in range(-(-n // R)):
            if i * R < first or (i + 1) * R > lo:
                table[s, i] = order[at]
                at += 1
    assert at <= pages
    return table


def _int(a):
    return torch.tensor(np.asarray(a, np.int32), device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.RandomState(seed % (1 << 31))
    R, st = case["page"], {"case": dict(case)}
    io = torch.float32 if case.get("io") == "fp32" else torch.bfloat16
    if case["op"] == "attend":
        lens = lengths(case)
        width = max(1, -(-case["longest"] // R))
        pages = 1 + sum(1 for s, n in enumerate(lens) for i in range(-(-n // R))
                        if i * R < visible(n, case["window"], case["sinks"])[0]
                        or (i + 1) * R > visible(n, case["window"], case["sinks"])[1])
        table = _tables(case, lens, pages, rng.permutation(pages), width, case["window"], case["sinks"])
        seqs = [s if s < case["batch"] - case["padded"] else -1 for s in range(case["batch"])]
        shape = (case["batch"], case["heads"], case["head_dim"])
        first = [visible(n, case["window"], case["sinks"]) for n in lens]
        st.update(pool=_pool(case, pages, gen), seqs=_int(seqs),
                  q=torch.randn(shape, device="cuda", generator=gen).to(io),
                  out=torch.zeros(shape, device="cuda", dtype=io),
                  span=max(1, max(a + n - lo for n, (a, lo) in zip(lens, first))))
    elif case["op"] == "rows":
        seq, pos, lens = token_plan(case)
        used = sum(-(-n // R) for n in lens)
        pages, width = used + 1, max(1, max(-(-n // R) for n in lens))
        table = _tables(case, lens, pages, rng.permutation(pages), width)
        shape = (case["tokens"], case["kv_heads"], case["head_dim"])
        # keys and values as they come: a few dimensions much larger than the rest
        big = 1 + 7 * (torch.rand(case["head_dim"], device="cuda", generator=gen) < 0.05)
        k, v = (torch.randn(shape, device="cuda", generator=gen) for _ in range(2))
        st.update(pool=_pool(case, pages, gen), seqs=_int(seq), positions=_int(pos), k=(k * big).to(io), v=v.to(io),
                  k_out=torch.zeros(shape, device="cuda", dtype=io), v_out=torch.zeros(shape, device="cuda", dtype=io))
    else:
        lens = lengths(case)
        width = -(-(case["longest"] + 1) // R) + 1
        if case["op"] == "beams":
            pages = sum(-(-n // R) for n in lens) + case["spare"]
            order = rng.permutation(pages)
            freed, parents, children, ahead = beam_plan(case)
            st.update(freed=_int(freed), parents=_int(parents), children=_int(children), ahead=_int(ahead))
        else:
            pages, order = case["pages"], _taken(case, case["mix"])
        table = _tables(case, lens, pages, order, width)
        st.update(pool=_pool(case, pages, gen))
    refs = np.zeros(pages, np.int32)
    np.add.at(refs, table[table >= 0], 1)
    st.update(table=_int(table), lens=_int(lens), refs=_int(refs))
    if case["op"] in ("beams", "compact"):
        st.update(table0=st["table"].clone(), lens0=st["lens"].clone(), refs0=st["refs"].clone())
    return st


# ---- one pass -------------------------------------------------------------------

def run(st):
    case = st["case"]
    if case["op"] in ("beams", "compact"):  # the same tables before every pass
        st["table"].copy_(st["table0"])
        st["lens"].copy_(st["lens0"])
        st["refs"].copy_(st["refs0"])
    if own:
        return _run_own(st)
    return {"attend": _attend, "rows": _rows, "beams": _beams, "compact": _compact}[case["op"]](st)


def _cache(st):
    """The library's view of the state's tensors: made once, as a serving program keeps it."""
    if "cache" not in st:
        from transformer_layer_decode_gb300 import kv
        c = st["case"]
        st["cache"] = kv.KVCache(n_layers=c["layers"], n_kv_heads=c["kv_heads"], head_dim=c["head_dim"],
                                 page_rows=c["page"], fmt=c.get("fmt", "bf16"), pool=st["pool"],
                                 table=st["table"], lens=st["lens"], refs=st["refs"])
    return st["cache"]


def _run_own(st):
    case, cache = st["case"], _cache(st)
    layer = case["layers"] - 1
    if case["op"] == "attend":
        return cache.attention(layer, st["q"], seqs=st["seqs"], window=case["window"], sinks=case["sinks"],
                               out=st["out"])
    if case["op"] == "rows":
        cache.append(layer, st["k"], st["v"], seqs=st["seqs"], positions=st["positions"])
        return cache.read(layer, st["seqs"], st["positions"], k_out=st["k_out"], v_out=st["v_out"])
    if case["op"] == "beams":
        cache.release(st["freed"])
        cache.fork(st["parents"], st["children"])
        cache.extend(st["ahead"])
        if case["window"]:
            cache.release(st["ahead"], window=case["window"], sinks=case["sinks"])
        return st["table"], st["lens"], st["refs"], st["pool"].view(torch.bfloat16)
    cache.compact()
    return st["table"], st["refs"], st["pool"].view(torch.bfloat16)


def _bf16_rows(pool, case):
    """[layers][pages][K, V][kv head][position][dim]"""
    L, pages, _ = pool.shape
    return pool.view(torch.bfloat16).view(L, pages, 2, case["kv_heads"], case["page"], case["head_dim"])


def _q4_parts(pool, case):
    """codes [layers][pages][K, V][kv head][position][bytes], scales [...][blocks] (fp16)"""
    L, pages, _ = pool.shape
    R, d = case["page"], case["head_dim"]
    heads = pool.view(L, pages, 2, case["kv_heads"], R * (d // 2 + d // 16))
    codes = heads[..., :R * d // 2].unflatten(-1, (R, d // 2))
    scales = heads[..., R * d // 2:].view(torch.float16).unflatten(-1, (R, d // 32))
    return codes, scales


def _gather(pool, case, which, page, row):
    """Rows of K (0) or V (1) as fp32 [..., kv head, dim]: the last layer's, by page and row of the page."""
    layer, d = case["layers"] - 1, case["head_dim"]
    if case.get("fmt", "bf16") == "bf16":
        return _bf16_rows(pool, case)[layer, :, which][page, :, row].float()
    codes, scales = _q4_parts(pool, case)
    b = codes[layer, :, which][page, :, row]
    s = scales[layer, :, which][page, :, row]
    n = torch.stack((b & 15, b >> 4), -1).flatten(-2)
    n = n.unflatten(-1, (8, d // 32, 4)).transpose(-3, -2).flatten(-2)
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
    k = _gather(st["pool"], case, 0, page, pos % R)
    s = torch.matmul(q, k.permute(0, 2, 3, 1)) / math.sqrt(case["head_dim"])
    del k
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    w = torch.exp(s - torch.where(top == -math.inf, 0, top))
    v = _gather(st["pool"], case, 1, page, pos % R)
    o = torch.matmul(w, v.permute(0, 2, 1, 3))
    total = w.sum(-1, keepdim=True)
    return torch.where(total > 0, o / total, 0).flatten(1, 2).to(st["out"].dtype)


def _rows(st):
    case = st["case"]
    layer, R, d = case["layers"] - 1, case["page"], case["head_dim"]
    real = st["seqs"] >= 0
    seq, pos = st["seqs"][real].long(), st["positions"][real].long()
    page, row = st["table"][seq, pos // R].long(), pos % R
    out = []
    for which, x, to in ((0, st["k"], st["k_out"]), (1, st["v"], st["v_out"])):
        x = x[real]
        if case["fmt"] == "bf16":
            _bf16_rows(st["pool"], case)[layer, :, which][page, :, row] = x.to(torch.bfloat16)
        else:
            x = x.float().unflatten(-1, (d // 32, 32))
            s = (x.abs().amax(-1) / 7).clamp(max=65504).half()
            step = s.double()[..., None]  # in 64 bits: a quotient next to a half
            n = torch.where(step > 0, x.double() / step, 0).round().clamp(-8, 7).int() + 8
            n = n.unflatten(-1, (8, 4)).transpose(-3, -2).flatten(-3)
            codes, scales = _q4_parts(st["pool"], case)
            codes[layer, :, which][page, :, row] = (n[..., 0::2] | (n[..., 1::2] << 4)).to(torch.uint8)
            scales[layer, :, which][page, :, row] = s
        back = torch.zeros_like(to)
        back[real] = _gather(st["pool"], case, which, page, row).to(to.dtype)
        out.append(back)
    return tuple(out)


def _free(refs):
    """Free pages, lowest first (then the others)."""
    return torch.sort((refs != 0).int(), stable=True).indices


def _count(refs, pages, by):
    """refs += by for each page named (a negative entry names none)."""
    pages = pages.flatten().long()
    refs.index_add_(0, pages.clamp(min=0), torch.where(pages >= 0, by, 0).int())


def _release(table, lens, refs, seqs):
    _count(refs, table[seqs], -1)
    table[seqs] = -1
    lens[seqs] = 0


def _beams(st):
    case, table, lens, refs, pool = st["case"], st["table"], st["lens"], st["refs"], st["pool"]
    R = case["page"]
    _release(table, lens, refs, st["freed"].long())
    # fork: full pages are shared, a partial last page is copied into a free one
    par, child = st["parents"].long(), st["children"].long()
    n = lens[par].long()
    part = n % R != 0
    new = _free(refs)[(part.cumsum(0) - 1).clamp(min=0)]
    rows, tail = table[par], (n // R)
    old = rows.gather(1, tail[:, None])[:, 0].long()
    keep = rows.gather(1, tail[:, None])
    rows.scatter_(1, tail[:, None], torch.where(part[:, None], -1, keep))
    _count(refs, rows, 1)
    rows.scatter_(1, tail[:, None], torch.where(part[:, None], new[:, None].int(), keep))
    table[child] = rows
    lens[child] = n.int()
    refs[new[part]] = 1
    pool[:, new[part]] = pool[:, old[part]]
    # one token on: a new page where the last one is full
    seq = st["ahead"].long()
    n = lens[seq].long()
    full = n % R == 0
    new = _free(refs)[(full.cumsum(0) - 1).clamp(min=0)]
    at = (n // R)[:, None]
    table[seq] = table[seq].scatter(1, at, torch.where(full[:, None], new[:, None].int(), table[seq].gather(1, at)))
    refs[new[full]] = 1
    lens[seq] = (n + 1).int()
    if case["window"]:  # pages between the first rows and the window are freed
        i = torch.arange(table.shape[1], device=table.device)[None] * R
        lo = (lens[seq].long() - case["window"])[:, None]
        gone = (i >= case["sinks"]) & (i + R <= lo)
        _count(refs, torch.where(gone, table[seq], -1), -1)
        table[seq] = torch.where(gone, -1, table[seq])
    return table, lens, refs, pool.view(torch.bfloat16)


def _compact(st):
    table, refs, pool = st["table"], st["refs"], st["pool"]
    i = torch.arange(refs.numel(), device=refs.device)
    live = refs > 0
    count = live.sum()
    to, of = i[~live & (i < count)], i[live & (i >= count)]
    pool[:, to] = pool[:, of]
    refs[to] = refs[of]
    refs[of] = 0
    name = i.int()
    name[of] = to.int()
    table.copy_(torch.where(table >= 0, name[table.long().clamp(min=0)], -1))
    return table, refs, pool.view(torch.bfloat16)


# ---- the definition in 64 bits ----------------------------------------------------

def _exact_pages(raw, case):
    """fp64 [page][K, V][kv head][position][dim] of whole pages (uint8 [m][page_bytes])."""
    R, d, kvh = case["page"], case["head_dim"], case["kv_heads"]
    if case["fmt"] == "bf16":
        return raw.view(torch.bfloat16).view(-1, 2, kvh, R, d).double()
    heads = raw.view(-1, 2, kvh, R * (d // 2 + d // 16))
    codes = heads[..., :R * d // 2].reshape(-1, 2, kvh, R, d // 2)
    scales = heads[..., R * d // 2:].contiguous().view(torch.float16).view(-1, 2, kvh, R, d // 32)
    e = torch.arange(d, device=raw.device)
    block, g, i = e // 32, e % 32 // 4, e % 4
    nibble = (g * (d // 32) + block) * 4 + i
    code = (codes[..., nibble // 2] >> (4 * (nibble % 2)).to(torch.uint8)) & 15
    return (code.double() - 8) * scales[..., block].double()


def exact(case, seed):
    st = prepare(case, seed)
    R, table, lens = case["page"], st["table"].cpu().numpy(), st["lens"].cpu().numpy()
    if case["op"] == "attend":
        d, kvh, heads = case["head_dim"], case["kv_heads"], case["heads"]
        out = torch.zeros(case["batch"], heads, d, dtype=torch.float64, device="cuda")
        for b in range(case["batch"] - case["padded"]):
            n = int(lens[b])
            pos = np.array([p for p in range(n) if not case["window"] or p >= n - case["window"] or p < case["sinks"]],
                           np.int64)
            if not len(pos):
                continue
            pages, which = np.unique(table[b][pos // R], return_inverse=True)
            raw = st["pool"][case["layers"] - 1][torch.tensor(pages, device="cuda").long()]
            at, row = torch.tensor(which.reshape(-1), device="cuda"), torch.tensor(pos % R, device="cuda")
            values = _exact_pages(raw, case)
            for h in range(kvh):
                group = slice(h * heads // kvh, (h + 1) * heads // kvh)
                s = values[:, 0, h][at, row] @ st["q"][b, group].double().T / math.sqrt(d)
                out[b, group] = torch.softmax(s, 0).T @ values[:, 1, h][at, row]
        return out
    if case["op"] == "rows":
        outs = []
        for x in (st["k"], st["v"]):
            if case["fmt"] == "bf16":
                y = x.to(torch.bfloat16).cpu().double().numpy()
            else:
                a = x.float().cpu().numpy().reshape(case["tokens"], case["kv_heads"], -1, 32)
                s = np.minimum(np.abs(a).max(-1, keepdims=True) / np.float32(7), np.float32(65504))
                s = s.astype(np.float16).astype(np.float64)
                with np.errstate(divide="ignore", invalid="ignore"):
                    c = np.where(s > 0, np.clip(np.rint(a.astype(np.float64) / s), -8, 7), 0)
                y = (c * s).reshape(x.shape)
            y[st["seqs"].cpu().numpy() < 0] = 0
            outs.append(torch.from_numpy(y))
        return tuple(outs)
    refs, pool = st["refs"].cpu().numpy(), st["pool"]
    if case["op"] == "beams":
        freed, parents, children, ahead = beam_plan(case)
        for s in freed:
            for i, p in enumerate(table[s]):
                if p >= 0:
                    refs[p] -= 1
                    table[s, i] = -1
            lens[s] = 0
        moves = []
        for a, b in zip(parents, children):
            lens[b] = lens[a]
            for i, p in enumerate(table[a].copy()):
                if p >= 0 and i == lens[a] // R and lens[a] % R:
                    moves.append((p, int(np.flatnonzero(refs == 0)[0])))
                    p = moves[-1][1]
                table[b, i] = p
                if p >= 0:
                    refs[p] += 1
        for a in ahead:
            if lens[a] % R == 0:
                table[a, lens[a] // R] = np.flatnonzero(refs == 0)[0]
                refs[table[a, lens[a] // R]] = 1
            lens[a] += 1
        for a in ahead if case["window"] else []:
            for i, p in enumerate(table[a]):
                if p >= 0 and i * R >= case["sinks"] and (i + 1) * R <= lens[a] - case["window"]:
                    refs[p] -= 1
                    table[a, i] = -1
        for src, dst in moves:
            pool[:, dst] = pool[:, int(src)]
        ints = [table, lens, refs]
    else:
        count, holes = int((refs > 0).sum()), [p for p in range(len(refs)) if refs[p] == 0]
        for src in range(count, len(refs)):
            if refs[src]:
                dst = holes.pop(0)
                pool[:, dst] = pool[:, src]
                table[table == src] = dst
                refs[dst], refs[src] = refs[src], 0
        ints = [table, refs]
    return tuple(torch.from_numpy(x) for x in ints) + (pool.view(torch.bfloat16).double(),)
