"""What the paged draft cache's operators are measured on: cases, inputs, a plain form in
elementary torch operations, and the definition in 64 bits.

Three groups of calls of `block_diffusion_speculative_03_b200.paging.PagePool`:
  pages   handing pages of a key/value cache out, sharing, copying, moving and freeing them;
  decode  attention of one new token per sequence over its pages;
  window  the same attention for one token, a draft block or a prompt chunk, with a sliding
          window and a few first positions that stay visible.

A pool holds [page][layer][K, V][kv head][position in page][head_dim]; a sequence owns the
positions [0, len) through a table of page ids, and a call's new rows sit at [len, len + rows).
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    # Cache sizes follow the drafter shapes of this repository: 5 layers of 8 key/value heads of
    # 128 (32 query heads), 4 key/value heads for the coder-shaped one, 2 layers of 64 in fp32
    # for the smallest.
    return [
        # one cycle of a small beam: every request forked once, room for a block of 16 made for
        # all (the half-filled last pages are copied); the launches count, not the bytes
        dict(name="beam_step", op="beam", dtype="bf16", layers=5, nkv=8, d=128, page=16, seqs=4, width=1,
             lo=100, hi=2100, grow=16, salt=1),
        # two long contexts copied whole, as when a sequence leaves for a place of its own
        dict(name="clone_long", op="clone", dtype="bf16", layers=5, nkv=8, d=128, page=64, seqs=2, width=1,
             lo=16384, hi=16384, grow=0, salt=2),
        # a pool that a day's requests have riddled with holes, pushed together
        dict(name="compact_pool", op="compact", dtype="bf16", layers=5, nkv=8, d=128, page=32, seqs=32, width=1,
             lo=512, hi=4096, grow=0, salt=3),
        # a batch in turnover on the fp32 drafter: some requests end, some are cut back, the rest
        # get room for their next rows, and the rows are written
        dict(name="turnover_f32", op="turnover", dtype="f32", layers=2, nkv=2, d=64, page=16, seqs=24, width=1,
             lo=3, hi=1500, grow=7, salt=4),
        # the headline drafter's context, one token: latency
        dict(name="decode_b1", op="decode", dtype="bf16", layers=5, nq=32, nkv=8, d=128, page=64, seqs=1,
             lo=2048, hi=2048, rows=1, ragged=False, causal=True, window=0, sinks=0, salt=5),
        # long thinking contexts: bandwidth
        dict(name="decode_long", op="decode", dtype="bf16", layers=2, nq=32, nkv=8, d=128, page=64, seqs=4,
             lo=32768, hi=32768, rows=1, ragged=False, causal=True, window=0, sinks=0, salt=6),
        # a serving batch of 32 of very different lengths, small pages, 8 query heads to a kv head
        dict(name="decode_ragged", op="decode", dtype="bf16", layers=2, nq=32, nkv=4, d=128, page=16, seqs=32,
             lo=1, hi=8191, rows=1, ragged=False, causal=True, window=0, sinks=0, salt=7),
        # fp32 storage, odd lengths
        dict(name="decode_f32", op="decode", dtype="f32", layers=2, nq=4, nkv=2, d=64, page=16, seqs=5,
             lo=33, hi=3001, rows=1, ragged=False, causal=True, window=0, sinks=0, salt=8),
        # one token of a long context that sees its last 1024 positions and the first 4
        dict(name="window_token", op="window", dtype="bf16", layers=2, nq=32, nkv=8, d=128, page=64, seqs=16,
             lo=8192, hi=32768, rows=1, ragged=False, causal=True, window=1024, sinks=4, salt=9),
        # a draft block of 16 whose positions see one another, over a long context's last 4096
        dict(name="window_block", op="window", dtype="bf16", layers=2, nq=32, nkv=8, d=128, page=64, seqs=4,
             lo=32768, hi=32768, rows=16, ragged=False, causal=False, window=4096, sinks=16, salt=10),
        # a prompt chunk of 2048 rows behind 6000 positions, causal
        dict(name="window_prompt", op="window", dtype="bf16", layers=2, nq=32, nkv=8, d=128, page=64, seqs=1,
             lo=6000, hi=6000, rows=2048, ragged=False, causal=True, window=2048, sinks=4, salt=11),
        # prompts and tokens of different lengths in one call, heads of 64, 3 query heads to a kv head
        dict(name="window_mixed", op="window", dtype="bf16", layers=2, nq=6, nkv=2, d=64, page=32, seqs=9,
             lo=1, hi=5000, rows=700, ragged=True, causal=True, window=333, sinks=5, salt=12),
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["beam", "clone", "compact", "turnover", "decode", "decode", "window", "window", "window"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = rng.choice([64, 128])
    nkv = rng.choice([1, 2, 3, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    salt = rng.randrange(1 << 30)
    if op in ("beam", "clone", "compact", "turnover"):
        layers = rng.choice([1, 2, 5, 8])
        seqs = log(1, 32)
        width = rng.choice([1, 1, 2, 3]) if op == "beam" else 1
        per = layers * 2 * nkv * d * (2 if dtype == "bf16" else 4)      # bytes of a position
        most = max(64, min(16384, (400 << 20) // (per * seqs)))
        hi = log(64, most)
        return dict(op=op, dtype=dtype, layers=layers, nkv=nkv, d=d, page=page, seqs=seqs, width=width,
                    lo=log(1, hi), hi=hi, grow=log(1, 100), salt=salt)
    group = rng.choice([1, 2, 3, 4, 8] if dtype == "bf16" else [1, 2, 4])
    seqs = log(1, 64)
    rows = 1 if op == "decode" else rng.choice([1, log(2, 32), log(2, 32), log(33, 1500)])
    if rows > 32:
        seqs = min(seqs, 6)
    # keys per sequence: the cost stays below the listed decode_long and window_prompt, and the
    # plain form's score matrix below 2^29 values
    most = min(32768, (120 << 20) // (seqs * nkv * d), (1 << 29) // (seqs * rows * nkv * group))
    if dtype == "f32":
        most = min(most, 8192 if rows == 1 else 1500)
    hi = log(16, max(17, most))
    causal = True if op == "decode" else rng.choice([True, True, False])
    window = 0 if op == "decode" else rng.choice([0, log(1, 64), log(64, 8192), log(64, 8192)])
    return dict(op=op, dtype=dtype, layers=rng.choice([1, 2]), nq=nkv * group, nkv=nkv, d=d, page=page, seqs=seqs,
                lo=log(1, hi), hi=hi, rows=rows, ragged=rows > 1 and rng.random() < 0.5, causal=causal, window=window,
                sinks=rng.choice([0, 1, 4, 70]) if window else 0, salt=salt)


def _spread(case, n, lo, hi, salt):
    """n whole numbers in [lo, hi], spread over their logarithm; fixed by the case."""
    r = random.Random(case["salt"] * 1000003 + salt)
    return [lo if lo == hi else max(lo, min(hi, int(round(math.exp(r.uniform(math.log(lo), math.log(hi)))))))
            for _ in range(n)]


def _shape(case):
    """Lengths, rows and table sizes of a case, the same for every seed."""
    n, page = case["seqs"], case["page"]
    lens = _spread(case, n, case["lo"], case["hi"], 1)
    if case["op"] in ("decode", "window"):
        rows = _spread(case, n, 1, case["rows"], 2) if case["ragged"] else [case["rows"]] * n
        total, grow = n, 0
    else:
        rows = [0] * n
        total, grow = n * (1 + case["width"]), case["grow"]
    need = [-(-(a + b) // page) for a, b in zip(lens, rows)]
    cap = max(a + b for a, b in zip(lens, rows)) + grow + 1
    cols = -(-cap // page)
    used = sum(need)
    grown = sum(-(-(a + grow) // page) + 1 for a in lens)
    pages = {"decode": used, "window": used, "beam": used + (1 + case.get("width", 1)) * grown,
             "clone": 2 * used, "compact": 2 * used, "turnover": used + grown}[case["op"]]
    return dict(lens=lens, rows=rows, need=need, max_len=cap, cols=cols, total=total, used=used, pages=pages + 3)


def _turnover(case, lens):
    """Which sequences end, which are cut back and to what, and which go on."""
    n = len(lens)
    ended = [i for i in range(n) if i % 4 == 3]
    cut = [i for i in range(n) if i % 4 == 1]
    keep = [lens[i] * 2 // 3 for i in cut]
    on = [i for i in range(n) if i % 4 != 3]
    rows = [1 + (5 * j + case["salt"]) % case["grow"] for j in range(len(on))]
    return ended, cut, keep, on, rows


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    s = _shape(case)
    dt = DTYPES[case["dtype"]]
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    layers, nkv, d, page = case["layers"], case["nkv"], case["d"], case["page"]

    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    # Page ids in no order. compact: half of the pages in use lie above the number in use.
    ids = torch.randperm(s["pages"], device=dev, generator=g)[:s["used"]]
    if case["op"] == "compact":
        low = torch.randperm(s["used"], device=dev, generator=g)[:s["used"] - s["used"] // 2]
        high = s["used"] + torch.randperm(s["pages"] - s["used"], device=dev, generator=g)[:s["used"] // 2]
        ids = torch.cat([low, high])[torch.randperm(s["used"], device=dev, generator=g)]
    ids = ids.to(torch.int32)
    table = torch.full((s["total"], s["cols"]), -1, dtype=torch.int32, device=dev)
    at = 0
    for i, n in enumerate(s["need"]):
        table[i, :n] = ids[at:at + n]
        at += n
    lens = i32(s["lens"] + [0] * (s["total"] - len(s["lens"])))

    st = dict(case=case, shape=s, page=page, n_pages=s["pages"], table0=table, len0=lens, dtype=dt)
    n, w = case["seqs"], case.get("width", 1)
    if case["op"] in ("beam", "clone"):
        st["src"] = i32([i for _ in range(w) for i in range(n)])
        st["dst"] = i32(list(range(n, n + n * w)))
        st["all"] = i32(list(range(n + n * w)))
        st["grow"] = i32([case["grow"]] * (n + n * w))
    if case["op"] == "turnover":
        ended, cut, keep, on, rows = _turnover(case, s["lens"])
        start = [sum(rows[:j]) for j in range(len(rows))]
        st.update(ended=i32(ended), cut=i32(cut), keep=i32(keep), on=i32(on), count=i32(rows), start=i32(start),
                  most=max(rows), which=i32([j for j, r in enumerate(rows) for _ in range(r)]),
                  place=i32([k for r in rows for k in range(r)]))
        st["k"], st["v"] = (torch.randn(sum(rows), nkv, d, device=dev, generator=g).to(dt) for _ in range(2))
    if case["op"] in ("decode", "window"):
        rows = s["rows"]
        start = [sum(rows[:j]) for j in range(len(rows))]
        st.update(count=i32(rows), start=i32(start), most=max(rows), n_max=max(a + b for a, b in zip(s["lens"], rows)),
                  which=torch.tensor([j for j, r in enumerate(rows) for _ in range(r)], device=dev),
                  place=torch.tensor([k for r in rows for k in range(r)], device=dev))
        st["q"] = (torch.randn(sum(rows), case["nq"], d, device=dev, generator=g) * 1.3).to(dt)

    if own:
        from block_diffusion_speculative_03_b200.paging import PagePool
        pool = PagePool(layers, case.get("nq", nkv), nkv, d, case["dtype"], n_pages=s["pages"], page_size=page,
                        max_seqs=s["total"], max_len=s["max_len"])
        slab = pool.slab()
        st["pool"] = pool
    else:
        slab = torch.empty(s["pages"], layers, 2, nkv, page, d, dtype=dt, device=dev)
    # keys and values of the spread that the drafter's projections give them
    for p in range(0, s["pages"], 256):
        part = slab[p:p + 256]
        part.copy_(torch.randn(part.shape, device=dev, generator=g) * 1.28)
    st["slab"] = slab
    if own and case["op"] in ("decode", "window"):
        pool.set_tables(lens, table)
    return st


def _bits(slab):
    """Copied values, to be compared as they are."""
    return slab.view(torch.int16 if slab.dtype == torch.bfloat16 else torch.int32)


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if op in ("decode", "window"):
        return _own_attention(state) if own else _attention(state)
    return _own_pages(state) if own else _pages(state)


def _own_attention(st):
    c, pool = st["case"], st["pool"]
    if c["rows"] == 1:
        return pool.attention(c["layers"] - 1, st["q"], causal=c["causal"], window=c["window"], sinks=c["sinks"])
    return pool.attention(c["layers"] - 1, st["q"], row_start=st["start"], row_count=st["count"], max_rows=st["most"],
                          causal=c["causal"], window=c["window"], sinks=c["sinks"])


def _own_pages(st):
    c, pool = st["case"], st["pool"]
    pool.set_tables(st["len0"], st["table0"])
    out = {}
    if c["op"] == "beam":
        pool.fork(st["src"], st["dst"])
        pool.reserve(st["grow"], st["all"])
    elif c["op"] == "clone":
        pool.fork(st["src"], st["dst"], deep=True)
    elif c["op"] == "compact":
        out["used"] = pool.compact()
    else:
        pool.free(st["ended"])
        pool.free(st["cut"], keep=st["keep"])
        pool.reserve(st["count"], st["on"])
        pool.write(c["layers"] - 1, st["k"], st["v"], st["on"], st["start"], st["count"], max_rows=st["most"])
        pool.advance(st["count"], st["on"])
    return dict(out, table=pool.table, len=pool.len, refs=pool.refs, slab=_bits(st["slab"]))


# -- plain form -----------------------------------------------------------------

def _attention(st):
    """Every sequence padded to the longest: gather the keys in reach, scores, masked softmax, values."""
    c, page = st["case"], st["page"]
    dev = st["q"].device
    nkv, d, layer = c["nkv"], c["d"], c["layers"] - 1
    b, most = c["seqs"], st["most"]
    length, count = st["len0"].long(), st["count"].long()
    row = torch.arange(most, device=dev)
    pos = length[:, None] + row
    last = torch.where(row < count[:, None], pos, 0) if c["causal"] else (length + count - 1)[:, None].expand(b, most)
    # the positions that some row may see: all, or the first few and those from the first row's window on
    n = st["n_max"]
    key = torch.arange(n, device=dev).expand(b, n)
    if c["window"] and c["sinks"] + c["window"] + most - 1 < n:
        n = c["sinks"] + c["window"] + most - 1
        low = (length - c["window"] + 1).clamp(min=c["sinks"])
        key = torch.arange(n, device=dev)
        key = torch.where(key < c["sinks"], key, low[:, None] + key - c["sinks"])                   # [b, n]
    at = st["table0"].gather(1, (key // page).clamp(max=st["table0"].shape[1] - 1)).long().clamp(min=0)
    k = st["slab"][at, layer, 0, :, key % page].float().permute(0, 2, 3, 1)      # [b, nkv, d, n]
    v = st["slab"][at, layer, 1, :, key % page].float().permute(0, 2, 1, 3)      # [b, nkv, n, d]
    take = (st["start"].long()[:, None] + row).clamp(max=st["q"].shape[0] - 1)   # [b, most]
    q = st["q"][take].float().view(b, most, nkv, -1, d).permute(0, 2, 3, 1, 4)   # [b, nkv, group, most, d]
    seen = key[:, None] <= last[:, :, None]
    if c["window"]:
        seen = seen & ((key[:, None] < c["sinks"]) | (key[:, None] > pos[:, :, None] - c["window"]))
    s = torch.matmul(q.reshape(b, nkv, -1, d), k).view(b, nkv, -1, most, n) * (1.0 / math.sqrt(d))
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-1e30))
    o = torch.matmul(p.reshape(b, nkv, -1, n), v) / p.sum(-1).reshape(b, nkv, -1, 1)
    o = o.view(b, nkv, -1, most, d).permute(0, 3, 1, 2, 4).reshape(b, most, -1, d)
    return o[st["which"], st["place"]].to(st["dtype"])


def _refs(table, n_pages):
    flat = torch.where(table < 0, n_pages, table).flatten().long()
    return torch.zeros(n_pages + 1, dtype=torch.int32, device=table.device).index_add_(
        0, flat, torch.ones_like(flat, dtype=torch.int32))[:n_pages]


def _reserve(st, table, length, seqs, grow):
    """Pages for `grow` more positions of each sequence; a page that another still holds is copied."""
    page, slab = st["page"], st["slab"]
    refs = _refs(table, st["n_pages"])
    t, ln = table[seqs], length[seqs].long()
    col = torch.arange(table.shape[1], device=table.device)
    first, past = ln // page, (ln + grow + page - 1) // page
    here = (col >= first[:, None]) & (col < past[:, None]) & (grow > 0)[:, None]
    held = here & (t >= 0)
    same = (t[:, None] == t[None]) & held[:, None] & held[None]                  # [i, earlier j, column]
    earlier = torch.tril(torch.ones(len(seqs), len(seqs), dtype=torch.bool, device=table.device), -1)
    before = (same & earlier[:, :, None]).sum(1)
    new = here & ((t < 0) | (refs[t.clamp(min=0).long()] - before > 1))
    free = torch.argsort((refs > 0).int(), stable=True)
    rank = (new.flatten().cumsum(0) - 1).clamp(min=0).view_as(new)
    t2 = torch.where(new, free[rank].int(), t)
    table[seqs] = t2
    spot = first.clamp(max=table.shape[1] - 1)[:, None]
    old, now = t.gather(1, spot)[:, 0].long(), t2.gather(1, spot)[:, 0].long()
    move = (new.gather(1, spot)[:, 0] & (old >= 0) & (ln % page > 0)).nonzero()[:, 0]
    keep = torch.arange(page, device=table.device)[None] < (ln % page)[move][:, None]
    slab[now[move]] = torch.where(keep[:, None, None, None, :, None], slab[old[move]], slab[now[move]])


def _pages(st):
    c, page, slab, n_pages = st["case"], st["page"], st["slab"], st["n_pages"]
    table, length = st["table0"].clone(), st["len0"].clone()
    col = torch.arange(table.shape[1], device=table.device)
    out = {}
    if c["op"] in ("beam", "clone"):
        src, dst = st["src"].long(), st["dst"].long()
        within = col < ((length[src] + page - 1) // page)[:, None]
        length[dst] = length[src]
        if c["op"] == "beam":
            table[dst] = torch.where(within, table[src], -1)
            _reserve(st, table, length, st["all"].long(), st["grow"].long())
        else:
            free = torch.argsort((_refs(table, n_pages) > 0).int(), stable=True)
            rank = (within.flatten().cumsum(0) - 1).clamp(min=0).view_as(within)
            table[dst] = torch.where(within, free[rank].int(), -1)
            slab[table[dst][within].long()] = slab[table[src][within].long()]
    elif c["op"] == "compact":
        used = _refs(table, n_pages) > 0
        out["used"] = used.sum(dtype=torch.int32).view(1)
        ids = torch.arange(n_pages, device=table.device)
        to = (~used & (ids < out["used"])).nonzero()[:, 0]
        of = (used & (ids >= out["used"])).nonzero()[:, 0]
        slab[to] = slab[of]
        ids[of] = to
        table = torch.where(table < 0, table, ids[table.clamp(min=0).long()].int())
    else:
        table[st["ended"].long()] = -1
        length[st["ended"].long()] = 0
        cut, keep = st["cut"].long(), st["keep"]
        table[cut] = torch.where(col < ((keep + page - 1) // page)[:, None], table[cut], -1)
        length[cut] = keep
        on, count = st["on"].long(), st["count"]
        _reserve(st, table, length, on, count.long())
        seq = on[st["which"].long()]
        pos = length[seq].long() + st["place"]
        at = table[seq, pos // page].long()
        slab[at, c["layers"] - 1, 0, :, pos % page] = st["k"]
        slab[at, c["layers"] - 1, 1, :, pos % page] = st["v"]
        length[on] += count
    return dict(out, table=table, len=length, refs=_refs(table, n_pages), slab=_bits(slab))


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    """Attention sequence by sequence and head by head in 64 bits; whole-number outputs have none."""
    if case["op"] not in ("decode", "window"):
        return None
    st = prepare(case, seed)
    s, page, layer = st["shape"], case["page"], case["layers"] - 1
    slab = st["slab"]
    group = case["nq"] // case["nkv"]
    out = torch.empty(st["q"].shape, dtype=torch.float64, device=st["q"].device)
    first = 0
    for b in range(case["seqs"]):
        ln, rows = s["lens"][b], s["rows"][b]
        n = ln + rows
        pages = st["table0"][b, :-(-n // page)].long()
        kv = slab[pages, layer].permute(1, 2, 0, 3, 4).reshape(2, case["nkv"], -1, case["d"])[:, :, :n].double()
        for r0 in range(0, rows, 512):
            r1 = min(rows, r0 + 512)
            i = torch.arange(ln + r0, ln + r1, device=slab.device)[:, None]
            j = torch.arange(n, device=slab.device)[None]
            hidden = torch.zeros(r1 - r0, n, dtype=torch.bool, device=slab.device)
            if case["causal"]:
                hidden |= j > i
            if case["window"]:
                hidden |= (i - j >= case["window"]) & (j >= case["sinks"])
            for h in range(case["nq"]):
                x = st["q"][first + r0:first + r1, h].double() @ kv[0, h // group].T / math.sqrt(case["d"])
                x[hidden] = -math.inf
                out[first + r0:first + r1, h] = torch.exp(x - torch.logsumexp(x, 1, True)) @ kv[1, h // group]
        first += rows
    return out


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    s = _shape(case)
    es = 2 if case["dtype"] == "bf16" else 4
    page, nkv, d = case["page"], case["nkv"], case["d"]
    if case["op"] in ("decode", "window"):
        keys = pairs = 0
        for ln, rows in zip(s["lens"], s["rows"]):
            n, w, sinks = ln + rows, case["window"] or 1 << 40, case["sinks"]
            low = max(0, ln - w + 1)
            keys += n - low + min(low, sinks)
            for r in range(rows):
                top, lo = (ln + r + 1 if case["causal"] else n), max(0, ln + r - w + 1)
                pairs += top - lo + min(lo, sinks)
        total = sum(s["rows"])
        return {"bytes": 2 * keys * nkv * d * es + 2 * total * case["nq"] * d * es, "flops": 4 * pairs * case["nq"] * d}
    row = case["layers"] * 2 * nkv * d * es                      # bytes of one position
    tables = 4 * (2 * s["total"] * s["cols"] + s["total"] + s["pages"])
    if case["op"] == "beam":      # of the 1 + width holders of a partial last page all but one copy it
        moved = sum(ln % page for ln in s["lens"]) * case["width"]
    elif case["op"] == "clone":
        moved = s["used"] * page
    elif case["op"] == "compact":
        moved = s["used"] // 2 * page
    else:
        moved = 0
        tables += 2 * sum(_turnover(case, s["lens"])[4]) * row // case["layers"]
    return {"bytes": 2 * moved * row + tables, "flops": 0}
