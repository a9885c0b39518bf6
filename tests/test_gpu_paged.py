"""Page operations and attention over a paged pool, against the plain model of
tests/paged_model.py: page operations exactly, attention within derived bounds."""
import random

import pytest
import torch

from block_diffusion_speculative_03_b200 import dflash as D
from block_diffusion_speculative_03_b200.paging import PagePool
from tests import paged_model as M

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def make_pool(dtype="bf16", layers=2, nq=4, nkv=2, d=64, pages=40, page=16, seqs=6, max_len=200, seed=0, fill=None):
    pool = PagePool(layers, nq, nkv, d, dtype, n_pages=pages, page_size=page, max_seqs=seqs, max_len=max_len)
    slab = pool.slab()
    if fill is not None:
        slab.fill_(fill)
    else:
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        slab.copy_(torch.randn(slab.shape, device="cuda", generator=g) * 1.28)
    return pool, M.PoolModel(pages, page, seqs, max_len, slab)


def same(pool, model, what):
    assert pool.len.tolist() == model.len, what
    assert pool.table.tolist() == model.table().tolist(), what
    assert pool.refs.tolist() == model.refs(), what
    bits = torch.int16 if pool.torch_dtype == torch.bfloat16 else torch.int32
    off = (pool.slab().view(bits) != model.slab.view(bits)).sum().item()
    assert off == 0, (what, off)
    st = pool.status()
    assert st in model.err if model.err else st == 0, (what, st, model.err)
    model.err = set()


# ---------------------------------------------------------------------------
# Page operations
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,d,page,seed", [("bf16", 64, 16, 0), ("bf16", 128, 32, 1), ("f32", 64, 16, 2),
                                               ("f32", 128, 64, 3), ("bf16", 64, 256, 4), ("bf16", 64, 16, 5)])
def test_random_operations_match_the_model(dtype, d, page, seed):
    r = random.Random(seed)
    seqs = 9
    max_len = 11 * page + 3
    pool, model = make_pool(dtype, 2, 4, 2, d, 60, page, seqs, max_len, seed)
    for step in range(120):
        op = r.choice(["reserve", "reserve", "grow", "grow", "fork", "deep", "free", "cut", "compact", "write"])
        n = r.randint(1, seqs)
        ids = [r.choice([-1, r.randrange(seqs), r.randrange(seqs), seqs]) if r.random() < 0.2 else i
               for i in r.sample(range(seqs), n)]
        if op in ("reserve", "grow"):
            grow = [r.choice([0, 1, 5, page, 3 * page + 1, -1 if r.random() < 0.1 else 2]) for _ in ids]
            pool.reserve(i32(grow), i32(ids))
            model.reserve(ids, grow)
            same(pool, model, (step, op, ids, grow))
            if op == "grow":
                pool.advance(i32(grow), i32(ids))
                model.advance(ids, grow)
        elif op in ("fork", "deep"):
            src = [r.randrange(seqs) for _ in ids]
            pool.fork(i32(src), i32(ids), deep=op == "deep")
            model.fork(src, ids, op == "deep")
        elif op == "free":
            pool.free(i32(ids))
            model.free(ids)
        elif op == "cut":
            keep = [r.randint(0, max(model.len) + 1) for _ in ids]
            pool.free(i32(ids), keep=i32(keep))
            model.free(ids, keep)
        elif op == "compact":
            used = pool.compact()
            assert used.item() == model.compact()
        else:
            count = [r.choice([0, 1, 3, page + 2]) for _ in ids]
            start = [sum(count[:j]) for j in range(len(ids))]
            total = sum(count) + 2
            k, v = (torch.randn(total, 2, d, device="cuda").to(DT[dtype]) for _ in range(2))
            layer = r.randrange(2)
            most = max(max(count), 1)
            pool.write(layer, k, v, i32(ids), i32(start), i32(count), max_rows=most)
            model.write(layer, k, v, ids, start, count, total, most)
        same(pool, model, (step, op, ids))


def test_reserve_of_many_sequences_and_pages():
    pool, model = make_pool(pages=5000, seqs=700, max_len=16 * 40, d=64, layers=1, nkv=1, nq=1)
    r = random.Random(3)
    grow = [r.choice([1, 17, 100, 16]) for _ in range(700)]
    pool.reserve(i32(grow))
    model.reserve(list(range(700)), grow)
    same(pool, model, "reserve")
    pool.advance(i32(grow))
    model.advance(list(range(700)), grow)
    gone = r.sample(range(700), 300)
    pool.free(i32(gone))
    model.free(gone)
    src = r.sample([i for i in range(700) if i not in gone], 100)
    pool.fork(i32(src), i32(gone[:100]))
    model.fork(src, gone[:100])
    same(pool, model, "fork")
    assert pool.compact().item() == model.compact()
    same(pool, model, "compact")
    pool.reserve(i32([9] * 700))
    model.reserve(list(range(700)), [9] * 700)
    same(pool, model, "copy on write")


def test_capacity_leaves_everything_as_it_was():
    pool, model = make_pool(pages=7, seqs=4, max_len=100)
    for _ in range(2):
        grow = [16, 40, 33, 0]       # 1 + 3 + 3 pages: all seven, then more than there are
        pool.reserve(i32(grow))
        model.reserve([0, 1, 2, 3], grow)
        same(pool, model, grow)
        pool.advance(i32(grow))
        model.advance([0, 1, 2, 3], grow)
    pool.fork(i32([1]), i32([3]), deep=True)
    model.fork([1], [3], deep=True)
    assert model.err == {-5}
    same(pool, model, "deep fork without room")


def test_shared_page_is_kept_by_its_last_writer():
    pool, model = make_pool(pages=20, seqs=4)
    for m, a in ((pool.reserve, (i32([20]), i32([0]))), (pool.advance, (i32([20]), i32([0])))):
        m(*a)
    model.reserve([0], [20])
    model.advance([0], [20])
    pool.fork(i32([0, 0, 0]), i32([1, 2, 3]))
    model.fork([0, 0, 0], [1, 2, 3])
    pool.reserve(i32([3, 3, 3, 3]), i32([2, 0, 3, 1]))
    model.reserve([2, 0, 3, 1], [3, 3, 3, 3])
    assert model.tab[1] == [0, 1]     # the last of the list
    same(pool, model, "four writers of one page")


def test_set_tables_checks_and_counts():
    pool, model = make_pool(pages=10, seqs=3, max_len=64)
    good = [[0, 3, -1, -1], [0, 3, 7, -1], [-1] * 4]
    pool.set_tables(i32([20, 40, 0]), i32(good))
    model.len, model.tab = [20, 40, 0], [[0, 3], [0, 3, 7], []]
    same(pool, model, "good")
    pool.set_tables(pool.len, pool.table)            # its own arrays
    same(pool, model, "own arrays")
    for lens, table in (([20, 40, 0], [[0, 3, -1, -1], [3, 0, 7, -1], [-1] * 4]),      # a page at two indices
                        ([20, 49, 0], good),                                           # too few pages
                        ([20, 40, 0], [[0, -1, 3, -1], [0, 1, 7, -1], [-1] * 4]),      # no prefix
                        ([20, 40, 0], [[0, 10, -1, -1], [0, 3, 7, -1], [-1] * 4]),     # no such page
                        ([20, -1, 0], good), ([20, 65, 0], good), ([20, 40, 0], [[0, -2, -1, -1]] + good[1:])):
        pool.set_tables(i32(lens), i32(table))
        assert pool.status() == -1
        assert pool.len.tolist() == [0, 0, 0] and pool.refs.sum().item() == 0 and (pool.table == -1).all()


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------

def check_attention(dtype, nq, nkv, d, page, lens, counts, causal, window, sinks, seed=0, scale=1.3, garbage=True,
                    layers=2, q_pad=0, uniform=False):
    """Sequences of `lens` with `counts` new rows each; every page and row that no query row may
    see is NaN."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = random.Random(seed)
    need = [M.ceil_div(a + b, page) for a, b in zip(lens, counts)]
    pages = sum(need) + 3
    pool, model = make_pool(dtype, layers, nq, nkv, d, pages, page, len(lens) + 1,
                            max(a + b for a, b in zip(lens, counts)) + 1, seed)
    ids = r.sample(range(pages), sum(need))
    slab = pool.slab()
    layer = layers - 1
    if garbage:
        keep = slab.clone()
        slab.fill_(float("nan"))
    tab = []
    for s, n in enumerate(need):
        tab.append([ids.pop() for _ in range(n)])
        total = lens[s] + counts[s]
        if garbage:
            seen = torch.zeros(n * page, dtype=torch.bool, device="cuda")
            lo = max(0, lens[s] - window + 1) if window else 0
            if counts[s]:
                seen[lo:total] = True
                seen[:min(sinks, total) if window else 0] = True
            for c, x in enumerate(tab[-1]):
                rows = seen[c * page:(c + 1) * page]
                slab[x, layer, :, :, rows] = keep[x, layer, :, :, rows]
    model.tab[:len(lens)], model.len[:len(lens)] = tab, list(lens)
    model.slab = slab
    pool.set_tables(i32(model.len), model.table().cuda())
    total = sum(counts)
    q = (torch.randn(total + 1, nq * d + q_pad, device="cuda", generator=g) * scale).to(DT[dtype])
    q = q[:total, :nq * d].unflatten(1, (nq, d))
    out = torch.full((total, nq, d), 7.0, device="cuda", dtype=DT[dtype])
    start = [sum(counts[:i]) for i in range(len(counts))]
    order = list(range(len(lens)))
    r.shuffle(order)
    if uniform:
        pool.attention(layer, q, out, causal=causal, window=window, sinks=sinks)
    else:
        pool.attention(layer, q, out, seqs=i32(order + [-1]), row_start=i32([start[i] for i in order] + [0]),
                       row_count=i32([counts[i] for i in order] + [1]), max_rows=max(counts), causal=causal,
                       window=window, sinks=sinks)
    assert pool.status() == 0
    worst = 0.0
    for s in range(len(lens)):
        if not counts[s]:
            continue
        kv = model.rows_of(s, lens[s] + counts[s])[layer]
        rows = slice(start[s], start[s] + counts[s])
        ref, mean, score = M.attention(q[rows], kv[0], kv[1], range(lens[s], lens[s] + counts[s]), causal, window, sinks)
        tol = M.bound(ref, mean, score, lens[s] + counts[s], d, DT[dtype])
        err = (out[rows].double() - ref).abs() / tol
        assert torch.isfinite(out[rows].float()).all(), s
        worst = max(worst, err.max().item())
        assert err.max().item() <= 1.0, (s, lens[s], counts[s], err.max().item())
    return worst


TOKENS = [0, 1, 14, 15, 16, 17, 31, 62, 63, 64, 65, 127, 128, 200, 511, 700]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq,nkv,d,page", [(4, 2, 64, 16), (8, 2, 128, 64), (3, 3, 128, 32), (16, 1, 64, 128),
                                           (12, 4, 64, 256), (20, 1, 128, 16)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (40, 4), (64, 70)])
def test_one_token(dtype, nq, nkv, d, page, window, sinks):
    print(check_attention(dtype, nq, nkv, d, page, TOKENS, [1] * len(TOKENS), True, window, sinks, seed=page + window))


@pytest.mark.parametrize("dtype,nq,nkv,d", [("bf16", 32, 8, 128), ("bf16", 8, 1, 64), ("f32", 4, 2, 64)])
@pytest.mark.parametrize("n", [1, 2, 5])
def test_one_token_of_long_contexts(dtype, nq, nkv, d, n):
    lens = [5000, 1, 2047, 9000, 3][:n]
    check_attention(dtype, nq, nkv, d, 64, lens, [1] * n, True, 0, 0, seed=n, uniform=n != 2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq,nkv,d,page", [(4, 2, 64, 16), (32, 8, 128, 64), (16, 2, 128, 32), (6, 2, 64, 128)])
@pytest.mark.parametrize("causal,window,sinks", [(True, 0, 0), (False, 0, 0), (True, 33, 4), (False, 50, 1),
                                                 (True, 200, 70), (False, 5, 0)])
def test_blocks(dtype, nq, nkv, d, page, causal, window, sinks):
    lens = [0, 1, 63, 64, 300, 130, 1000, 17]
    counts = [16, 3, 1, 16, 7, 0, 16, 2]
    # with a window, V rows of the first rows' reach are seen by some rows and not by others: finite
    check_attention(dtype, nq, nkv, d, page, lens, counts, causal, window, sinks, seed=page)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq,nkv,d", [(8, 2, 128), (6, 2, 64), (5, 1, 128)])
@pytest.mark.parametrize("causal,window,sinks", [(True, 0, 0), (True, 100, 4), (False, 90, 0), (False, 0, 0)])
def test_prompts(dtype, nq, nkv, d, causal, window, sinks):
    check_attention(dtype, nq, nkv, d, 32, [0, 77, 500, 5], [333, 129, 64, 1], causal, window, sinks, seed=nq,
                    q_pad=8)


def test_one_long_prompt():
    check_attention("bf16", 32, 8, 128, 64, [700], [1111], True, 256, 4, seed=1)


def test_large_scores_and_row_order():
    # scores of hundreds: the running maximum moves often, most weights vanish
    check_attention("bf16", 8, 2, 128, 16, [700, 90], [1, 1], True, 0, 0, seed=9, scale=12.0)
    check_attention("bf16", 8, 2, 128, 16, [700, 90], [16, 9], True, 0, 0, seed=9, scale=12.0)
    check_attention("f32", 8, 2, 64, 16, [700, 90], [16, 1], True, 30, 2, seed=9, scale=12.0)


def test_skipped_entries_and_untouched_rows():
    for dtype in ("bf16", "f32"):
        for count in (1, 12):
            pool, model = make_pool(dtype, 1, 8, 2, 128, 30, 16, 4, 300)
            lens = [40, 16 * 3, 7, 0]
            model.reserve([0, 2], [40 + count, 7 + count])
            pool.reserve(i32([40 + count, 7 + count]), i32([0, 2]))
            pool.reserve(i32([48]), i32([1]))
            pool.advance(i32(lens))
            assert pool.status() == 0
            q = torch.randn(6 * count, 8, 128, device="cuda").to(DT[dtype])
            out = torch.full_like(q, 7.0)
            # rows 0.. of a sequence without room (1), a good one (2), a sequence that does not exist, padding
            pool.attention(0, q, out, seqs=i32([1, 2, 4, -1]), row_start=i32([0, count, 2 * count, 3 * count]),
                           row_count=i32([count] * 4), max_rows=count)
            assert pool.status() in (-1, -5)
            assert (out[:count] == 0).all() and (out[2 * count:3 * count] == 0).all()
            assert (out[3 * count:] == 7).all()
            assert torch.isfinite(out[count:2 * count].float()).all() and (out[count:2 * count] != 7).any()
            # row ranges that do not exist are not written at all
            out.fill_(7.0)
            pool.attention(0, q, out, seqs=i32([2, 2, 2]), row_start=i32([-1, 6 * count, 0]),
                           row_count=i32([count, count, count + 1]), max_rows=count)
            assert pool.status() == -1
            assert (out == 7).all()


def test_infinite_and_nan_scores_stay_in_their_rows():
    pool, _ = make_pool("bf16", 1, 4, 2, 64, 30, 16, 3, 200)
    pool.reserve(i32([101, 101, 101]))
    pool.advance(i32([100, 100, 100]))
    slab = pool.slab()
    tab = pool.table.tolist()
    slab[tab[1][2], 0, 0, 0, 3] = float("nan")           # a key of sequence 1, kv head 0
    q = torch.randn(3, 4, 64, device="cuda").to(torch.bfloat16)
    out = pool.attention(0, q)
    assert torch.isnan(out[1, :2].float()).all()          # its two query heads
    assert torch.isfinite(out[1, 2:].float()).all() and torch.isfinite(out[[0, 2]].float()).all()


def test_same_results_whatever_stands_beside():
    # a sequence's result does not depend on the batch around it (bf16: an integer base,
    # exact powers of two; the split points move, so sums may differ in the last fp32 bits)
    pool, _ = make_pool("bf16", 1, 8, 2, 128, 400, 16, 8, 1200)
    lens = [1000, 5, 300, 64, 700, 0, 17, 900]
    pool.reserve(i32([n + 1 for n in lens]))
    pool.advance(i32(lens))
    q = torch.randn(8, 8, 128, device="cuda").to(torch.bfloat16)
    a = pool.attention(0, q)
    assert torch.equal(a, pool.attention(0, q))           # and twice the same call is the same
    for i in range(8):
        b = pool.attention(0, q[i:i + 1], seqs=i32([i]))
        assert (a[i].float() - b[0].float()).abs().max().item() <= 2 ** -7 * a[i].float().abs().max().item()
