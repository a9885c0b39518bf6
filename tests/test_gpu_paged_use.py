"""The paged pool as a program uses it: decode cycles, captured graphs, side streams, strided
tensors, many entries, large pools, the bridge to the draft cache, and the draft step with a
sliding window."""
import threading

import pytest
import torch

from block_diffusion_speculative_03_b200 import dflash as D
from block_diffusion_speculative_03_b200 import inputs as I
from block_diffusion_speculative_03_b200.drafter import Drafter, shape_from_workload
from block_diffusion_speculative_03_b200.paging import PagePool
from tests import paged_model as M
from tests.test_gpu_paged import DT, i32, make_pool, same

pytestmark = pytest.mark.gpu


def check_rows(out, q, kv, lo, n_keys, d, dtype, causal=True, window=0, sinks=0):
    """Rows at positions lo, lo + 1, ... over kv [2, nkv, n, d]."""
    ref, mean, score = M.attention(q, kv[0], kv[1], range(lo, lo + q.shape[0]), causal, window, sinks)
    tol = M.bound(ref, mean, score, n_keys, d, dtype)
    err = ((out.double() - ref).abs() / tol).max().item()
    assert err <= 1.0, err


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_cycles_of_forked_sequences(dtype):
    """Prompt, fork, tokens on both sides, free, compact: every attention against the model."""
    layers, nq, nkv, d, page = 2, 8, 2, 64, 16
    pool, model = make_pool(dtype, layers, nq, nkv, d, 60, page, 5, 300)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)

    def rand(*shape):
        return torch.randn(*shape, device="cuda", generator=g).to(DT[dtype])

    def step(seqs, counts, causal=True, window=0, sinks=0):
        total, most = sum(counts), max(counts)
        start = [sum(counts[:i]) for i in range(len(counts))]
        pool.reserve(i32(counts), i32(seqs))
        model.reserve(seqs, counts)
        for layer in range(layers):
            # slices of one projection, as a program has them
            qkv = rand(total, (nq + 2 * nkv) * d)
            q = qkv[:, :nq * d].unflatten(1, (nq, d))
            k = qkv[:, nq * d:(nq + nkv) * d].unflatten(1, (nkv, d))
            v = qkv[:, (nq + nkv) * d:].unflatten(1, (nkv, d))
            pool.write(layer, k, v, i32(seqs), i32(start), i32(counts), max_rows=most)
            model.write(layer, k, v, seqs, start, counts, total, most)
            out = pool.attention(layer, q, None, i32(seqs), i32(start), i32(counts), most, causal, window, sinks)
            for i, s in enumerate(seqs):
                n = model.len[s] + counts[i]
                check_rows(out[start[i]:start[i] + counts[i]], q[start[i]:start[i] + counts[i]],
                           model.rows_of(s, n)[layer], model.len[s], n, d, DT[dtype], causal, window, sinks)
        pool.advance(i32(counts), i32(seqs))
        model.advance(seqs, counts)
        same(pool, model, (seqs, counts))

    step([0, 1], [70, 5])
    pool.fork(i32([0, 0, 1]), i32([2, 3, 4]))
    model.fork([0, 0, 1], [2, 3, 4])
    step([4, 2, 0, 3, 1], [1, 1, 1, 1, 1])
    step([2, 3], [16, 9], causal=False, window=20, sinks=3)
    pool.free(i32([3, 1]))
    model.free([3, 1])
    assert pool.compact().item() == model.compact()
    same(pool, model, "compact")
    step([0, 2, 4], [1, 1, 1], window=33, sinks=1)
    pool.free(i32([0]), keep=i32([20]))
    model.free([0], [20])
    step([0], [40])


def test_captured_cycle_equals_eager():
    """A decode cycle captured once and replayed: lengths, pages and outputs as run eagerly."""
    layers, nq, nkv, d, n, steps = 2, 8, 2, 128, 3, 40
    torch.manual_seed(0)
    q, k, v = (torch.randn(steps, n, h, d, device="cuda").bfloat16() for h in (nq, nkv, nkv))
    results = []
    for captured in (False, True):
        pool, _ = make_pool("bf16", layers, nq, nkv, d, 40, 16, 6, 100)
        ones = i32([1] * n)
        pool.reserve(i32([20, 3, 40]))
        pool.advance(i32([20, 3, 40]))
        pool.fork(i32([0]), i32([5]))                  # the first step copies a shared page
        qs, ks, vs = (torch.empty_like(t[0]) for t in (q, k, v))
        outs = torch.empty(layers, n, nq, d, device="cuda", dtype=torch.bfloat16)

        def cycle():
            pool.reserve(ones)
            for layer in range(layers):
                pool.write(layer, ks, vs)
                pool.attention(layer, qs, outs[layer], window=50, sinks=2)
            pool.advance(ones)

        if captured:
            keep = (pool.len.clone(), pool.table.clone())
            warm = torch.cuda.Stream()
            warm.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(warm):
                cycle()
                pool.set_tables(*(x for x in keep))
            torch.cuda.current_stream().wait_stream(warm)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                cycle()
        got = []
        for t in range(steps):
            for dst, src in ((qs, q), (ks, k), (vs, v)):
                dst.copy_(src[t])
            graph.replay() if captured else cycle()
            got.append(outs.clone())
        assert pool.status() == 0
        results.append((torch.stack(got), pool.len.clone()))
    assert torch.equal(results[0][0], results[1][0])
    assert torch.equal(results[0][1], results[1][1])


def test_two_graphs_of_one_pool_take_turns():
    """Two captured attentions of one pool share its scratch: replayed in any order, their results
    are those of eager calls."""
    pool, _ = make_pool("bf16", 1, 8, 1, 128, 300, 16, 4, 1100)
    pool.reserve(i32([1001, 301, 17, 801]))
    pool.advance(i32([985, 285, 1, 785]))
    torch.manual_seed(1)
    qa, qb = torch.randn(4, 8, 128, device="cuda").bfloat16(), torch.randn(64, 8, 128, device="cuda").bfloat16()
    start, count = i32([0, 16, 32, 48]), i32([16] * 4)
    oa, ob = torch.empty_like(qa), torch.empty_like(qb)
    calls = [lambda: pool.attention(0, qa, oa), lambda: pool.attention(0, qb, ob, None, start, count, 16)]
    want = []
    for f, o in zip(calls, (oa, ob)):
        f()
        want.append(o.clone())
    graphs = []
    for f in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f()
        graphs.append(g)
    for i in (0, 1, 1, 0, 0, 1, 0, 1):
        (oa if i == 0 else ob).fill_(0)
        graphs[i].replay()
        assert torch.equal((oa, ob)[i], want[i])
    assert pool.status() == 0


def test_side_stream():
    pool, model = make_pool("bf16", 1, 4, 2, 64, 30, 16, 3, 200)
    side = torch.cuda.Stream()
    torch.manual_seed(2)
    k, v = (torch.randn(90, 2, 64, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(3, 4, 64, device="cuda").bfloat16()
    start, count = i32([0, 50, 80]), i32([50, 30, 10])
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pool.reserve(i32([51, 31, 11]))
        pool.write(0, k, v, None, start, count, max_rows=50)
        pool.advance(count)
        pool.write(0, k[:3], v[:3])
        out = pool.attention(0, q)
        st = pool.status()
    assert st == 0
    model.reserve([0, 1, 2], [51, 31, 11])
    model.write(0, k, v, [0, 1, 2], [0, 50, 80], [50, 30, 10], 90, 50)
    model.advance([0, 1, 2], [50, 30, 10])
    model.write(0, k[:3], v[:3], [0, 1, 2], [0, 1, 2], [1, 1, 1], 3, 1)
    for s in range(3):
        n = model.len[s] + 1
        check_rows(out[s:s + 1], q[s:s + 1], model.rows_of(s, n)[0], n - 1, n, 64, torch.bfloat16)


@pytest.mark.parametrize("n,left_out", [(9, []), (9, [3]), (1023, []), (1023, [0, 700])])
def test_wide_forks_write_at_once(n, left_out):
    """Every holder of a shared page reserves in one call, in a shuffled order: all but the last copy
    it, or all of them when a holder stands aside."""
    pool, model = make_pool("bf16", 1, 2, 1, 64, 3 * n + 40, 16, n + 1, 80)
    pool.reserve(i32([40]), i32([0]))
    model.reserve([0], [40])
    pool.advance(i32([37]), i32([0]))
    model.advance([0], [37])
    pool.fork(i32([0] * n), i32(list(range(1, n + 1))))
    model.fork([0] * n, list(range(1, n + 1)))
    g = torch.Generator()
    g.manual_seed(n)
    order = [s for s in torch.randperm(n + 1, generator=g).tolist() if s not in left_out]
    grow = [(s * 7) % 25 for s in order]
    pool.reserve(i32(grow), i32(order))
    model.reserve(order, grow)
    same(pool, model, "reserve")
    counts = [min(x, 9) for x in grow]
    if left_out:                                            # (room for a sequence that is listed twice)
        order, counts = order + order[:1], counts + [1]
    pool.advance(i32(counts), i32(order))
    model.advance(order, counts)
    same(pool, model, "advance")


@pytest.mark.parametrize("rows,window,page,d", [(16, 4096, 64, 128), (16, 300, 16, 64), (1, 0, 64, 128),
                                                (60, 500, 64, 128), (9, 0, 32, 64)])
def test_many_calls_with_a_cold_cache(rows, window, page, d):
    """The same call hundreds of times, its keys in the L2 cache or flushed from it: loads that come
    early or late change nothing."""
    pool, _ = make_pool("bf16", 1, 16, 4, d, 4 * 8300 // page, page, 4, 8300)
    lens = [8192, 8000, 100, 5001]
    pool.reserve(i32([n + rows for n in lens]))
    pool.advance(i32(lens))
    torch.manual_seed(rows)
    q = torch.randn(4 * rows, 16, d, device="cuda").bfloat16()
    args = (i32([0, 1, 2, 3]), i32([0, rows, 2 * rows, 3 * rows]), i32([rows] * 4), rows, rows == 1)
    flush = torch.empty(40 << 20, dtype=torch.int32, device="cuda")
    want = pool.attention(0, q, None, *args, window, 16).clone()
    slab = pool.slab()
    for s, n in enumerate(lens):
        pages = pool.table[s, :M.ceil_div(n + rows, page)].long()
        kv = slab[pages, 0].permute(1, 2, 0, 3, 4).flatten(2, 3)[:, :, :n + rows]
        mine = slice(s * rows, (s + 1) * rows)
        check_rows(want[mine], q[mine], kv, n, n + rows, d, torch.bfloat16, rows == 1, window, 16)
    out, off = torch.empty_like(want), torch.zeros((), dtype=torch.int64, device="cuda")
    for k in range(600):
        if k % 5 == 0:
            flush.fill_(k)
        pool.attention(0, q, out, *args, window, 16)
        off += (out.view(torch.int16) != want.view(torch.int16)).sum()
    assert off.item() == 0 and pool.status() == 0


def test_two_pools_on_two_streams():
    """Calls of different pools at once: tokens, blocks and page operations beside one another."""
    torch.manual_seed(5)
    pools, calls, want = [], [], []
    for k in range(2):
        pool, _ = make_pool("bf16", 1, 8, 2, 128, 400, 16, 5, 1500, seed=k)
        pool.reserve(i32([1200, 40, 700, 3]))
        pool.advance(i32([1184, 24, 684, 0]))
        qa, qb = torch.randn(4, 8, 128, device="cuda").bfloat16(), torch.randn(64, 8, 128, device="cuda").bfloat16()
        oa, ob = torch.empty_like(qa), torch.empty_like(qb)
        args = (i32([0, 1, 2, 3]), i32([0, 16, 32, 48]), i32([16, 16, 16, 3]))
        src, dst = i32([2]), i32([4])

        def call(pool=pool, qa=qa, qb=qb, oa=oa, ob=ob, args=args, src=src, dst=dst):
            pool.attention(0, qb, ob, *args, 16, window=500, sinks=4)
            pool.attention(0, qa, oa, args[0])
            pool.fork(src, dst, deep=True)
            pool.free(dst)

        call()
        pools.append(pool)
        calls.append(call)
        want.append((oa, oa.clone(), ob, ob.clone()))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(30):
        for st, call in zip(streams, calls):
            with torch.cuda.stream(st):
                call()
    torch.cuda.synchronize()
    for pool, (oa, wa, ob, wb) in zip(pools, want):
        assert pool.status() == 0
        assert torch.equal(oa, wa) and torch.equal(ob[:51], wb[:51])


def test_two_pools_from_two_threads():
    """Host threads with a pool each: the library keeps nothing that they share unguarded."""
    def work(k, errors):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                pool, model = make_pool(("bf16", "f32")[k], 1, 8, 2, 64, 60, 16, 4, 300, seed=k)
                seqs = [0, 1, 2]
                for step in range(25):
                    counts = [(step * 5 + s * 3) % 9 + 1 for s in seqs]
                    pool.reserve(i32(counts))
                    model.reserve(seqs, counts)
                    q = torch.randn(sum(counts), 8, 64, device="cuda").to(pool.torch_dtype)
                    start = [0, counts[0], counts[0] + counts[1]]
                    out = pool.attention(0, q, None, None, i32(start), i32(counts), max(counts))
                    for s in seqs:
                        rows = slice(start[s], start[s] + counts[s])
                        n = model.len[s] + counts[s]
                        check_rows(out[rows], q[rows], model.rows_of(s, n)[0], model.len[s], n, 64, pool.torch_dtype)
                    pool.advance(i32(counts))
                    model.advance(seqs, counts)
                same(pool, model, k)
        except BaseException as e:      # noqa: B036 (handed to the test's own thread)
            errors.append(e)

    errors = []
    threads = [threading.Thread(target=work, args=(k % 2, errors)) for k in range(4)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors, errors


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 3, 40])
def test_many_entries_of_few_sequences(dtype, rows):
    """More entries than threads, sequences repeated, every third entry padding."""
    nq, nkv, d = 4, 2, 64
    pool, model = make_pool(dtype, 1, nq, nkv, d, 60, 16, 7, 200)
    lens = [0, 1, 15, 63, 64, 100, 7]
    pool.reserve(i32([n + rows for n in lens]))
    model.reserve(list(range(7)), [n + rows for n in lens])
    pool.advance(i32(lens))
    model.advance(list(range(7)), lens)
    n = 1000
    seqs = [-1 if i % 3 == 2 else (i * 5) % 7 for i in range(n)]
    q = torch.randn(n * rows, nq, d, device="cuda").to(DT[dtype])
    out = torch.full_like(q, 7.0)
    pool.attention(0, q, out, i32(seqs), i32([i * rows for i in range(n)]), i32([rows] * n), rows)
    assert pool.status() == 0
    for i in list(range(0, n, 37)) + [2, 998, 999]:
        mine = slice(i * rows, (i + 1) * rows)
        if seqs[i] < 0:
            assert (out[mine] == 7).all()
        else:
            s = seqs[i]
            check_rows(out[mine], q[mine], model.rows_of(s, lens[s] + rows)[0], lens[s], lens[s] + rows, d, DT[dtype])


@pytest.mark.parametrize("nq,nkv,d,rows", [(8, 2, 128, 4), (8, 2, 64, 8), (8, 2, 128, 16), (8, 2, 64, 16),
                                           (8, 2, 128, 60), (12, 4, 64, 43)])
@pytest.mark.parametrize("ctx", [300, 6000])
@pytest.mark.parametrize("window", [0, 170])
def test_rising_and_falling_scores(nq, nkv, d, rows, ctx, window):
    """The running maximum of some rows rises by 2^50 every 64 keys, of others it falls: every tile moves
    bases, in each of the kernels' row layouts, within a share and across shares."""
    pool, _ = make_pool("bf16", 1, nq, nkv, d, 120, 64, 1, ctx + rows)
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)
    slab = pool.slab()
    pool.reserve(i32([ctx + rows]))
    pool.advance(i32([ctx]))
    n = ctx + rows
    k = torch.randn(nkv, n, d, device="cuda", generator=g)
    ramp = torch.arange(n, device="cuda") // 8 * (4.0 if ctx < 1000 else 0.5)      # scores: times q[.., 0] / sqrt(d)
    k[:, :, 0] = ramp
    v = torch.randn(nkv, n, d, device="cuda", generator=g)
    q = torch.randn(rows, nq, d, device="cuda", generator=g)
    q[:, :, 0] = torch.where(torch.rand(rows, nq, device="cuda", generator=g) < 0.5, 1.0, -1.0) * d ** 0.5
    pages = pool.table[0, :M.ceil_div(n, 64)].long()
    for kind, x in ((0, k), (1, v)):
        x = torch.nn.functional.pad(x, (0, 0, 0, len(pages) * 64 - n)).unflatten(1, (-1, 64)).transpose(0, 1)
        slab[pages, 0, kind] = x.bfloat16()
    kv = slab[pages, 0].permute(1, 2, 0, 3, 4).flatten(2, 3)[:, :, :n]
    q = q.bfloat16()
    out = pool.attention(0, q, None, i32([0]), i32([0]), i32([rows]), rows, True, window, 3)
    assert pool.status() == 0 and torch.isfinite(out.float()).all()
    check_rows(out, q, kv, ctx, n, d, torch.bfloat16, True, window, 3)


@pytest.mark.parametrize("rows", [4, 8, 16, 50])
@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_bad_keys_stay_in_the_rows_that_see_them(rows, bad):
    """A key of the call's own rows that is not a number: the rows before it do not see it."""
    pool, model = make_pool("bf16", 1, 8, 2, 128, 40, 16, 2, 400)
    ctx, at = 250, rows // 2
    pool.reserve(i32([ctx + rows, ctx + rows]))
    pool.advance(i32([ctx, ctx]))
    model.reserve([0, 1], [ctx + rows] * 2)
    slab = pool.slab()
    page = pool.table[0, (ctx + at) // 16].item()
    slab[page, 0, 0, 1, (ctx + at) % 16] = float(bad)
    q = torch.randn(2 * rows, 8, 128, device="cuda").bfloat16()
    out = pool.attention(0, q, None, None, i32([0, rows]), i32([rows, rows]), rows)
    for s in range(2):
        kv = model.rows_of(s, ctx + rows)[0]           # (the model's rows are as they were before)
        good = at if s == 0 else rows
        check_rows(out[s * rows:s * rows + good], q[s * rows:s * rows + good], kv, ctx, ctx + rows, 128, torch.bfloat16)
    assert torch.isfinite(out[at:rows, :4].float()).all()          # the other kv head
    seen = out[at:rows, 4:].float()
    assert torch.isnan(seen).any() if bad == "inf" else torch.isnan(seen).all()


def test_large_pool_and_long_context():
    """Pages past 4 GB of the slab, and a context of 200000 positions."""
    layers, nkv, d, page = 10, 2, 128, 64
    per = layers * 2 * nkv * page * d * 2
    pages = (6 << 30) // per
    n = 200000
    pool = PagePool(layers, 8, nkv, d, "bf16", n_pages=pages, page_size=page, max_seqs=2, max_len=n + 64)
    slab = pool.slab()
    need = M.ceil_div(n + 17, page)
    tab = torch.full((2, pool.max_pages), -1, dtype=torch.int32)
    tab[1, :need] = torch.arange(pages - 1, pages - 1 - need, -1, dtype=torch.int32)
    pool.set_tables(i32([0, n]), tab.cuda())
    layer = layers - 1
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    for x in range(0, need, 256):
        ids = tab[1, x:min(need, x + 256)].long().cuda()
        slab[ids, layer] = (torch.randn(len(ids), 2, nkv, page, d, device="cuda", generator=g)).bfloat16()
    kv = slab[tab[1, :need].long().cuda(), layer].permute(1, 2, 0, 3, 4).flatten(2, 3)
    for rows in (1, 17):
        # large scores: a few keys make up a row's result, so a wrong page shows
        q = torch.randn(rows, 8, d, device="cuda", generator=g).bfloat16() * 8
        out = pool.attention(layer, q, None, i32([1]), i32([0]), i32([rows]), rows)
        assert pool.status() == 0
        check_rows(out, q, kv[:, :, :n + rows], n, n + rows, d, torch.bfloat16)
    k, v = (torch.randn(1, nkv, d, device="cuda", generator=g).bfloat16() for _ in range(2))
    pool.write(layer, k, v, i32([1]))
    assert torch.equal(slab[tab[1, n // page], layer, 0, :, n % page], k[0])
    assert torch.equal(slab[tab[1, n // page], layer, 1, :, n % page], v[0])
    # the context copied to the pages at the other end, then moved there
    pool.fork(i32([1]), i32([0]), deep=True)
    whole = M.ceil_div(n, page)
    assert pool.table[0, :whole].tolist() == list(range(whole))
    for x in range(0, whole, 256):
        ids = tab[1, x:min(whole, x + 256)].long().cuda()
        assert torch.equal(slab[x:x + len(ids)], slab[ids])
    pool.free(i32([0]))
    assert pool.compact().item() == need and pool.status() == 0
    moved = pool.table[1, :need].long()
    assert moved.max().item() == need - 1
    assert torch.equal(slab[moved, layer].permute(1, 2, 0, 3, 4).flatten(2, 3)[:, :, :n], kv[:, :, :n])


def drafter(w):
    W = I.make_weights(w, device="cuda")
    return Drafter(shape_from_workload(w), W, max_batch=w.batch, max_rows=512, max_position=600, max_gamma=w.gamma)


@pytest.mark.parametrize("dtype,nkv,d,page", [("bf16", 2, 128, 32), ("f32", 2, 64, 16), ("bf16", 1, 64, 64)])
def test_store_and_load(dtype, nkv, d, page):
    """Contexts from a draft cache to pages and back, appended, shared and refused."""
    w = I.Workload("bridge", 256, 2, 4, nkv, d, 512, 1000, 1, 256, 1e6, 1e-6, dtype, batch=3, gamma=4,
                   context=[1, 1, 1], mask_id=999, seed=5)
    dr = drafter(w)
    cache, back = dr.new_cache(3, 260), dr.new_cache(3, 200)
    torch.manual_seed(3)
    for c in (cache, back):
        c.slab().copy_(torch.randn(c.slab().shape, device="cuda"))
    pool = dr.new_pool(40, page, 5, 300)
    cache.set_len(torch.tensor([100, 17, 230], dtype=torch.int32))
    pool.reserve(i32([230, 100, 17]), i32([4, 0, 2]))
    pool.store(cache, i32([0, 2, 4]))
    assert pool.status() == 0 and pool.len.tolist() == [100, 0, 17, 0, 230]
    slab, src = pool.slab(), cache.slab()

    def rows(s, n):
        ids = pool.table[s, :M.ceil_div(n, page)].long()
        return slab[ids].permute(1, 2, 3, 0, 4, 5).flatten(3, 4)[:, :, :, :n]

    for s, b, n in ((0, 0, 100), (2, 1, 17), (4, 2, 230)):
        assert torch.equal(rows(s, n), src[b, :, :, :, :n])
    # nothing to add: nothing happens; more: only the rest is written
    before = pool.slab().view(torch.uint8).clone()             # bytes: unwritten rows may read as NaN
    pool.store(cache, i32([0, 2, 4]))
    assert torch.equal(pool.slab().view(torch.uint8), before) and pool.status() == 0
    cache.set_len(torch.tensor([103, 17, 230], dtype=torch.int32))
    pool.store(cache, i32([0, -1, 4]))
    assert pool.status() == (0 if M.ceil_div(103, page) <= M.ceil_div(100, page) else -5)
    pool.reserve(i32([10]), i32([0]))
    src[0, :, :, :, :100] = 0
    pool.store(cache, i32([0]), i32([0]))
    assert pool.status() == 0 and pool.len[0].item() == 103
    assert (rows(0, 100) != 0).any()
    assert torch.equal(rows(0, 103)[:, :, :, 100:], src[0, :, :, :, 100:103])
    # a page that a fork holds too is refused; reserved (copied) first, it is written
    pool.fork(i32([2]), i32([1]))
    cache.set_len(torch.tensor([103, 19, 230], dtype=torch.int32))
    pool.store(cache, i32([1]), i32([1]))
    shared = 17 % page != 0
    assert pool.status() == (-6 if shared else -5)
    pool.reserve(i32([2]), i32([1]))
    pool.store(cache, i32([1]), i32([1]))
    assert pool.status() == 0 and pool.len[1].item() == 19
    assert torch.equal(rows(1, 19), src[1, :, :, :, :19]) and torch.equal(rows(2, 17), src[1, :, :, :, :17])
    # back into another cache: appended to what it has, too long refused
    back.set_len(torch.tensor([3, 0, 5], dtype=torch.int32))
    keep = back.slab().clone()
    pool.load(back, i32([0, 1, 4]))
    assert pool.status() == -5
    assert back.len.tolist() == [103, 19, 5] and back.committed.tolist() == [103, 19, 5]
    got = back.slab()
    assert torch.equal(got[0, :, :, :, 3:103], rows(0, 103)[:, :, :, 3:])
    assert torch.equal(got[0, :, :, :, :3], keep[0, :, :, :, :3])
    assert torch.equal(got[1, :, :, :, :19], rows(1, 19)) and torch.equal(got[2], keep[2])
    assert torch.equal(got[0, :, :, :, 103:], keep[0, :, :, :, 103:])
    # the same request twice, requests and sequences that do not exist
    pool.load(back, i32([4, 0]), i32([2, 2]))
    assert pool.status() in (-1, -5)
    for seqs, reqs in (([5], [0]), ([0], [3]), ([-2], [0])):
        pool.load(back, i32(seqs), i32(reqs))
        assert pool.status() == -1
    w.n_layers = 1
    with pytest.raises(D.DflashError):                                # another shape
        pool.store(drafter(w).new_cache(3, 64))


@pytest.mark.parametrize("gamma,nq,nkv,d", [(16, 8, 2, 128), (4, 4, 2, 64), (16, 8, 1, 128), (5, 6, 2, 64)])
@pytest.mark.parametrize("window,sinks", [(64, 4), (7, 0), (100000, 0), (300, 90)])
def test_draft_step_with_a_window(gamma, nq, nkv, d, window, sinks):
    """Every layer's attention of a drafted block against the formula on the step's own q, K and V;
    the same step without the window is left as it was."""
    w = I.Workload("win", 256, 2, nq, nkv, d, 512, 1000, 1, 256, 1e6, 1e-6, "bf16", batch=3, gamma=gamma,
                   context=[500, 3, 130], mask_id=999, seed=6)
    dr = drafter(w)
    cache = dr.new_cache(3, 540)
    lens = [500, 3, 130]
    slab = cache.slab()
    for b in range(3):
        for l in range(2):
            for kind in (0, 1):
                slab[b, l, kind, :, :lens[b]] = I.synthetic_cache_rows(w, l, kind, b, lens[b], device="cuda")
    cache.set_len(torch.tensor(lens, dtype=torch.int32))
    anchors = I.make_anchors(w, device="cuda")
    logits = torch.empty(3, gamma - 1, 1000, device="cuda")
    plain = dr.draft_block(cache, anchors, gamma, logits=logits).clone()
    plain_logits = logits.clone()
    assert cache.status() == 0
    q = torch.zeros(2, 3 * gamma, nq * d, device="cuda", dtype=torch.bfloat16)
    o = torch.zeros_like(q)
    cache.set_window(window, sinks)
    D.dflash_diag_draft_capture_stages(dr.handle, q=q.data_ptr(), o=o.data_ptr())
    dr.draft_block(cache, anchors, gamma, logits=logits)
    D.dflash_diag_draft_capture_stages(dr.handle)
    assert cache.status() == 0

    def check(l, b):
        rows = slice(b * gamma, (b + 1) * gamma)
        kv = slab[b, l, :, :, :lens[b] + gamma]
        check_rows(o[l, rows].unflatten(1, (nq, d)), q[l, rows].unflatten(1, (nq, d)), kv, lens[b], lens[b] + gamma, d,
                   torch.bfloat16, causal=False, window=window, sinks=sinks)

    for l in range(2):
        for b in range(3):
            check(l, b)
    # a request that cannot be drafted (its anchor does not exist) is skipped, the others proceed
    # (their keys are split in another way then: the same results to rounding)
    bad = anchors.clone()
    bad[1] = 1000
    o.zero_()
    D.dflash_diag_draft_capture_stages(dr.handle, q=q.data_ptr(), o=o.data_ptr())
    dr.draft_block(cache, bad, gamma, logits=logits)
    D.dflash_diag_draft_capture_stages(dr.handle)
    assert cache.status() == -7
    for l in range(2):
        check(l, 0)
        check(l, 2)
    cache.set_window(0)
    again = dr.draft_block(cache, anchors, gamma, logits=logits)
    assert torch.equal(again, plain) and torch.equal(logits, plain_logits)


@pytest.mark.parametrize("window,sinks", [(32, 2), (1, 0), (100000, 0)])
def test_ingest_with_a_window(window, sinks):
    """Rows appended through the layers: the first layer's attention against the formula (the last
    layer has none), causally."""
    w = I.Workload("win", 256, 2, 8, 2, 128, 512, 1000, 1, 256, 1e6, 1e-6, "bf16", batch=2, gamma=16,
                   context=[200, 3], mask_id=999, seed=7)
    dr = drafter(w)
    cache = dr.new_cache(2, 260)
    slab = cache.slab()
    for b, n in enumerate(w.context):
        for l in range(2):
            for kind in (0, 1):
                slab[b, l, kind, :, :n] = I.synthetic_cache_rows(w, l, kind, b, n, device="cuda")
    cache.set_len(torch.tensor(w.context, dtype=torch.int32))
    cache.set_window(window, sinks)
    ctx = I.normal(3, 1, (32, 256), 1.0, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(2, 32, 8 * 128, device="cuda", dtype=torch.bfloat16)
    o = torch.zeros_like(q)
    D.dflash_diag_draft_capture_stages(dr.handle, q=q.data_ptr(), o=o.data_ptr())
    dr.ingest_fused_input(cache, ctx, 16)
    D.dflash_diag_draft_capture_stages(dr.handle)
    assert cache.status() == 0 and cache.len.tolist() == [216, 19]
    for b, n in enumerate(w.context):
        rows = slice(b * 16, (b + 1) * 16)
        check_rows(o[0, rows].unflatten(1, (8, 128)), q[0, rows].unflatten(1, (8, 128)), slab[b, 0, :, :, :n + 16], n,
                   n + 16, 128, torch.bfloat16, causal=True, window=window, sinks=sinks)


def test_window_is_refused():
    w = I.Workload("f", 256, 1, 4, 2, 64, 512, 1000, 1, 256, 1e6, 1e-6, "f32", batch=1, gamma=4, context=[1],
                   mask_id=999, seed=5)
    cache = drafter(w).new_cache(1, 64)
    with pytest.raises(D.DflashError) as e:
        cache.set_window(8)
    assert e.value.status == -2                                       # fp32 handles
    w.dtype = "bf16"
    dr = drafter(w)
    cache = dr.new_cache(1, 64)
    for args, status in (((-1, 0), -1), ((8, -1), -1)):
        with pytest.raises(D.DflashError) as e:
            cache.set_window(*args)
        assert e.value.status == status
    buf = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    assert D.dflash_cache_set_window(cache.handle, 8, 0, buf.data_ptr() // 256 * 256 + 256, 1 << 19, check=False) == -4
    assert D.dflash_cache_set_window(cache.handle, 8, 0, None, 1 << 30, check=False) == -1


def test_arguments_are_refused_before_anything_runs():
    pool, model = make_pool("bf16", 1, 4, 2, 64, 8, 16, 2, 64)
    lib, h = D.lib(), pool.handle
    q = torch.zeros(2, 4, 64, device="cuda", dtype=torch.bfloat16)
    o, n = torch.zeros_like(q), pool.launch_count()
    qp, op = q.data_ptr(), o.data_ptr()
    ok = dict(seqs=None, n=2, layer=0, q=qp, stride=256, start=None, count=None, total=2, rows=1, causal=1, window=0,
              sinks=0, out=op)
    for kw in (dict(n=-1), dict(n=3), dict(layer=-1), dict(layer=1), dict(total=1), dict(rows=0), dict(window=-1),
               dict(sinks=-1), dict(q=None), dict(q=qp + 2), dict(out=None), dict(out=op + 8), dict(stride=255),
               dict(stride=260), dict(start=qp), dict(count=qp), dict(total=-1), dict(rows=-1)):
        a = dict(ok, **kw)
        assert lib.dflash_paged_attention(h, *a.values(), None) == -1, kw
    k = torch.zeros(2, 2, 64, device="cuda", dtype=torch.bfloat16).data_ptr()
    ok = dict(seqs=None, n=2, layer=0, k=k, v=k, stride=128, start=None, count=None, total=2, rows=1)
    for kw in (dict(n=-1), dict(n=3), dict(layer=1), dict(total=1), dict(rows=0), dict(k=None), dict(v=k + 4),
               dict(stride=127), dict(stride=132), dict(start=k)):
        assert lib.dflash_pages_write(h, *dict(ok, **kw).values(), None) == -1, kw
    assert lib.dflash_pages_reserve(h, None, None, 1, None) == -1
    assert lib.dflash_pages_reserve(h, None, k, 3, None) == -1
    assert lib.dflash_pages_fork(h, k, None, 1, 0, None) == -1
    assert lib.dflash_pages_compact(h, None, None) == -1
    assert lib.dflash_pool_set_tables(h, k, None, None) == -1
    assert pool.launch_count() == n
    # no entries, no rows: fine, and nothing runs
    assert lib.dflash_paged_attention(h, None, 0, 0, qp, 256, None, None, 2, 1, 1, 0, 0, op, None) == 0
    pool.reserve(torch.empty(0, dtype=torch.int32, device="cuda"))
    assert pool.attention(0, q[:0]).shape == (0, 4, 64)
    assert pool.launch_count() == n
    same(pool, model, "untouched")
    # the Python layer's own checks
    for bad in (q.float(), q.cpu(), q[:, :2], q.transpose(1, 2).contiguous().transpose(1, 2)):
        with pytest.raises(ValueError):
            pool.attention(0, bad)
    with pytest.raises(ValueError):
        pool.attention(0, q, torch.empty(2, 4, 64, device="cuda"))
    with pytest.raises(ValueError):
        pool.reserve(torch.ones(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        pool.reserve(torch.ones(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        pool.reserve(i32([1, 1]), i32([0]))
    with pytest.raises(ValueError):
        pool.attention(0, q, row_start=i32([0]))
    with pytest.raises(ValueError):
        pool.attention(0, q, seqs=i32([0, 1, 0]))
    with pytest.raises(ValueError):
        pool.write(0, q[:, :2], q[:1, :2])
    with pytest.raises(ValueError):
        pool.set_tables(pool.len, pool.table[:1].contiguous())
