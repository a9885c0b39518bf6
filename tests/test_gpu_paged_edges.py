"""Calls at the edge of what the paged pool's documents allow: padding beside stale ids, refused
entries among good ones, windows as long as an int holds."""
import math
import random

import pytest
import torch

from block_diffusion_speculative_03_b200 import inputs as I
from tests import paged_model as M
from tests.test_gpu_paged import i32, make_pool, same
from tests.test_gpu_paged_use import drafter

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# Padding
# ---------------------------------------------------------------------------

def model_fork(model, src, dst, deep):
    """The model's fork of the pairs that are no padding."""
    pairs = [(a, b) for a, b in zip(src, dst) if a != -1 and b != -1]
    model.fork([a for a, _ in pairs], [b for _, b in pairs], deep)


@pytest.mark.parametrize("deep", [False, True])
@pytest.mark.parametrize("src,dst", [
    ([-1, 0], [5, 5]),                 # the destination stands beside a padding source first
    ([-1, -1, 0, 1], [5, 4, 4, 5]),
    ([-1, 0], [99, 5]), ([-1, 0], [-7, 5]),        # .. or an id that does not exist does
    ([99, 0], [-1, 5]), ([-7, 0], [-1, 5]),
    ([0, 0], [-1, 5]), ([-1, -1], [-1, -1]), ([-1, 0, 0], [0, 5, 4]),
])
def test_padding_pairs_of_a_fork(deep, src, dst):
    pool, model = make_pool(seqs=6)
    pool.reserve(i32([20, 37]), i32([0, 1]))
    pool.advance(i32([20, 37]), i32([0, 1]))
    model.reserve([0, 1], [20, 37])
    model.advance([0, 1], [20, 37])
    pool.fork(i32(src), i32(dst), deep=deep)
    model_fork(model, src, dst, deep)
    assert not model.err
    same(pool, model, (src, dst))


@pytest.mark.parametrize("deep", [False, True])
def test_a_destination_in_src_is_refused_beside_padding_too(deep):
    pool, model = make_pool(seqs=6)
    pool.reserve(i32([20]), i32([0]))
    pool.advance(i32([20]), i32([0]))
    model.reserve([0], [20])
    model.advance([0], [20])
    pool.fork(i32([0, 5]), i32([5, -1]), deep=deep)
    model.err = {-1}
    same(pool, model, "refused")


@pytest.mark.parametrize("seed", range(4))
def test_random_forks_with_padding_on_either_side(seed):
    r = random.Random(seed)
    seqs, page = 12, 16
    pool, model = make_pool(pages=90, page=page, seqs=seqs, max_len=90, seed=seed)
    for step in range(60):
        n = r.randint(1, seqs)
        dst = [r.choice([-1, seqs, s, r.randrange(seqs)]) if r.random() < 0.4 else s for s in r.sample(range(seqs), n)]
        src = []
        for b in dst:
            a = r.choice([-1, -1, seqs + 3, -2, r.randrange(seqs)]) if r.random() < 0.5 else r.randrange(seqs)
            src.append(-1 if b == -1 and a in dst else a)      # (no destination beside a dst of -1)
        deep = r.random() < 0.5
        pool.fork(i32(src), i32(dst), deep=deep)
        model_fork(model, src, dst, deep)
        same(pool, model, (step, src, dst, deep))
        ids = r.sample(range(seqs), 4)
        pool.free(i32(ids))
        model.free(ids)
        grow = [r.choice([0, 3, 17, 33]) for _ in ids[:2]]
        pool.reserve(i32(grow), i32(ids[:2]))
        model.reserve(ids[:2], grow)
        same(pool, model, (step, "reserve"))
        if not model.err:
            pool.advance(i32(grow), i32(ids[:2]))
            model.advance(ids[:2], grow)
            same(pool, model, (step, "advance"))


def test_padding_pairs_of_store_and_load():
    w = I.Workload("pad", 256, 2, 4, 2, 64, 512, 1000, 1, 256, 1e6, 1e-6, "bf16", batch=3, gamma=4, context=[1, 1, 1],
                   mask_id=999, seed=5)
    dr = drafter(w)
    cache, back = dr.new_cache(3, 200), dr.new_cache(3, 200)
    torch.manual_seed(3)
    for c in (cache, back):
        c.slab().copy_(torch.randn(c.slab().shape, device="cuda"))
    cache.set_len(torch.tensor([50, 17, 90], dtype=torch.int32))
    pool = dr.new_pool(40, 16, 6, 200)
    pool.reserve(i32([90, 90]), i32([0, 3]))
    # a sequence beside a padding request, a request beside a padding sequence, ids that do not exist
    pool.store(cache, i32([0, 0, -1, -1, 77, 3]), i32([-1, 2, 1, 44, -1, 1]))
    assert pool.status() == 0 and pool.len.tolist() == [90, 0, 0, 17, 0, 0]
    ids = pool.table[0, :6].long()
    assert torch.equal(pool.slab()[ids].permute(1, 2, 3, 0, 4, 5).flatten(3, 4)[:, :, :, :90], cache.slab()[2, :, :, :, :90])
    pool.load(back, i32([-1, 0, 3, 3, -1, 77]), i32([1, 1, -1, 0, 44, -1]))
    assert pool.status() == 0 and back.len.tolist() == [17, 90, 0] and back.committed.tolist() == [17, 90, 0]
    assert torch.equal(back.slab()[1, :, :, :, :90], cache.slab()[2, :, :, :, :90])
    assert torch.equal(back.slab()[0, :, :, :, :17], cache.slab()[1, :, :, :, :17])
    # the same on both sides is still once only
    pool.store(cache, i32([1, 1]), i32([0, 0]))
    assert pool.status() in (-1, -5)
    pool.load(back, i32([0, 0]), i32([2, 2]))
    assert pool.status() == -1 and back.len.tolist() == [17, 90, 90]


# ---------------------------------------------------------------------------
# Windows that reach past every key
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,nq,nkv,d,rows", [("bf16", 8, 2, 128, 64), ("bf16", 4, 2, 64, 64), ("bf16", 2, 2, 64, 100),
                                                 ("bf16", 16, 2, 128, 300), ("bf16", 4, 2, 64, 3), ("f32", 4, 2, 64, 64)])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("window,sinks", [(2 ** 31 - 1, 0), (2 ** 31 - 40, 0), (2 ** 31 - 1, 2 ** 31 - 1), (1 << 30, 5)])
def test_a_window_longer_than_any_context(dtype, nq, nkv, d, rows, causal, window, sinks):
    lens = [100, 0, 700]
    pool, model = make_pool(dtype, 1, nq, nkv, d, 120, 16, 3, 700 + rows)
    pool.reserve(i32([n + rows for n in lens]))
    pool.advance(i32(lens))
    model.reserve([0, 1, 2], [n + rows for n in lens])
    q = torch.randn(3 * rows, nq, d, device="cuda").to(pool.torch_dtype)
    out = pool.attention(0, q, None, None, i32([0, rows, 2 * rows]), i32([rows] * 3), rows, causal, window, sinks)
    assert pool.status() == 0
    for s, n in enumerate(lens):
        mine = slice(s * rows, (s + 1) * rows)
        kv = model.rows_of(s, n + rows)[0]
        ref, mean, score = M.attention(q[mine], kv[0], kv[1], range(n, n + rows), causal, 0, 0)     # sees all
        tol = M.bound(ref, mean, score, n + rows, d, pool.torch_dtype)
        assert ((out[mine].double() - ref).abs() <= tol).all(), s


# ---------------------------------------------------------------------------
# Refused entries among good ones
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,rows", [(20, 1), (20, 7), (20, 130), (500, 1), (500, 33)])
def test_refused_entries_are_zeroed_and_the_others_right(dtype, n, rows):
    """Every third entry without room, every seventh of a sequence that does not exist, some padding:
    on both sides of 32 entries, with one row tile and several."""
    nq, nkv, d = 4, 2, 64
    pool, model = make_pool(dtype, 1, nq, nkv, d, 60, 16, 4, 300)
    lens = [100, 0, 37, 64]
    pool.reserve(i32([n + rows for n in lens[:3]] + [64]))
    pool.advance(i32(lens))
    model.reserve([0, 1, 2], [n + rows for n in lens[:3]])
    seqs = [3 if i % 3 == 0 else 4 + i if i % 7 == 0 else -1 if i % 11 == 0 else i % 3 for i in range(n)]
    total = n * rows + 5
    q = torch.randn(total, nq, d, device="cuda").to(pool.torch_dtype)
    out = torch.full_like(q, 7.0)
    pool.attention(0, q, out, i32(seqs), i32([i * rows for i in range(n)]), i32([rows] * n), rows)
    assert pool.status() in (-1, -5)
    assert (out[n * rows:] == 7).all()
    for i, s in enumerate(seqs):
        mine = slice(i * rows, (i + 1) * rows)
        if s == -1:
            assert (out[mine] == 7).all(), i
        elif s >= 3:
            assert (out[mine] == 0).all(), i
        elif i < 40:
            kv = model.rows_of(s, lens[s] + rows)[0]
            ref, mean, score = M.attention(q[mine], kv[0], kv[1], range(lens[s], lens[s] + rows), True, 0, 0)
            tol = M.bound(ref, mean, score, lens[s] + rows, d, pool.torch_dtype)
            assert ((out[mine].double() - ref).abs() <= tol).all(), i


def test_a_refused_prompt_does_not_hold_up_the_call():
    """A chunk of 2048 rows without room beside a block: its 16 MB of zeros are written by the whole
    device (a few microseconds; one thread took milliseconds)."""
    pool, _ = make_pool("bf16", 1, 32, 8, 128, 40, 64, 2, 2200)
    pool.reserve(i32([100]), i32([0]))
    q = torch.randn(2048 + 16, 32, 128, device="cuda").bfloat16()
    out = torch.empty_like(q)
    args = (i32([1, 0]), i32([0, 2048]), i32([2048, 16]), 2048)
    times = []
    for _ in range(8):
        out.fill_(7.0)
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        pool.attention(0, q, out, *args)
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b) * 1e3)
    assert pool.status() == -5
    assert (out[:2048] == 0).all() and torch.isfinite(out[2048:].float()).all() and (out[2048:] != 7).any()
    print(sorted(times))
    assert min(times) < 300, times


# ---------------------------------------------------------------------------
# Accuracy of few rows
# ---------------------------------------------------------------------------

def two_terms_bound(out, mean, score, n, d):
    """As M.bound for bf16, with weights kept in two bf16 terms: the first is off by half a step, 2^-8 of
    the weight, what is left (exact in fp32) is rounded by 2^-8 of that: 2^-16."""
    f32 = 2 * (2 * d * 2.0 ** -23 * score) + 2.0 ** -20 + 2 * n * 2.0 ** -23
    e = (2.0 ** -16 + f32) * mean
    return e + 2.0 ** -8 * (out.abs() + e) + 1e-30


def one_term(q, k, v):
    """What one bf16 term gives: o = sum R(2^(t - b)) v / sum 2^(t - b) in 64 bits, b the integer below
    the row's maximum (rows q [1, nq, d] that see all of k, v [nkv, n, d])."""
    q, k, v = q.double(), k.double(), v.double()
    k, v = (x.repeat_interleave(q.shape[1] // x.shape[0], 0) for x in (k, v))
    t = (k @ q[0, :, :, None])[..., 0] / math.sqrt(q.shape[2]) * math.log2(math.e)
    w = torch.exp2(t - t.amax(1, keepdim=True).floor())
    return (((w.float().bfloat16().double()[..., None] * v).sum(1)) / w.sum(1, keepdim=True))[None]


@pytest.mark.parametrize("nq,nkv,d,page", [(32, 8, 128, 64), (8, 8, 64, 16), (16, 1, 64, 16), (12, 2, 128, 32)])
def test_few_rows_keep_16_bits_of_the_weights(nq, nkv, d, page):
    """Contexts of 1 to 7 positions, scores near 0: weighted sums of few values that nearly cancel, where
    a weight of 8 bits shows before the result's own rounding does."""
    lens = [1, 2, 3, 4, 5, 6, 7, 3] * 8
    pool, model = make_pool("bf16", 1, nq, nkv, d, len(lens), page, len(lens), 16, seed=d)
    pool.reserve(i32([n + 1 for n in lens]))
    pool.advance(i32(lens))
    model.reserve(list(range(len(lens))), [n + 1 for n in lens])
    g = torch.Generator(device="cuda")
    g.manual_seed(page)
    q = (torch.randn(len(lens), nq, d, device="cuda", generator=g) * 0.25).bfloat16()
    out = pool.attention(0, q)
    assert pool.status() == 0
    shows = 0
    for s, n in enumerate(lens):
        kv = model.rows_of(s, n + 1)[0]
        ref, mean, score = M.attention(q[s:s + 1], kv[0], kv[1], [n], True, 0, 0)
        tol = two_terms_bound(ref, mean, score, n + 1, d)
        assert ((out[s:s + 1].double() - ref).abs() <= tol).all(), s
        # the result of one term, rounded or not, is outside in many places
        one = one_term(q[s:s + 1], kv[0], kv[1])
        shows += ((one - ref).abs() > tol).sum().item()
    assert shows > 100
    print(shows, out.numel())
