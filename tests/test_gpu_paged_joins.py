"""Long joins of the paged attention of few rows while other work holds the device: whichever share
of an item arrives last, the ones that go on with the next item read their own plan."""
import pytest
import torch

from tests import paged_model as M
from tests.test_gpu_paged import i32, make_pool
from tests.test_paged_plan_cpu import LONG, end_holders

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nq,nkv,d,lens", LONG)
def test_long_joins_beside_other_work(nq, nkv, d, lens):
    page, n = 64, len(lens)
    pool, _ = make_pool("bf16", 1, nq, nkv, d, sum(M.ceil_div(x + 1, page) for x in lens), page, n, max(lens) + 1)
    pool.reserve(i32([x + 1 for x in lens]))
    pool.advance(i32(lens))
    torch.manual_seed(len(lens) + d)
    q = torch.randn(n, nq, d, device="cuda").bfloat16()
    want = pool.attention(0, q).clone()
    slab = pool.slab()
    for s, x in enumerate(lens):
        kv = slab[pool.table[s, :M.ceil_div(x + 1, page)].long(), 0].permute(1, 2, 0, 3, 4).flatten(2, 3)[:, :, :x + 1]
        ref, mean, score = M.attention(q[s:s + 1], kv[0], kv[1], [x], True, 0, 0)
        tol = M.bound(ref, mean, score, x + 1, d, torch.bfloat16)
        assert ((want[s:s + 1].double() - ref).abs() <= tol).all()

    # another pool's blocks and tokens on another stream take the SMs away from some shares for a while
    other, _ = make_pool("bf16", 1, 16, 4, 128, 300, 64, 4, 4200, seed=1)
    other.reserve(i32([4100, 3000, 900, 64]))
    other.advance(i32([4080, 2980, 880, 40]))
    start, count = i32([0, 16, 32, 48]), i32([16] * 4)
    qb = torch.randn(64, 16, 128, device="cuda").bfloat16()
    ob = torch.empty_like(qb)
    beside = torch.cuda.Stream()
    beside.wait_stream(torch.cuda.current_stream())
    out, off = torch.empty_like(want), torch.zeros((), dtype=torch.int64, device="cuda")
    for k in range(200):
        with torch.cuda.stream(beside):
            other.attention(0, qb, ob, None, start, count, 16)
            if k % 3 == 0:
                other.attention(0, qb[:4], ob[:4])
        out.fill_(7.0)
        pool.attention(0, q, out)
        off += (out.view(torch.int16) != want.view(torch.int16)).sum()
    torch.cuda.synchronize()
    assert off.item() == 0
    # and the counts of arrivals are as a call finds them: alone again, the same bits
    out.fill_(7.0)
    assert torch.equal(pool.attention(0, q, out), want)
    assert pool.status() == 0 and other.status() == 0


@pytest.mark.parametrize("nq,nkv,d,lens", LONG)
def test_last_to_arrive_goes_on_with_the_next_item(nq, nkv, d, lens):
    """Single shares that start late.  Blocks start in order, so work that holds k SMs when a call
    starts makes the last k of its shares late: with k chosen so that the first of them holds the end of
    an item and the start of the next, that one is the last of its item to arrive, and goes on."""
    page, n = 64, len(lens)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    pool, _ = make_pool("bf16", 1, nq, nkv, d, sum(M.ceil_div(x + 1, page) for x in lens), page, n, max(lens) + 1)
    pool.reserve(i32([x + 1 for x in lens]))
    pool.advance(i32(lens))
    torch.manual_seed(len(lens) + d)
    q = torch.randn(n, nq, d, device="cuda").bfloat16()
    want = pool.attention(0, q).clone()
    # a softmax over k long rows holds k SMs, a block of 1024 threads on each
    rows = torch.randn(sms, 200000, device="cuda")
    held = torch.empty_like(rows)
    out = torch.empty_like(want)
    beside = torch.cuda.Stream()
    for _, left, share in end_holders(lens, nkv, sms):
        k = sms - share
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            beside.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(beside):
                torch.softmax(rows[:k], 1, out=held[:k])
            out.fill_(7.0)
            pool.attention(0, q, out)
            torch.cuda.current_stream().wait_stream(beside)
        for _ in range(10):
            graph.replay()
            assert torch.equal(out, want), (k, left)
    assert torch.equal(pool.attention(0, q, out), want)
    assert pool.status() == 0


@pytest.mark.parametrize("dtype,nq,nkv,d,lens,rows,causal,window", [
    ("bf16", 8, 1, 64, [9000], 1, True, 0), ("bf16", 16, 4, 128, [8000, 40, 5000], 3, False, 0),
    ("bf16", 32, 8, 128, [8000, 100], 16, False, 2000), ("bf16", 8, 2, 128, [4000, 3000], 8, True, 0),
    ("bf16", 16, 2, 128, [1500], 300, True, 0), ("f32", 8, 8, 64, [3000], 1, True, 0),
    ("f32", 4, 2, 128, [2500, 900], 8, False, 500)])
def test_late_shares_change_no_bits(dtype, nq, nkv, d, lens, rows, causal, window):
    """Every kernel with its last blocks held up for a while, by many or few: the same bits."""
    page, n = 64, len(lens)
    pool, _ = make_pool(dtype, 1, nq, nkv, d, sum(M.ceil_div(x + rows, page) for x in lens), page, n, max(lens) + rows)
    pool.reserve(i32([x + rows for x in lens]))
    pool.advance(i32(lens))
    torch.manual_seed(rows)
    q = torch.randn(n * rows, nq, d, device="cuda").to(pool.torch_dtype)
    args = (i32(list(range(n))), i32([i * rows for i in range(n)]), i32([rows] * n), rows, causal, window, 4)
    want = pool.attention(0, q, None, *args).clone()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    x = torch.randn(sms, 200000, device="cuda")
    held, out, beside = torch.empty_like(x), torch.empty_like(want), torch.cuda.Stream()
    for k in range(3, sms, 8):
        long = (50000, 200000)[k // 8 % 2]
        a, b = x[:k, :long].contiguous(), held.view(-1)[:k * long].view(k, long)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            beside.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(beside):
                torch.softmax(a, 1, out=b)
            out.fill_(7.0)
            pool.attention(0, q, out, *args)
            torch.cuda.current_stream().wait_stream(beside)
        for _ in range(3):
            out.fill_(0.0)
            graph.replay()
            assert torch.equal(out, want), k
    assert pool.status() == 0
