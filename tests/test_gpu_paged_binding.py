"""The paged pool through the binding's C names, with pointers, beside the same calls of a PagePool."""
import pytest
import torch

from block_diffusion_speculative_03_b200 import dflash as D
from block_diffusion_speculative_03_b200 import inputs as I
from tests.test_gpu_paged import i32
from tests.test_gpu_paged_use import drafter

pytestmark = pytest.mark.gpu


def test_a_step_through_the_c_names():
    w = I.Workload("names", 256, 2, 4, 2, 64, 512, 1000, 1, 256, 1e6, 1e-6, "bf16", batch=2, gamma=4, context=[1, 1],
                   mask_id=999, seed=5)
    dr = drafter(w)
    cache = dr.new_cache(2, 200)
    torch.manual_seed(0)
    cache.slab().copy_(torch.randn(cache.slab().shape, device="cuda"))
    cache.set_len(torch.tensor([70, 33], dtype=torch.int32))
    one, two = (dr.new_pool(40, 16, 4, 200) for _ in range(2))
    back = [dr.new_cache(2, 200) for _ in range(2)]
    for c in (one, two):
        c.slab().zero_()
    for c in back:
        c.slab().zero_()
    q, k, v = (torch.randn(3, h, 64, device="cuda").bfloat16() for h in (4, 2, 2))
    oa, ob = torch.zeros_like(q), torch.zeros_like(q)
    ua, ub = i32([0]), i32([0])
    grow, ids, ones, src, dst = i32([80, 40]), i32([0, 1]), i32([1, 1, 1]), i32([0, 1]), i32([2, 3])
    listed, keep, start = i32([0, 1, 2]), i32([21]), i32([0, 1, 2])
    h, st, P = two.handle, torch.cuda.current_stream().cuda_stream, torch.Tensor.data_ptr

    one.reserve(grow, ids)
    D.dflash_pages_reserve(h, P(ids), P(grow), 2, st)
    one.store(cache, ids)
    D.dflash_pages_store(h, P(ids), cache.handle, None, 2, st)
    one.fork(src, dst)
    D.dflash_pages_fork(h, P(src), P(dst), 2, False, st)
    one.reserve(ones, listed)
    D.dflash_pages_reserve(h, P(listed), P(ones), 3, st)
    one.write(1, k, v, listed, start, ones)
    D.dflash_pages_write(h, P(listed), 3, 1, P(k), P(v), 128, P(start), P(ones), 3, 3, st)
    one.attention(1, q, oa, listed, start, ones, 1, True, 50, 2)
    D.dflash_paged_attention(h, P(listed), 3, 1, P(q), 256, P(start), P(ones), 3, 1, True, 50, 2, P(ob), st)
    one.advance(None, listed)
    D.dflash_pages_advance(h, P(listed), None, 3, st)
    one.free(i32([3]), keep)
    three = i32([3])
    D.dflash_pages_free(h, P(three), P(keep), 1, st)
    one.free(ids[:1])
    D.dflash_pages_free(h, P(ids), None, 1, st)
    one.compact(ua)
    D.dflash_pages_compact(h, P(ub), st)
    one.load(back[0], listed[1:])
    D.dflash_pages_load(h, P(listed[1:]), back[1].handle, None, 2, st)
    one.set_tables(one.len, one.table)
    D.dflash_pool_set_tables(h, P(two.len), P(two.table), st)

    assert one.status() == 0 and D.dflash_pool_status(h, st) == 0
    assert one.launch_count() == D.dflash_pool_launch_count(h) > 0
    assert (oa != 0).any() and torch.equal(oa, ob) and ua.item() == ub.item() > 0
    assert one.len.tolist() == two.len.tolist() == [0, 34, 71, 21]
    assert torch.equal(one.table, two.table) and torch.equal(one.refs, two.refs)
    assert torch.equal(one.slab(), two.slab())
    assert back[0].len.tolist() == back[1].len.tolist() == [34, 71]
    assert torch.equal(back[0].slab(), back[1].slab())
    # statuses come back as exceptions, or as values when asked for
    for call in (lambda **kw: D.dflash_pages_reserve(h, None, None, 1, st, **kw),
                 lambda **kw: D.dflash_pages_fork(h, None, P(dst), 1, True, st, **kw),
                 lambda **kw: D.dflash_pages_free(h, None, None, -1, st, **kw),
                 lambda **kw: D.dflash_pages_advance(h, None, None, 5, st, **kw),
                 lambda **kw: D.dflash_pages_compact(h, None, st, **kw),
                 lambda **kw: D.dflash_pages_write(h, None, 1, 2, P(k), P(v), 128, None, None, 1, 1, st, **kw),
                 lambda **kw: D.dflash_pages_store(h, None, None, None, 1, st, **kw),
                 lambda **kw: D.dflash_pages_load(h, None, None, None, 1, st, **kw),
                 lambda **kw: D.dflash_paged_attention(h, None, 1, 0, None, 256, None, None, 1, 1, True, 0, 0, P(ob), st, **kw),
                 lambda **kw: D.dflash_pool_set_tables(h, None, P(two.table), st, **kw)):
        assert call(check=False) == -1
        with pytest.raises(D.DflashError):
            call()
    assert D.dflash_pool_status(h, st) == 0
