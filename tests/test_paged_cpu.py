"""Host side of the paged pool, without a GPU: exported symbols, configurations that are
refused, null arguments, and the plain model of the page operations on worked cases."""
import os
import re

import pytest
import torch

from block_diffusion_speculative_03_b200 import build, dflash as D
from block_diffusion_speculative_03_b200.paging import PagePool
from tests import paged_model as M

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    build.build()
    return D.lib()


def test_exports_every_declared_symbol(lib):
    src = open(os.path.join(ROOT, "include", "dflash_paged.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = set(re.findall(r"\b(dflash_\w+)\s*\(", src))
    assert names == set(D.paged_symbols())
    for n in names:
        assert hasattr(lib, n), n


def cfg(**kw):
    c = D.dflash_pool_config(n_layers=5, n_q_heads=32, n_kv_heads=8, head_dim=128, dtype=D.DFLASH_BF16, n_pages=100,
                             page_size=64, max_seqs=8, max_len=4096)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def test_pool_bytes_count_the_slab(lib):
    a, b = (D.dflash_pool_bytes(cfg(n_pages=n)) for n in (100, 200))
    page = 5 * 2 * 8 * 64 * 128 * 2
    assert 100 * page <= b - a <= 100 * page + 100 * 48 + 4096
    assert D.dflash_pool_bytes(cfg(dtype=D.DFLASH_F32)) > a + 100 * page - 4096


@pytest.mark.parametrize("kw,status", [
    (dict(n_layers=0), -1), (dict(n_q_heads=0), -1), (dict(n_kv_heads=0), -1), (dict(n_q_heads=30), -1),
    (dict(dtype=2), -1), (dict(n_pages=0), -1), (dict(max_seqs=0), -1), (dict(max_seqs=1025), -1),
    (dict(max_len=0), -1), (dict(max_len=(1 << 30) + 1), -1),
    (dict(head_dim=96), -2), (dict(head_dim=256), -2), (dict(page_size=8), -2), (dict(page_size=48), -2),
    (dict(page_size=512), -2), (dict(n_q_heads=8 * 129), -2),
    (dict(n_pages=(1 << 31) - 1), -2), (dict(n_layers=1 << 28), -2),
    (dict(max_seqs=1024, max_len=1 << 30, page_size=16), -2),
])
def test_configurations_that_are_refused(lib, kw, status):
    assert D.dflash_pool_bytes(cfg(**kw), check=False) == status


def test_null_arguments(lib):
    assert lib.dflash_pool_bytes(None, None) == -1
    one = 4096
    assert D.dflash_pool_init(cfg(), None, 1 << 40, check=False) == -1
    assert D.dflash_pool_init(cfg(), 1000, 1 << 40, check=False) == -1        # not 1024-byte aligned
    assert D.dflash_pool_init(cfg(), 1024, 100, check=False) == -4            # too small
    assert lib.dflash_pool_get_info(None, None) == -1
    assert lib.dflash_pool_status(None, None) == -1
    assert lib.dflash_pool_launch_count(None) == 0
    assert lib.dflash_pool_set_tables(None, one, one, None) == -1
    assert lib.dflash_pages_reserve(None, one, one, 1, None) == -1
    assert lib.dflash_pages_fork(None, one, one, 1, 0, None) == -1
    assert lib.dflash_pages_free(None, one, one, 1, None) == -1
    assert lib.dflash_pages_compact(None, one, None) == -1
    assert lib.dflash_pages_write(None, None, 1, 0, one, one, 64, None, None, 1, 1, None) == -1
    assert lib.dflash_pages_advance(None, None, None, 1, None) == -1
    assert lib.dflash_pages_store(None, None, None, None, 1, None) == -1
    assert lib.dflash_pages_load(None, None, None, None, 1, None) == -1
    assert lib.dflash_paged_attention(None, None, 1, 0, one, 64, None, None, 1, 1, 1, 0, 0, one, None) == -1
    assert lib.dflash_cache_set_window(None, 1, 0, one, 1 << 30, None) == -1
    assert lib.dflash_window_scratch_bytes(None) == -1
    assert D.dflash_window_scratch_bytes() > 0
    lib.dflash_pool_release(None)


def test_a_pool_wants_a_gpu():
    with pytest.raises(ValueError):
        PagePool(1, 4, 2, 64, "bf16", n_pages=4, page_size=16, max_seqs=2, max_len=64, device="cpu")
    with pytest.raises(KeyError):
        PagePool(1, 4, 2, 64, "fp16", n_pages=4, page_size=16, max_seqs=2, max_len=64, device="cuda:0")


def model(pages=10, page=4, seqs=4, max_len=20):
    rows = torch.arange(pages * page, dtype=torch.float32).view(pages, 1, 1, 1, page, 1)
    return M.PoolModel(pages, page, seqs, max_len, rows.expand(pages, 1, 2, 1, page, 1))


def test_model_shares_and_copies():
    m = model()
    m.reserve([0], [6])
    m.advance([0], [6])
    m.fork([0, 0], [1, 2])
    assert m.tab[:3] == [[0, 1]] * 3 and m.refs()[:2] == [3, 3]
    m.reserve([1, 0], [1, 1])                  # two of three holders write: both copy
    assert m.tab[:3] == [[0, 3], [0, 2], [0, 1]]
    assert m.slab[2, 0, 0, 0, :2, 0].tolist() == [4, 5] and m.slab[2, 0, 0, 0, 2:, 0].tolist() == [10, 11]
    m.free([0, 2])
    assert m.refs() == [1, 0, 1, 0, 0, 0, 0, 0, 0, 0]
    assert m.compact() == 2 and m.tab[1] == [0, 1]
    assert m.slab[1, 0, 0, 0, :, 0].tolist() == [4, 5, 10, 11]


def test_model_attention_is_a_softmax_over_what_a_row_sees():
    torch.manual_seed(0)
    q, k, v = torch.randn(2, 2, 4), torch.randn(1, 5, 4), torch.randn(1, 5, 4)
    out, mean, score = M.attention(q, k, v, [3, 4], True, 2, 1)
    for r, seen in ((0, [0, 2, 3]), (1, [0, 3, 4])):
        for h in range(2):
            w = torch.softmax((k[0, seen].double() @ q[r, h].double()) / 2.0, 0)
            assert torch.allclose(out[r, h], w @ v[0, seen].double())
    # a wrong window misses the result by far more than the bound allows
    other, _, _ = M.attention(q, k, v, [3, 4], True, 3, 1)
    assert ((other - out).abs() > M.bound(out, mean, score, 5, 4, torch.bfloat16)).any()
