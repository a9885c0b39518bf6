"""Arithmetic of the paged attention's plan on the host: room for the joins, and which shares of a
call go on with another item behind the end of a long one."""
import pytest

from block_diffusion_speculative_03_b200 import build, dflash as D

# The cases of tests/test_gpu_paged_joins.py: query heads, kv heads, head_dim, positions of each sequence.
LONG = [(8, 8, 128, [16384]), (8, 8, 128, [32768]), (32, 8, 128, [32768]), (16, 8, 64, [16384]),
        (64, 8, 64, [32768]), (16, 4, 128, [32768, 32768]), (32, 8, 128, [15976, 15976])]


@pytest.fixture(scope="module")
def lib():
    build.build()
    return D.lib()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", range(1, 17))
def test_joins_keep_to_their_room(lib, d, rows):
    pairs, pairs_fit, floats, floats_fit = D.dflash_diag_paged_decode_join(d, rows)
    # by hand: eight warps with 16 rows each; teams of rows * d / 4 of the 256 threads, at most eight
    team = rows * d // 4
    assert pairs == max(128, min(8, 256 // team) * team) <= 256
    assert pairs <= pairs_fit and floats <= floats_fit


def test_shapes_without_a_join_are_refused(lib):
    for d, rows in ((96, 1), (64, 0), (128, 17), (64, -1)):
        with pytest.raises(D.DflashError):
            D.dflash_diag_paged_decode_join(d, rows)


def end_holders(lens, nkv, ctas=148, overhead=4, least=3):
    """(units of a long item's end, tiles of the next item, share) of the shares that hold both; long: in
    nine shares and more."""
    items = [(n + 1 + 63) // 64 + overhead for n in lens for _ in range(nkv)]
    starts = [sum(items[:i]) for i in range(len(items) + 1)]
    units = starts[-1]
    shares = min(ctas, units // least)
    begin = [c * units // shares for c in range(shares + 1)]
    owner = lambda u: next(c for c in range(shares) if begin[c] <= u < begin[c + 1])
    out = []
    for i in range(len(items) - 1):
        first, last = owner(starts[i] + overhead), owner(starts[i + 1] - 1)
        left = begin[last + 1] - starts[i + 1] - overhead
        if last - first >= 8 and left > 0:
            out.append((starts[i + 1] - max(begin[last], starts[i]), left, last))
    return out


@pytest.mark.parametrize("nq,nkv,d,lens", LONG)
def test_long_cases_have_shares_that_go_on(nq, nkv, d, lens):
    assert end_holders(lens, nkv)


def test_share_by_hand():
    # one sequence of 32769 keys, 8 kv heads: 8 items of 513 + 4 units over 148 shares of 27 or 28
    assert end_holders([32768], 8)[0] == (14, 9, 18)
    assert end_holders([2047], 8) == []                 # shares end where items do
