"""Paged-cache operators at the ends of what their arguments allow: values that are no numbers, scales, rows
and lengths out of range, modes of torch that a call has to notice."""

import pytest
import torch

from rolling_kv_cache_b200 import paged

from paged_util import Batch, randn

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(autouse=True)
def _status_stays_clear():
    yield
    paged.device_status()


def _wide(bt):
    """A table with room for 2^18 tokens: the batch is cut evenly over the GPU."""
    table = torch.full((len(bt.lens), 2 ** 18 // bt.page), -7, dtype=torch.int32, device="cuda")
    table[:, :bt.page_table.shape[1]] = bt.page_table
    return table


def _prefix(bt, n, pages=None):
    """n tokens of a prefix in the batch's spare pages, or over and over in the first `pages` of them."""
    count = (n + bt.page - 1) // bt.page
    have = torch.tensor(bt.free[:pages or count], dtype=torch.int32, device="cuda")
    table = have.repeat((count + len(have) - 1) // len(have))[:count].contiguous()
    for pool in (bt.k_pages, bt.v_pages):
        pool[have.long()] = randn(bt.gen, len(have), bt.hk, bt.page, bt.d, dtype=bt.dtype)
    return table, n


def _attend(bt, max_q, prefix=None, **kw):
    if prefix is None:
        return paged.paged_attention(*bt.args(), max_q=max_q, return_lse=True, **kw)
    return paged.prefix_attention(*bt.args()[:3], *prefix, *bt.args()[3:], max_q=max_q, return_lse=True, **kw)


@pytest.mark.parametrize("n", [1, 2, 17, 33, 65, 129, 1025])
@pytest.mark.parametrize("path", ["clusters", "cut", "many"])
@pytest.mark.parametrize("what", ["query", "last key"])
def test_a_row_whose_scores_are_nan_is_nan(n, path, what):
    """Also where a block, a warp or a part of its unit sees no other score: out and lse."""
    bt = Batch(101, [(1, n), (1, 70), (1, 3)], 4, 2, 64, 16)
    if path == "cut":
        bt.page_table = _wide(bt)
    max_q = 17 if path == "many" else 1
    want, wl = _attend(bt, max_q)
    hit = torch.zeros(3, 4, dtype=torch.bool, device="cuda")
    if what == "query":
        bt.q[0, 1, 7] = NAN
        hit[0, 1] = True
    else:
        bt.k_pages[int(bt.page_table[0, (n - 1) // 16]), 1, (n - 1) % 16, 5] = NAN
        hit[0, 2:] = True
    o, lse = _attend(bt, max_q)
    assert bool(o[hit].isnan().all()) and bool(lse.T[hit].isnan().all())
    assert torch.equal(o[~hit], want[~hit]) and torch.equal(lse.T[~hit], wl.T[~hit])


PREFIXES = [  # q heads, kv heads, d, page; lengths behind the first sequence; prefix, max_q
    (2, 2, 64, 16, [(1, 30)], 200, 1),           # clusters
    (12, 12, 128, 64, [(1, 40)] * 20, 435, 1),   # two passes and the join
    (12, 12, 64, 16, [(20, 40)] * 70, 500, 20),  # two passes and the merge
    (4, 2, 128, 32, [(300, 300)], 257, 300),     # walked
]


@pytest.mark.parametrize("case", PREFIXES, ids=["clusters", "join", "merge", "walked"])
def test_a_nan_key_of_a_sequence_behind_a_prefix(case):
    hq, hk, d, page, rest, n, max_q = case
    bt = Batch(102, [(1, 1)] + rest, hq, hk, d, page, spare=(n + page - 1) // page + 1)
    prefix = _prefix(bt, n)
    want, wl = _attend(bt, max_q, prefix)
    bt.k_pages[int(bt.page_table[0, 0]), 1, 0, 3] = NAN
    hit = torch.zeros(bt.n_tok, hq, dtype=torch.bool, device="cuda")
    hit[0, hq // hk:2 * (hq // hk)] = True
    o, lse = _attend(bt, max_q, prefix)
    assert bool(o[hit].isnan().all()) and bool(lse.T[hit].isnan().all())
    assert torch.equal(o[~hit], want[~hit]) and torch.equal(lse.T[~hit], wl.T[~hit])


@pytest.mark.parametrize("case", PREFIXES, ids=["clusters", "join", "merge", "walked"])
def test_a_nan_key_of_the_prefix_reaches_sequences_without_tokens(case):
    hq, hk, d, page, rest, n, max_q = case
    bt = Batch(103, [(1, 0)] + rest[:-1] + [(rest[-1][0], 0)], hq, hk, d, page, spare=(n + page - 1) // page + 1)
    prefix = _prefix(bt, n)
    want, wl = _attend(bt, max_q, prefix)
    assert bool(torch.isfinite(want).all()) and bool(torch.isfinite(wl).all())
    bt.k_pages[int(prefix[0][-1]), 1, (n - 1) % page, 3] = NAN
    hit = torch.zeros(bt.n_tok, hq, dtype=torch.bool, device="cuda")
    hit[:, hq // hk:2 * (hq // hk)] = True
    o, lse = _attend(bt, max_q, prefix)
    assert bool(o[hit].isnan().all()) and bool(lse.T[hit].isnan().all())
    assert torch.equal(o[~hit], want[~hit]) and torch.equal(lse.T[~hit], wl.T[~hit])
