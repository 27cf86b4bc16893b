"""Paged-cache operators at the ends of what their arguments allow: values that are no numbers, scales, rows
and lengths out of range, modes of torch that a call has to notice."""
import math
import os
import subprocess
import sys
import threading

import pytest
import torch

from rolling_kv_cache_b200 import binding as B
from rolling_kv_cache_b200 import paged

from paged_util import F64, UNIT, Batch, assert_attend, assert_turned, generator, randn, visible

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
NAN = float("nan")


@pytest.fixture(autouse=True)
def _status_stays_clear():
    yield
    paged.device_status()


def _reported():
    with pytest.raises(B.RcError) as e:
        paged.device_status()
    assert e.value.status == B.RC_ERANGE


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


def _one_axis(bt):
    """Queries along the first axis, keys whose first element is a multiple of 1/16 below 8: every score is exact in
    fp32, and the largest comes up several times."""
    bt.q.zero_()
    bt.q[..., 0] = torch.randint(1, 3, bt.q.shape[:2], generator=bt.gen, device="cuda").to(bt.dtype)
    bt.q[..., 0] *= torch.randint(0, 2, bt.q.shape[:2], generator=bt.gen, device="cuda").to(bt.dtype) * 2 - 1
    first = torch.randint(-127, 128, bt.k_pages.shape[:3], generator=bt.gen, device="cuda") / 16
    bt.k_pages[..., 0] = torch.where(bt.k_pages[..., 0].isnan(), NAN, first.float()).to(bt.dtype)


def _assert_exact_scores(got, bt, scale, prefix=None):
    """Against the softmax in 64 bits. Scores and their differences are exact, so a weight's exponent, t nats below
    the row's largest, is off by at most t 2^-22 (its factor and its product are rounded, once more where the stale maximum moved; the
    sum of all the distances is at most t and 8 / log2(e) behind and before it). The exponential is allowed 2^-13, the weight's
    rounding to the type UNIT (fp16: 2^-25 at least), sums of m terms in fp32 m 2^-23, the output's rounding UNIT."""
    out, lse = got
    u, dt = UNIT[bt.dtype], bt.dtype
    sc = float(torch.tensor(scale, dtype=F32))
    for b, (a, n) in enumerate(bt.lens):
        if not a:
            continue
        seen = visible(n - a, a, n, 1, 0, 0)
        j = torch.arange(n, device="cuda")
        k, v = (bt.rows(x, bt.page_table[b], j) for x in (bt.k_pages, bt.v_pages))
        if prefix is not None:
            i = torch.arange(prefix[1], device="cuda")
            k, v = (torch.cat((bt.rows(p, prefix[0], i), x)) for p, x in ((bt.k_pages, k), (bt.v_pages, v)))
            seen = torch.cat((seen.new_ones(a, prefix[1]), seen), 1)
        r = slice(bt.cu[b], bt.cu[b + 1])
        for h in range(bt.hq):
            kh, vh = k[:, h // (bt.hq // bt.hk)], v[:, h // (bt.hq // bt.hk)]
            x = (bt.q[r, h].to(F64) @ kh.T * sc).masked_fill(~seen, -math.inf)
            t = (x.amax(1, keepdim=True) - x).masked_fill(~seen, 0)
            w = torch.softmax(x, -1)
            m = seen.sum(1, keepdim=True)
            rel = w * (u + 2.0 ** -13 + (m + 16) * 2.0 ** -23 + t * 2.0 ** -22)
            rel = rel + (seen * 2.0 ** -25 if dt == F16 else 0)
            o = w @ vh
            tol = rel @ vh.abs() + rel.sum(1, keepdim=True) * o.abs()
            tol = tol + u * (o.abs() + tol) + (2.0 ** -25 if dt == F16 else 0)
            err = (out[r, h].to(F64) - o).abs()
            assert bool((err <= tol).all()), (b, h, float(err.max()))
            ls = torch.logsumexp(x, -1)
            if float(ls.abs().max()) > 2e38:
                continue
            ltol = 2.0 ** -21 * (ls.abs() + 1) + rel.sum(1)
            assert bool(((lse[h, r].to(F64) - ls).abs() <= ltol).all()), (b, h)


@pytest.mark.parametrize("scale", [1e2, 1e4, 1e6, 1e7, 1e9, 1e30])
@pytest.mark.parametrize("path", ["clusters", "cut", "many"])
@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F16, 64)])
def test_large_scales_leave_the_largest_scores_their_weight(scale, path, dtype, d):
    a = 30 if path == "many" else 2
    bt = Batch(104, [(a, 1000), (a, 300), (1, 5), (a, 2500)], 4, 2, d, 16, dtype)
    if path == "cut":
        bt.page_table = _wide(bt)
    _one_axis(bt)
    _assert_exact_scores(_attend(bt, a, scale=scale), bt, scale)


@pytest.mark.parametrize("scale", [1e4, 1e9, 1e30])
@pytest.mark.parametrize("case", PREFIXES, ids=["clusters", "join", "merge", "walked"])
def test_large_scales_over_a_prefix(case, scale):
    hq, hk, d, page, rest, n, max_q = case
    bt = Batch(105, [(1, 9)] + rest, hq, hk, d, page, spare=(n + page - 1) // page + 1)
    prefix = _prefix(bt, n)
    _one_axis(bt)
    _assert_exact_scores(_attend(bt, max_q, prefix, scale=scale), bt, scale, prefix)


@pytest.mark.parametrize("path", ["clusters", "cut", "many"])
@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F16, 64)])
def test_scores_that_pass_fp32_with_the_scale_still_weigh(path, dtype, d):
    """Their log-sum-exp is infinite in fp32; the weights go by differences of the scores."""
    a = 30 if path == "many" else 2
    bt = Batch(117, [(a, 1000), (a, 300), (a, 40)], 4, 2, d, 16, dtype)
    if path == "cut":
        bt.page_table = _wide(bt)
    _one_axis(bt)
    bt.q[..., 0] *= 2 ** 13
    bt.k_pages[..., 0] *= 2 ** 12
    o, lse = _attend(bt, a, scale=1e30)
    _assert_exact_scores((o, lse), bt, 1e30)
    # 1000 keys of 255 values: a largest score above 7.5 2^25, with the scale 3.6e38 to the base 2
    assert bool(torch.isinf(lse[:, a - 1]).all()) and not bool(lse.isnan().any())


@pytest.mark.parametrize("path", ["clusters", "cut", "many"])
def test_a_score_of_minus_infinity_has_no_weight(path):
    a = 30 if path == "many" else 2
    bt = Batch(118, [(a, 500), (a, 90)], 4, 2, 64, 16)
    if path == "cut":
        bt.page_table = _wide(bt)
    bt.q[..., 0] = 1
    at = [(int(bt.page_table[0, j // 16]), j % 16) for j in (0, 17, 63, 400)]
    got = []
    for value in (-3e38, -math.inf):
        for page, row in at:
            bt.k_pages[page, :, row, 0] = value
        got.append(_attend(bt, a))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert bool(torch.isfinite(got[1][0]).all()) and bool(torch.isfinite(got[1][1]).all())


@pytest.mark.parametrize("path", ["clusters", "cut", "many"])
@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F16, 64)])
def test_maxima_that_grow_past_the_border_of_steep_rows(path, dtype, d):
    """Scores of 90852 + i / 64, exact in fp32, i growing along the sequence: the largest passes 2^24 in units of the
    exponential's base in steps of 2.9, so that sums from before and behind that border meet."""
    a = 30 if path == "many" else 2
    bt = Batch(116, [(a, 2500), (a, 700)], 4, 2, d, 16, dtype)
    if path == "cut":
        bt.page_table = _wide(bt)
    bt.q.zero_()
    bt.q[..., 0], bt.q[..., 1], bt.q[..., 2] = 256, 1, 1
    for b, (_, n) in enumerate(bt.lens):
        j = torch.arange(n, device="cuda")
        page, row = bt.page_table[b][j // 16].long(), j % 16
        for i, x in enumerate((354.0, 228.0, (j * 26 // n / 64)[:, None])):
            bt.k_pages[page, :, row, i] = (torch.zeros(n, 2, device="cuda") + x).to(dtype)
    _assert_exact_scores(_attend(bt, a, scale=128.0), bt, 128.0)


PATHS = ["clusters", "cut", "many", "prefix clusters", "prefix join", "prefix walked", "prefix merge"]


def _path(bt, path):
    """(table, max_q, prefix) that take the path for a batch of two sequences of a few rows."""
    prefix = None
    if path.startswith("prefix"):
        # a pass of its own from 2^18 tokens on, where few rows are many-row work: the same pages over and over
        prefix = _prefix(bt, 2 ** 18 if path.endswith("merge") else 40, 3)
    table = _wide(bt) if path in ("cut", "prefix join") else bt.page_table
    return table, 3 if path in ("clusters", "cut", "prefix clusters", "prefix join") else 30, prefix


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("cu", [[0, 3, 7], [3, 3, 5], [0, 0, 5], [5, 5, 5]])
def test_sequences_left_without_rows_by_what_is_out_of_range_are_reported(path, cu):
    """Rows past the tokens, rows before the first sequence, a length past its table."""
    n_tok = 3 if cu[-1] == 7 else 5
    bt = Batch(106, [(max(0, e - s), 40) for s, e in zip(cu, cu[1:])], 4, 2, 64, 16, spare=8)
    bt.page_table, max_q, prefix = _path(bt, path)
    bt.q = randn(bt.gen, n_tok, 4, 64)
    bt.cu_q = torch.tensor(cu, dtype=torch.int32, device="cuda")
    if cu[0] == 0 and cu[1] == 0:
        bt.kv_len[0] = -1
    out = torch.full_like(bt.q, 7.0)
    got = _attend(bt, max_q, prefix, out=out)
    _reported()
    first, last = cu[0], min(cu[-1], n_tok)
    assert bool((out[:first] == 7).all()) and bool((out[last:] == 7).all())
    bt.cu, bt.lens, bt.n_tok = [min(c, n_tok) for c in cu], [(min(e, n_tok) - min(s, n_tok), n) for (s, e), (_, n) in
                                                            zip(zip(cu, cu[1:]), bt.lens)], n_tok
    if path == "prefix merge":
        return  # 2^18 keys a row: the formula's bound says nothing
    # rows of a sequence, in place
    for b, (a, _) in enumerate(bt.lens):
        if a:
            one = Batch.__new__(Batch)
            one.__dict__.update(bt.__dict__)
            r = slice(bt.cu[b], bt.cu[b + 1])
            one.lens, one.cu, one.n_tok, one.q, one.page_table = [bt.lens[b]], [0, a], a, bt.q[r], bt.page_table[b:b + 1]
            assert_attend((got[0][r], got[1][:, r]), one, prefix=prefix)


def test_a_first_call_under_inference_mode_leaves_a_status_that_can_be_cleared():
    code = """
import torch
from rolling_kv_cache_b200 import binding as B, paged
tables = paged.rope_tables((4,), (32,))
x = torch.zeros(2, 1, 64, dtype=torch.bfloat16, device="cuda")
with torch.inference_mode():
    paged.rope_axes(x, torch.tensor([[9], [0]], dtype=torch.int32, device="cuda"), tables)
for _ in range(2):
    try:
        paged.device_status()
        print("clear")
    except B.RcError as e:
        print("status", e.status)
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.split("\n")[:2] == [f"status {B.RC_ERANGE}", "clear"], r.stdout


def _small(seed):
    bt = Batch(seed, [(2, 30), (1, 9)], 4, 2, 64, 16)
    return bt, paged.rope_tables((9,), (32,)), torch.zeros(3, 1, dtype=torch.int32, device="cuda")


def test_tangents_of_forward_mode_are_refused():
    """Also one that comes in by a gradient, forward over backward."""
    import torch.autograd.forward_ad as fw
    bt, tables, pos = _small(108)
    q, k_pages, v_pages, *rest = bt.args()
    k = randn(bt.gen, 3, 2, 64)
    with fw.dual_level():
        dual = lambda t: fw.make_dual(t, torch.ones_like(t))  # noqa: E731
        calls = [lambda: paged.rope_axes(dual(q), pos, tables), lambda: paged.rope_axes((q, dual(k)), pos, tables),
                 lambda: paged.rope_axes(dual(q), pos, tables, out=torch.empty_like(q)),
                 lambda: paged.rope_axes(q, pos, (dual(tables[0]),)),
                 lambda: paged.paged_append(dual(q), k, k, k_pages, v_pages, *rest),
                 lambda: paged.paged_append(None, k, dual(k), k_pages, v_pages, *rest),
                 lambda: paged.paged_attention(dual(q), k_pages, v_pages, *rest, max_q=2),
                 lambda: paged.paged_attention(q, k_pages, dual(v_pages), *rest, max_q=2)]
        for call in calls:
            for mode in (torch.enable_grad, torch.no_grad):
                with mode(), pytest.raises(ValueError, match="forward-mode"):
                    call()
        paged.rope_axes(q, pos, tables)  # plain tensors pass
        x = q.float().requires_grad_(True)
        y = paged.rope_axes(x, pos, tables)
        with pytest.raises((ValueError, RuntimeError), match="forward-mode"):
            torch.autograd.grad(y, (x,), dual(torch.ones_like(y)))
        base = torch.zeros(3, 8, 64, dtype=BF16, device="cuda")
        with pytest.raises(ValueError, match="forward-mode"):  # a view of such a tensor
            paged.rope_axes(dual(base)[:, :4], pos, tables)


def test_calls_under_a_trace_are_refused():
    from torch.fx.experimental.proxy_tensor import make_fx
    bt, tables, pos = _small(109)
    q, k_pages, v_pages, *rest = bt.args()
    k = randn(bt.gen, 3, 2, 64)
    for f in (lambda x: paged.rope_axes(x, pos, tables),
              lambda x: paged.paged_append(x, k, k, k_pages, v_pages, *rest),
              lambda x: paged.paged_attention(x, k_pages, v_pages, *rest, max_q=2)):
        with pytest.raises(ValueError, match="trace"):
            torch.jit.trace(f, (q,), check_trace=False)
        with pytest.raises(ValueError, match="trace"):
            make_fx(f)(q)
        f(q)


def test_tables_that_ask_for_a_gradient_are_refused():
    bt, tables, pos = _small(110)
    q, k_pages, v_pages, *rest = bt.args()
    learned = (tables[0].clone().requires_grad_(True),)
    x = q.float().requires_grad_(True)
    for t in (q, x):
        with pytest.raises(ValueError, match="tables"):
            paged.rope_axes(t, pos, learned)
    with pytest.raises(ValueError):
        paged.paged_append(q, q[:, :2], q[:, 2:], k_pages, v_pages, *rest, pos=pos, tables=learned)
    with torch.no_grad():
        y = paged.rope_axes(q, pos, learned)
    assert_turned(y, q, pos, tables, False)


def test_negated_views_are_refused_and_their_gradients_read():
    bt, tables, pos = _small(111)
    q, k_pages, v_pages, *rest = bt.args()
    for call in (lambda: paged.rope_axes(torch._neg_view(q), pos, tables),
                 lambda: paged.rope_axes(q, pos, tables, out=torch._neg_view(torch.empty_like(q))),
                 lambda: paged.paged_append(None, torch._neg_view(q[:, :2]), q[:, 2:], k_pages, v_pages, *rest),
                 lambda: paged.paged_attention(torch._neg_view(q), k_pages, v_pages, *rest, max_q=2)):
        with pytest.raises(ValueError, match="negated"):
            call()
    x = q.float().requires_grad_(True)
    gy = randn(bt.gen, 3, 4, 64, dtype=F32)
    (dx,) = torch.autograd.grad(paged.rope_axes(x, pos, tables), (x,), torch._neg_view(gy))
    assert_turned(dx, -gy, pos, tables, False, inverse=True)


@pytest.mark.parametrize("cu,n_tok", [([0, 3, 7], 3), ([2, 3, 5], 5), ([3, 3, 5], 5), ([0, 3, 7], 6)])
def test_an_append_reports_rows_of_no_sequence_and_rows_that_are_not_there(cu, n_tok):
    bt = Batch(107, [(max(0, e - s), 40) for s, e in zip(cu, cu[1:])], 4, 2, 64, 16, fill=3.0)
    k, v = randn(bt.gen, n_tok, 2, 64), randn(bt.gen, n_tok, 2, 64)
    kp, vp = bt.k_pages.clone(), bt.v_pages.clone()
    for b in range(2):
        for tok in range(cu[b], min(cu[b + 1], n_tok)):
            at = 40 - (cu[b + 1] - tok)
            kp[int(bt.page_table[b, at // 16]), :, at % 16] = k[tok]
            vp[int(bt.page_table[b, at // 16]), :, at % 16] = v[tok]
    cu_q = torch.tensor(cu, dtype=torch.int32, device="cuda")
    paged.paged_append(None, k, v, bt.k_pages, bt.v_pages, cu_q, bt.kv_len, bt.page_table)
    _reported()
    assert torch.equal(bt.k_pages, kp) and torch.equal(bt.v_pages, vp)


def test_threads_on_streams_of_their_own_finish_with_the_same_bits():
    batches = [Batch(112, [(1, 900), (1, 40)] * 6, 8, 2, 128, 16), Batch(113, [(130, 400), (31, 31)], 8, 2, 128, 16)]
    want = [_attend(b, max(a for a, _ in b.lens)) for b in batches]
    torch.cuda.synchronize()
    done, errors = [0, 0], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got = _attend(batches[i], max(a for a, _ in batches[i].lens))
                    torch.cuda.current_stream().synchronize()
                    assert torch.equal(got[0], want[i][0]) and torch.equal(got[1], want[i][1])
                    done[i] += 1
        except BaseException as e:  # reported by the main thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,), daemon=True) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=300)
        assert not t.is_alive()
    assert not errors and done == [20, 20], errors


def test_a_captured_append_reports_a_replay_without_a_page():
    bt = Batch(114, [(1, 30), (1, 90)], 4, 2, 64, 16, fill=3.0)
    k, v = randn(bt.gen, 2, 2, 64), randn(bt.gen, 2, 2, 64)
    call = lambda: paged.paged_append(None, k, v, bt.k_pages, bt.v_pages, bt.cu_q, bt.kv_len, bt.page_table)  # noqa: E731
    call()
    paged.device_status()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        call()
    kp = bt.k_pages.clone()
    bt.kv_len.fill_(55)  # the first sequence has two pages
    k.fill_(1.0)
    gr.replay()
    kp[int(bt.page_table[1, 3]), :, 54 % 16] = 1.0
    _reported()
    assert torch.equal(bt.k_pages, kp)


@pytest.mark.parametrize("cu", [[0, 5, 2, 6], [0, 2, 500, 6], [-3, 2, 5, 6], [4, 4, 4, 2 ** 31 - 1]])
def test_an_append_of_rows_listed_out_of_order_writes_their_places_only(cu):
    """A token goes to the sequence that a bisection for the last start at or before it finds, if it lies in that."""
    bt = Batch(115, [(2, 40), (3, 30), (1, 9)], 4, 2, 64, 16, fill=3.0)
    k, v = randn(bt.gen, 6, 2, 64), randn(bt.gen, 6, 2, 64)
    kp, vp = bt.k_pages.clone(), bt.v_pages.clone()
    places = set()
    for tok in range(6):
        lo, hi = 0, 2
        while lo < hi:
            mid = (lo + hi + 1) >> 1
            lo, hi = (mid, hi) if cu[mid] <= tok else (lo, mid - 1)
        at = bt.lens[lo][1] - (cu[lo + 1] - tok)
        if not cu[lo] <= tok < cu[lo + 1] or at < 0:
            continue
        page = int(bt.page_table[lo, at // 16])
        assert (page, at % 16) not in places
        places.add((page, at % 16))
        if page >= 0:
            kp[page, :, at % 16], vp[page, :, at % 16] = k[tok], v[tok]
    paged.paged_append(None, k, v, bt.k_pages, bt.v_pages, torch.tensor(cu, dtype=torch.int32, device="cuda"), bt.kv_len,
                       bt.page_table)
    torch.cuda.synchronize()
    assert torch.equal(bt.k_pages, kp) and torch.equal(bt.v_pages, vp)
    if cu[0] != 0 or cu[-1] > 6 or max(cu) > 6:
        _reported()
    else:
        try:
            paged.device_status()
        except B.RcError as e:
            assert e.status == B.RC_ERANGE
