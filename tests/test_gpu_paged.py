"""Paged-cache operators against their 64-bit forms: rotary positions over
several axes, the append into pages, attention over pages and over a shared prefix."""
import pytest
import torch

from rolling_kv_cache_b200 import binding as B
from rolling_kv_cache_b200 import paged

from paged_util import Batch, assert_attend, assert_turned, attend, generator, randn, turned

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(autouse=True)
def _status_stays_clear():
    yield
    paged.device_status()


def _positions(gen, n_tok, sizes):
    return torch.stack([torch.randint(0, n, (n_tok,), generator=gen, device="cuda") for n in sizes], -1).int()


# ------------------------------------------------------------------ rotation

ROPE = [  # tokens, heads of q and k, d, pairs, positions
    (1, 1, 1, 64, (32,), (7,)),
    (3, 5, 1, 128, (64,), (70000,)),
    (257, 12, 12, 128, (22, 21, 21), (40, 30, 52)),
    (1000, 2, 7, 64, (12, 10, 10), (9, 4, 4)),
    (33, 40, 8, 128, (0, 32, 32), (1, 64, 65)),
    (4097, 3, 1, 64, (16, 16), (65, 64)),
]


@pytest.mark.parametrize("case", ROPE)
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
def test_rope_axes(case, dtype, pairing):
    n, hq, hk, d, pairs, sizes = case
    g = generator(n)
    tables = paged.rope_tables(sizes, pairs)
    pos = _positions(g, n, sizes)
    fused = randn(g, n, hq + 2 * hk, d, dtype=dtype)  # q, k, v of one projection: strided rows
    q, k = fused[:, :hq], fused[:, hq:hq + hk]
    yq, yk = paged.rope_axes((q, k), pos, tables, pairing=pairing)
    halves = pairing == "halves"
    assert_turned(yq, q, pos, tables, halves)
    assert_turned(yk, k, pos, tables, halves)
    back = paged.rope_axes(k, pos, tables, pairing=pairing, inverse=True)
    assert_turned(back, k, pos, tables, halves, inverse=True)
    v = fused[:, hq + hk:].clone()
    paged.rope_axes((q, k), pos, tables, pairing=pairing, out=(q, k))  # in place
    assert torch.equal(q, yq) and torch.equal(k, yk) and torch.equal(fused[:, hq + hk:], v)


@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
def test_rope_axes_gradient(pairing):
    g = generator(5)
    n, d, halves = 37, 64, pairing == "halves"
    tables = paged.rope_tables((9, 4, 4), (12, 10, 10))
    pos = _positions(g, n, (9, 4, 4))
    x = randn(g, n, 3, d, dtype=F32).requires_grad_(True)
    one = randn(g, n, 1, d, dtype=F32).requires_grad_(True)
    shared = one.expand(n, 4, d)  # a head read by four: its gradient is their sum
    gy, gs = randn(g, n, 3, d, dtype=F32).requires_grad_(True), randn(g, n, 4, d, dtype=F32)
    y, ys = paged.rope_axes((x, shared), pos, tables, pairing=pairing)
    dx, done = torch.autograd.grad((y, ys), (x, one), (gy, gs), create_graph=True)
    assert_turned(dx.detach(), gy, pos, tables, halves, inverse=True)
    want, mag = turned(gs, pos, tables, halves, inverse=True)
    err = (done.detach().double() - want.sum(1, keepdim=True)).abs()
    # each of the four within 3 roundings of its pair's magnitude and one of its own, then 3 additions
    assert bool((err <= 8 * 2.0 ** -24 * mag.sum(1, keepdim=True)).all())
    # the gradient's gradient with respect to gy is the turn again
    w = randn(g, n, 3, d, dtype=F32)
    (again,) = torch.autograd.grad(dx, (gy,), w)
    assert_turned(again, w, pos, tables, halves)
    # differences: the turn is linear, so a whole step is exact up to the roundings of
    # x + e (1), of each turn (4) and of dx (4), each 2^-24 of a pair's magnitude (at most 2 max)
    e = randn(g, n, 3, d, dtype=F32)
    with torch.no_grad():
        moved = paged.rope_axes(x + e, pos, tables, pairing=pairing).double() - y.double()
        got, want = (moved * gy.double()).sum(), (dx.double() * e.double()).sum()
        most = 2 * float(x.abs().max() + e.abs().max())
        assert abs(float(got - want)) <= 13 * 2.0 ** -24 * most * float(gy.abs().sum())


def test_rope_axes_gradients_as_autograd_hands_them():
    g = generator(6)
    n, d = 19, 128
    tables = paged.rope_tables((40,), (64,))
    pos = _positions(g, n, (40,))
    x = randn(g, n, 3, d, dtype=F32).requires_grad_(True)
    z = randn(g, n, 2, d, dtype=F32).requires_grad_(True)
    # expanded (strides 0), with the other output unused
    y, _ = paged.rope_axes((x, z), pos, tables)
    dx, dz = torch.autograd.grad(y.sum(), (x, z), allow_unused=True)
    assert_turned(dx, torch.ones(n, 3, d, device="cuda"), pos, tables, False, inverse=True)
    assert dz is None or bool((dz == 0).all())
    # starting 4 bytes past a 16-byte boundary, and transposed
    for odd in (randn(g, n * 3 * d + 1, dtype=F32)[1:].view(n, 3, d), randn(g, n, d, 3, dtype=F32).transpose(1, 2)):
        (dx,) = torch.autograd.grad(paged.rope_axes(x, pos, tables), (x,), odd)
        assert_turned(dx, odd, pos, tables, False, inverse=True)
    # only k needs one
    q = randn(g, n, 3, d, dtype=F32)
    yq, yk = paged.rope_axes((q, z), pos, tables)
    gz = randn(g, n, 2, d, dtype=F32)
    (dz,) = torch.autograd.grad((yq * 2).sum() + (yk * gz).sum(), (z,))
    assert_turned(dz, gz, pos, tables, False, inverse=True)


def test_rope_axes_position_out_of_its_table():
    g = generator(7)
    tables = paged.rope_tables((6,), (32,))
    x = randn(g, 4, 2, 64)
    pos = torch.tensor([[5], [6], [-1], [2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    y = paged.rope_axes(x, pos, tables)
    assert_turned(y, x, pos.clamp(0, 5), tables, False)
    with pytest.raises(B.RcError) as e:
        paged.device_status()
    assert e.value.status == B.RC_ERANGE


def test_rope_axes_no_tokens():
    tables = paged.rope_tables((6,), (32,))
    x = torch.empty((0, 3, 64), dtype=BF16, device="cuda")
    assert paged.rope_axes(x, torch.empty((0, 1), dtype=torch.int32, device="cuda"), tables).shape == (0, 3, 64)


# -------------------------------------------------------------------- append

APPEND = [  # (queries, tokens) of the sequences, q heads, kv heads, d, page
    ([(1, 1)], 1, 1, 64, 16),
    ([(1, 17), (1, 16), (1, 700), (1, 33)], 32, 8, 128, 16),
    ([(5, 5), (0, 9), (70, 200), (1, 64)], 14, 2, 64, 32),
    ([(300, 813), (129, 129)], 12, 12, 128, 128),
    ([(47, 64)], 3, 1, 128, 64),
]


@pytest.mark.parametrize("case", APPEND)
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("pairing", ["adjacent", "halves", None])
@pytest.mark.parametrize("nhd", [False, True])
def test_paged_append(case, dtype, pairing, nhd):
    lens, hq, hk, d, page = case
    bt = Batch(11, lens, hq, hk, d, page, dtype, fill=3.0, pad=3, nhd=nhd)
    g = bt.gen
    fused = randn(g, bt.n_tok, hq + 2 * hk, d, dtype=dtype)
    q, k, v = fused.split((hq, hk, hk), 1)
    c = d // 6
    tables = paged.rope_tables((50, 7, 9), (d // 2 - 2 * c, c, c))
    pos = _positions(g, bt.n_tok, (50, 7, 9))
    kp, vp = bt.k_pages.clone(), bt.v_pages.clone()
    turn = dict(pos=pos, tables=tables, pairing=pairing) if pairing else {}
    q_out = torch.full((bt.n_tok, hq, d), 5.0, dtype=dtype, device="cuda")
    out = paged.paged_append(q, k, v, bt.k_pages, bt.v_pages, bt.cu_q, bt.kv_len, bt.page_table, q_out=q_out, **turn)
    assert out is q_out
    n = bt.cu[-1]
    assert bool((q_out[n:] == 5).all())  # rows behind the last sequence
    touched = torch.zeros(kp.shape[0], page, dtype=torch.bool, device="cuda")
    for b, (a, m) in enumerate(lens):
        r = slice(bt.cu[b], bt.cu[b + 1])
        j = torch.arange(m - a, m, device="cuda")
        pg, row = bt.page_table[b][j // page].long(), j % page
        touched[pg, row] = True
        gk = bt.k_pages[pg, :, row]
        if not a:
            continue
        if pairing:
            assert_turned(gk, k[r], pos[r], tables, pairing == "halves")
        else:
            assert torch.equal(gk, k[r])
        assert torch.equal(bt.v_pages[pg, :, row], v[r])
    if pairing:
        assert_turned(q_out[:n], q[:n], pos[:n], tables, pairing == "halves")
    else:
        assert torch.equal(q_out[:n], q[:n])
    keep = ~touched[:, None, :, None].expand_as(kp)
    assert torch.equal(bt.k_pages[keep], kp[keep]) and torch.equal(bt.v_pages[keep], vp[keep])
    # keys alone, and queries in place
    k2, v2 = bt.k_pages.clone(), bt.v_pages.clone()
    bt.k_pages.copy_(kp)
    bt.v_pages.copy_(vp)
    assert paged.paged_append(None, k, v, bt.k_pages, bt.v_pages, bt.cu_q, bt.kv_len, bt.page_table, **turn) is None
    paged.paged_append(q, k, v, bt.k_pages, bt.v_pages, bt.cu_q, bt.kv_len, bt.page_table, q_out=q, **turn)
    assert torch.equal(q[:n], q_out[:n]) and torch.equal(bt.k_pages, k2) and torch.equal(bt.v_pages, v2)


def test_paged_append_keeps_bad_places_out_of_the_pool():
    bt = Batch(12, [(2, 40), (1, 20), (3, 2), (1, 1000)], 4, 2, 64, 16, fill=3.0)
    bt.page_table[0, 2] = bt.k_pages.shape[0]      # one past the pool
    bt.page_table[1, 1] = -5
    bt.page_table = bt.page_table[:, :40].contiguous()  # the last sequence's place lies past its row
    kp, vp = bt.k_pages.clone(), bt.v_pages.clone()
    k, v = randn(bt.gen, bt.n_tok, 2, 64), randn(bt.gen, bt.n_tok, 2, 64)
    q = paged.paged_append(bt.q, k, v, bt.k_pages, bt.v_pages, bt.cu_q, bt.kv_len, bt.page_table)
    assert torch.equal(q, bt.q)
    # sequence 2 has 3 queries but 2 tokens: its first is at position -1, the others have places
    pg = int(bt.page_table[2, 0])
    kp[pg, :, :2], vp[pg, :, :2] = k[4:6].transpose(0, 1), v[4:6].transpose(0, 1)
    assert torch.equal(bt.k_pages, kp) and torch.equal(bt.v_pages, vp)
    with pytest.raises(B.RcError) as e:
        paged.device_status()
    assert e.value.status == B.RC_ERANGE


# ----------------------------------------------------------------- attention

# (queries, tokens), q heads, kv heads, d, page, (frame, sinks, window)
DECODE = [
    ([(1, 1)], 1, 1, 64, 16, (1, 0, 0)),
    ([(1, 777)], 12, 12, 64, 16, (1, 0, 0)),
    ([(1, 63), (1, 64), (1, 65), (1, 0), (0, 50), (1, 1), (1, 2000)], 32, 8, 128, 16, (1, 0, 0)),
    ([(1, 9000)], 5, 1, 128, 32, (1, 0, 0)),
    ([(1, 5000), (1, 130), (1, 3)], 40, 8, 128, 32, (1, 4, 100)),
    ([(1, 500), (1, 17)], 16, 1, 64, 64, (1, 200, 64)),
    ([(4, 300), (3, 3), (2, 1), (4, 64)], 8, 2, 128, 128, (1, 0, 0)),
    ([(16, 1000), (7, 40)], 2, 2, 64, 16, (4, 1, 3)),
    ([(2, 700), (1, 129)], 14, 2, 128, 64, (16, 0, 2)),
    ([(1, n) for n in range(1, 300, 7)], 3, 3, 64, 16, (1, 0, 0)),
    ([(1, 70)] * 400, 2, 1, 64, 16, (1, 0, 0)),
]


@pytest.mark.parametrize("case", DECODE)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_paged_attention_few_rows(case, dtype):
    lens, hq, hk, d, page, (f, sinks, window) = case
    bt = Batch(21, lens, hq, hk, d, page, dtype, nhd=page == 32)
    max_q = max(a for a, _ in lens)
    assert max_q * (hq // hk) <= 16
    got = paged.paged_attention(*bt.args(), max_q=max_q, frame_seqlen=f, sink_frames=sinks, window_frames=window,
                                return_lse=True)
    assert_attend(got, bt, f=f, sinks=sinks, window=window)


@pytest.mark.parametrize("case", DECODE)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_paged_attention_few_rows_in_a_wide_table(case, dtype):
    """A table with room for long streams: the batch is cut evenly over the GPU, few short units too."""
    lens, hq, hk, d, page, (f, sinks, window) = case
    bt = Batch(22, lens, hq, hk, d, page, dtype, nhd=page == 32)
    wide = torch.full((len(lens), 2 ** 18 // page), -7, dtype=torch.int32, device="cuda")
    wide[:, :bt.page_table.shape[1]] = bt.page_table
    bt.page_table = wide
    got = paged.paged_attention(*bt.args(), max_q=max(a for a, _ in lens), frame_seqlen=f, sink_frames=sinks,
                                window_frames=window, return_lse=True)
    assert_attend(got, bt, f=f, sinks=sinks, window=window)


@pytest.mark.parametrize("units", [1, 2, 16, 17, 32, 33, 64, 65])
@pytest.mark.parametrize("n", [1, 64, 65, 449, 513, 1000])
def test_single_tokens_by_the_number_of_units(units, n):
    """Few short units are each shared by 8, 4 or 2 blocks, more are cut evenly: every count of tiles to a block."""
    bt = Batch(23, [(1, n)] * units, 1, 1, 64, 16)
    assert_attend(paged.paged_attention(*bt.args(), max_q=1, return_lse=True), bt)


PREFILL = [
    ([(1, 1)], 1, 1, 64, 16, (1, 0, 0)),
    ([(17, 17)], 1, 1, 128, 16, (1, 0, 0)),
    ([(128, 128), (129, 129), (256, 300), (257, 257)], 2, 2, 128, 32, (1, 0, 0)),
    ([(37, 37), (300, 900), (1, 500), (0, 7), (5, 3)], 28, 4, 128, 64, (1, 0, 0)),
    ([(900, 900)], 5, 1, 64, 128, (1, 3, 70)),
    ([(200, 1500), (64, 64)], 12, 4, 128, 16, (1, 130, 257)),
    ([(480, 1920)], 3, 3, 128, 64, (160, 1, 6)),
    ([(320, 2000), (160, 160)], 6, 6, 64, 16, (160, 2, 3)),
    ([(96, 700)], 2, 1, 64, 32, (1 << 30, 0, 0)),
    ([(3, 400), (2, 90)], 128, 1, 64, 32, (1, 0, 0)),
    ([(40, 2500)], 100, 1, 128, 128, (1, 0, 0)),
    ([(1200, 1300), (700, 2048)], 16, 8, 128, 16, (7, 1, 40)),
]


@pytest.mark.parametrize("case", PREFILL)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_paged_attention_many_rows(case, dtype):
    lens, hq, hk, d, page, (f, sinks, window) = case
    bt = Batch(22, lens, hq, hk, d, page, dtype, nhd=page == 32)
    got = paged.paged_attention(*bt.args(), frame_seqlen=f, sink_frames=sinks, window_frames=window, return_lse=True,
                                max_q=max(17, max(a for a, _ in lens)))
    assert_attend(got, bt, f=f, sinks=sinks, window=window)


PREFIX = [  # as above, and the prefix's length
    ([(1, 1)], 1, 1, 64, 16, (1, 0, 0), 1),
    ([(1, n) for n in (1, 5, 64, 300, 0)], 32, 8, 128, 16, (1, 0, 0), 1111),
    ([(1, 40)] * 70, 8, 2, 64, 32, (1, 0, 0), 500),
    ([(160, 320), (160, 160), (3, 200)], 4, 4, 128, 64, (160, 0, 0), 700),
    ([(33, 400), (90, 90)], 14, 2, 64, 128, (1, 2, 50), 129),
    # sequences that fill their query tiles walk the prefix themselves
    ([(300, 300), (513, 700), (260, 1000)], 2, 2, 128, 16, (1, 0, 0), 257),
    ([(640, 1280), (320, 320)], 4, 1, 64, 64, (160, 1, 3), 1000),
    ([(290, 290), (0, 5), (700, 900)], 4, 4, 64, 32, (1, 3, 40), 128),
    # and so do short ones, where that is little work
    ([(30, 30)] * 12 + [(0, 9), (1, 77)], 6, 3, 128, 32, (1, 0, 0), 260),
    # many short sequences: the prefix in a pass of its own before a pass for many rows
    ([(20, 20)] * 70, 12, 12, 64, 16, (1, 0, 0), 500),
    ([(5, 60)] * 60 + [(0, 3), (1, 1), (90, 300)], 32, 8, 128, 32, (1, 2, 30), 1000),
    ([(16, 48)] * 50 + [(17, 20)], 24, 8, 64, 128, (16, 0, 2), 1111),
    ([(30, 0)] * 40, 10, 10, 128, 64, (1, 0, 0), 700),
    # few single tokens, in clusters; and many, or a long prefix, in two passes
    ([(1, 39)], 5, 1, 128, 32, (1, 0, 0), 6051),
    ([(1, 259), (0, 7), (1, 0), (3, 90)], 4, 2, 64, 128, (1, 1, 40), 200),
    ([(4, 25), (2, 8)], 16, 8, 128, 64, (1, 0, 0), 1030),
    ([(1, 1000)], 3, 3, 64, 16, (16, 1, 5), 64),
    ([(1, 7)] * 20, 12, 12, 128, 64, (1, 0, 0), 435),
    ([(1, 30)], 1, 1, 64, 16, (1, 0, 0), 9000),
    ([(1, 300), (3, 3)], 20, 5, 128, 32, (1, 0, 0), 40000),
    ([(1, n) for n in range(1, 130, 2)], 8, 2, 64, 64, (1, 0, 0), 777),
]


@pytest.mark.parametrize("case", PREFIX)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_prefix_attention(case, dtype):
    lens, hq, hk, d, page, (f, sinks, window), n = case
    pages = (n + page - 1) // page
    bt = Batch(23, lens, hq, hk, d, page, dtype, spare=pages + 1)
    table = torch.tensor(bt.free[:pages], dtype=torch.int32, device="cuda")
    j = torch.arange(n, device="cuda")
    for pool in (bt.k_pages, bt.v_pages):
        pool[table[j // page].long(), :, j % page] = randn(bt.gen, n, hk, d, dtype=dtype)
    got = paged.prefix_attention(*bt.args()[:3], table, n, *bt.args()[3:], max_q=max(a for a, _ in lens),
                                 frame_seqlen=f, sink_frames=sinks, window_frames=window, return_lse=True)
    assert_attend(got, bt, f=f, sinks=sinks, window=window, prefix=(table, n))


@pytest.mark.parametrize("max_q", [1, 64])
def test_scale_and_out_and_rows_behind_the_last_sequence(max_q):
    lens = [(1, 300), (1, 40)] if max_q == 1 else [(64, 300), (9, 40)]
    bt = Batch(24, lens, 4, 2, 64, 16, pad=5)
    out = torch.full((bt.n_tok, 6, 64), 7.0, dtype=BF16, device="cuda")[:, 1:5]
    o, lse = paged.paged_attention(*bt.args(), max_q=max_q, scale=0.3, out=out, return_lse=True)
    assert o is out and bool((out[bt.cu[-1]:] == 7).all())
    assert_attend((o, lse), bt, scale=0.3)


@pytest.mark.parametrize("max_q", [1, 40])
def test_pages_that_are_none_are_left_out(max_q):
    bt = Batch(25, [(max_q, 500), (max_q, 90)], 4, 2, 64, 16)
    bt.page_table[0, 3], bt.page_table[1, 0] = bt.k_pages.shape[0] + 7, -1
    ref = Batch(25, [(max_q, 500), (max_q, 90)], 4, 2, 64, 16)
    o, lse = paged.paged_attention(*bt.args(), max_q=max_q, return_lse=True)
    # without those pages' keys: the mask of the plain form has no such hole, so move the keys together
    for b, hole in ((0, 3), (1, 0)):
        n = ref.lens[b][1] - 16
        t = ref.page_table[b].tolist()
        one = Batch(25, [(max_q, 500), (max_q, 90)], 4, 2, 64, 16)
        one.lens = [(max_q, n)]
        one.cu = [0, max_q]
        one.n_tok = max_q
        one.q = bt.q[bt.cu[b]:bt.cu[b + 1]]
        one.page_table = torch.tensor([t[:hole] + t[hole + 1:]], dtype=torch.int32, device="cuda")
        assert_attend((o[bt.cu[b]:bt.cu[b + 1]], lse[:, bt.cu[b]:bt.cu[b + 1]]), one)
    with pytest.raises(B.RcError) as e:
        paged.device_status()
    assert e.value.status == B.RC_ERANGE


def test_more_queries_than_max_q_says():
    bt = Batch(26, [(3, 50), (1, 9)], 8, 1, 64, 16)
    out = torch.full_like(bt.q, 7.0)
    paged.paged_attention(*bt.args(), max_q=2, out=out)  # 24 rows in the kernel for 16: 2 queries of 8 heads
    want = paged.paged_attention(*bt.args(), max_q=3)
    assert bool((out[2] == 7).all())
    err = (out[[0, 1, 3]].float() - want[[0, 1, 3]].float()).abs()
    assert float(err.max()) <= 4 * 2.0 ** -8 * float(bt.v_pages[~bt.v_pages.isnan()].abs().max())
    with pytest.raises(B.RcError) as e:
        paged.device_status()
    assert e.value.status == B.RC_ERANGE


# ------------------------------------------------- calls together, and their surroundings

def _cold():
    return torch.empty(96 * 2 ** 20, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("case", [
    ([(1, 300 + 211 * i) for i in range(24)], 32, 8, 128, 32, (1, 0, 0), None),
    ([(1, 4000 + 97 * i) for i in range(9)], 12, 12, 64, 16, (1, 4, 700), None),
    ([(200 + 31 * i, 700 + 40 * i) for i in range(5)], 14, 2, 128, 64, (1, 0, 0), None),
    ([(1, 1 + 13 * i) for i in range(40)], 16, 4, 128, 16, (1, 0, 0), 900),
], ids=["decode", "window", "prompts", "prefix"])
def test_same_bits_on_every_run_with_cold_and_warm_caches(case):
    lens, hq, hk, d, page, (f, sinks, window), n = case
    pages = ((n or 0) + page - 1) // page
    bt = Batch(31, lens, hq, hk, d, page, spare=pages + 1, fill=0.0)
    kw = dict(max_q=max(a for a, _ in lens), frame_seqlen=f, sink_frames=sinks, window_frames=window,
              return_lse=True)
    if n:
        table = torch.tensor(bt.free[:pages], dtype=torch.int32, device="cuda")
        j = torch.arange(n, device="cuda")
        for pool in (bt.k_pages, bt.v_pages):
            pool[table[j // page].long(), :, j % page] = randn(bt.gen, n, hk, d)
        call = lambda: paged.prefix_attention(*bt.args()[:3], table, n, *bt.args()[3:], **kw)  # noqa: E731
    else:
        call = lambda: paged.paged_attention(*bt.args(), **kw)  # noqa: E731
    o, lse = call()
    flush = _cold()
    for i in range(40):
        if i % 2:
            flush.fill_(i)  # the caches hold something else
        o2, lse2 = call()
        assert torch.equal(o, o2) and torch.equal(lse, lse2), i


def _place(n, device="cuda"):
    g = torch.arange(n, device=device)
    return torch.stack((g // 64, g // 8 % 8, g % 8), -1).int()


@pytest.mark.parametrize("q_len,group,f,window", [(1, 4, 1, 0), (1, 1, 1, 40), (48, 2, 16, 5), (150, 1, 64, 0)])
def test_a_stream_appended_and_attended_step_by_step(q_len, group, f, window):
    """Tokens go in through the append, queries come out rotated and attend; after every step the output is that
    of the formula over all tokens so far, rotated by the library's own tables in 64 bits."""
    hk, d, page, steps, sinks = 2, 64, 16, 3, 1 if window else 0
    start = [5, 130, 0]
    bt = Batch(41, [(q_len, n + steps * q_len) for n in start], hk * group, hk, d, page)
    c = d // 6
    tables = paged.rope_tables((500, 8, 8), (d // 2 - 2 * c, c, c))
    g = bt.gen
    bt.k_pages.fill_(float("nan"))
    bt.v_pages.fill_(float("nan"))
    done = [0, 0, 0]
    for step in range(steps + 1):
        new = start if step == 0 else [q_len] * 3
        total = [a + b for a, b in zip(done, new)]
        cu = torch.tensor([0, new[0], new[0] + new[1], sum(new)], dtype=torch.int32, device="cuda")
        kv_len = torch.tensor(total, dtype=torch.int32, device="cuda")
        n = sum(new)
        fused = randn(g, n, hk * group + 2 * hk, d)
        q, k, v = fused.split((hk * group, hk, hk), 1)
        pos = torch.cat([_place(t)[t - m:] for t, m in zip(total, new)])
        qr = paged.paged_append(q, k, v, bt.k_pages, bt.v_pages, cu, kv_len, bt.page_table, pos=pos, tables=tables)
        assert_turned(qr, q, pos, tables, False)
        o, lse = paged.paged_attention(qr, bt.k_pages, bt.v_pages, cu, kv_len, bt.page_table, max_q=max(new),
                                       frame_seqlen=f, sink_frames=sinks, window_frames=window, return_lse=True)
        one = Batch.__new__(Batch)
        one.__dict__.update(bt.__dict__)
        one.lens, one.cu, one.n_tok, one.q = list(zip(new, total)), cu.tolist(), n, qr
        assert_attend((o, lse), one, f=f, sinks=sinks, window=window)
        done = total
    # what lies in the pages is what was appended
    assert not bool(bt.k_pages[bt.page_table[1][0].long()].isnan().any())


def test_continuations_of_a_prefix_equal_whole_sequences():
    """prefix_attention over (prefix, own tokens) against paged_attention over sequences that hold both."""
    n, own, hq, hk, d, page = 160, [1, 33, 70], 8, 2, 128, 16
    whole = Batch(43, [(1, n + m) for m in own], hq, hk, d, page, spare=20)
    for b in range(1, len(own)):  # all sequences begin with the first one's pages
        whole.page_table[b, :n // page] = whole.page_table[0, :n // page]
    a, la = paged.paged_attention(*whole.args(), max_q=1, return_lse=True)
    table = whole.page_table[0, :n // page].contiguous()
    own_table = torch.full_like(whole.page_table, -1)
    own_table[:, :whole.page_table.shape[1] - n // page] = whole.page_table[:, n // page:]
    kv = torch.tensor(own, dtype=torch.int32, device="cuda")
    o, lo = paged.prefix_attention(*whole.args()[:3], table, n, whole.cu_q, kv, own_table, max_q=1, return_lse=True)
    bound = attend(whole)[2]
    assert bool(((a.double() - o.double()).abs() <= 2 * bound).all())
    assert float((la - lo).abs().max()) <= 2.0 ** -11


def test_paged_stream_equals_the_ring():
    """A stream short enough to keep every frame: the ring's step and the paged append and attention agree."""
    from rolling_kv_cache_b200.cache import RollingKVCache, make_config
    H, d, gh, gw, chunk = 4, 128, 6, 10, 3
    F = gh * gw
    cfg = make_config(layers=1, heads=H, head_dim=d, grid_h=gh, grid_w=gw, sink_frames=1, window_frames=9,
                      chunk_frames=chunk)
    cache = RollingKVCache(cfg)
    c = (d // 2) // 3
    tables = paged.rope_tables((64, gh, gw), (d // 2 - 2 * c, c, c))
    g = generator(44)
    chunks = 3
    pages = (chunks * chunk * F + 63) // 64
    k_pages, v_pages = (torch.full((pages + 2, H, 64, d), float("nan"), dtype=BF16, device="cuda") for _ in range(2))
    table = torch.randperm(pages + 2, generator=g, device="cuda")[:pages].int()[None].contiguous()
    for i in range(chunks):
        q, k, v = (randn(g, chunk * F, H, d) for _ in range(3))
        lse = torch.empty((H, chunk * F), dtype=torch.float32, device="cuda")
        want = cache.step(0, q, k, v, i * chunk, lse=lse)
        t = torch.arange(i * chunk * F, (i + 1) * chunk * F, device="cuda")
        pos = torch.stack((t // F, t % F // gw, t % gw), -1).int()
        cu = torch.tensor([0, chunk * F], dtype=torch.int32, device="cuda")
        kv = torch.tensor([(i + 1) * chunk * F], dtype=torch.int32, device="cuda")
        qr = paged.paged_append(q, k, v, k_pages, v_pages, cu, kv, table, pos=pos, tables=tables)
        got, l2 = paged.paged_attention(qr, k_pages, v_pages, cu, kv, table, frame_seqlen=F, return_lse=True)
        # both round P and the output to bf16: 2 * (2^-8 + 2^-8) of the largest value weighted, and as much
        # again for rotated keys that round differently (the ring's products are rounded apart)
        assert float((got.float() - want.float()).abs().max()) <= 2e-2
        assert float((l2 - lse).abs().max()) <= 1e-2
    cache.close()


@pytest.mark.parametrize("kind", ["decode", "prompt", "prefix"])
def test_captured_calls_see_each_replays_lengths(kind):
    lens = [(1, 100), (1, 20)] if kind != "prompt" else [(40, 100), (40, 40)]
    bt = Batch(45, [(a, n + 60) for a, n in lens], 8, 2, 128, 16, spare=8)
    table = torch.tensor(bt.free[:5], dtype=torch.int32, device="cuda")
    j = torch.arange(70, device="cuda")
    for pool in (bt.k_pages, bt.v_pages):
        pool[table[j // 16].long(), :, j % 16] = randn(bt.gen, 70, 2, 128)
    max_q = lens[0][0]

    def call():
        if kind == "prefix":
            return paged.prefix_attention(*bt.args()[:3], table, 70, *bt.args()[3:], max_q=max_q, return_lse=True)
        return paged.paged_attention(*bt.args(), max_q=max_q, return_lse=True)

    call()
    graphs = []
    for _ in range(2):  # two graphs of one call share nothing
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            got = call()
        graphs.append((gr, got))
    for extra in (0, 7, 60):
        now = [(a, n + extra) for a, n in lens]
        bt.kv_len.copy_(torch.tensor([n for _, n in now], dtype=torch.int32))
        bt.q.copy_(randn(bt.gen, *bt.q.shape))
        bt.lens = now
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        graphs[0][0].replay()
        with torch.cuda.stream(side):
            graphs[1][0].replay()
        torch.cuda.synchronize()
        for _, got in graphs:
            assert_attend(got, bt, **(dict(prefix=(table, 70)) if kind == "prefix" else {}))


def test_captured_append_and_rotation():
    bt = Batch(46, [(1, 30), (1, 90)], 4, 2, 64, 16, fill=0.0)
    k, v = randn(bt.gen, 2, 2, 64), randn(bt.gen, 2, 2, 64)
    tables = paged.rope_tables((200,), (32,))
    pos = torch.tensor([[29], [89]], dtype=torch.int32, device="cuda")
    paged.paged_append(bt.q, k, v, bt.k_pages, bt.v_pages, bt.cu_q, bt.kv_len, bt.page_table, pos=pos, tables=tables)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = paged.paged_append(bt.q, k, v, bt.k_pages, bt.v_pages, bt.cu_q, bt.kv_len, bt.page_table, pos=pos,
                                 tables=tables)
    for n in (17, 55):
        k.copy_(randn(bt.gen, 2, 2, 64))
        bt.kv_len.fill_(n)
        pos.fill_(n - 1)
        gr.replay()
        torch.cuda.synchronize()
        assert_turned(out, bt.q, pos, tables, False)
        for b in range(2):
            pg = int(bt.page_table[b, (n - 1) // 16])
            if pg >= 0:
                assert_turned(bt.k_pages[pg, :, (n - 1) % 16][None], k[b:b + 1], pos[b:b + 1], tables, False)
    paged_status_or_clear()


def paged_status_or_clear():
    try:
        paged.device_status()
    except B.RcError:
        pass  # sequence 0 has no page for 55 tokens: that is reported, and kept out


def test_rotation_gradient_captured_into_a_graph():
    g = generator(47)
    tables = paged.rope_tables((50,), (64,))
    pos = _positions(g, 20, (50,))
    x = randn(g, 20, 3, 128, dtype=F32).requires_grad_(True)
    gy = randn(g, 20, 3, 128, dtype=F32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # warm-up as graphs ask for
        for _ in range(2):
            torch.autograd.grad(paged.rope_axes(x, pos, tables), (x,), gy)
    torch.cuda.current_stream().wait_stream(side)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        (dx,) = torch.autograd.grad(paged.rope_axes(x, pos, tables), (x,), gy)
    gy.copy_(randn(g, 20, 3, 128, dtype=F32))
    gr.replay()
    torch.cuda.synchronize()
    assert_turned(dx, gy, pos, tables, False, inverse=True)


def test_two_streams_and_two_threads_at_once():
    import threading
    batches = [Batch(50 + i, [(1, 900 + 100 * i), (1, 40)] * 6, 8, 2, 128, 16) for i in range(2)]
    batches += [Batch(60 + i, [(130, 400), (31, 31)], 8, 2, 128, 16) for i in range(2)]
    want = [paged.paged_attention(*b.args(), max_q=max(a for a, _ in b.lens)) for b in batches]
    torch.cuda.synchronize()
    errors = []

    def work(b, w):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got = paged.paged_attention(*b.args(), max_q=max(a for a, _ in b.lens))
                    torch.cuda.current_stream().synchronize()
                    if not torch.equal(got, w):
                        errors.append("differs")
        except Exception as e:  # reported by the main thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=x) for x in zip(batches, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=300)
    assert not errors, errors


def test_refusals_on_the_device():
    bt = Batch(70, [(1, 30)], 4, 2, 64, 16)
    q, k_pages, v_pages, cu, kv, table = bt.args()
    bad = [
        dict(q=q[:, :, ::2]), dict(q=q.float()), dict(q=q[:, :3]), dict(cu_q=cu.long()), dict(kv_len=kv[:0]),
        dict(page_table=table[0]), dict(v_pages=v_pages[:, :1]), dict(q=q.cpu()), dict(q=q.half()),
        dict(out=torch.empty_like(q)[:, :2]), dict(scale=0.0), dict(scale=-1.0), dict(frame_seqlen=0),
        dict(max_q=-1), dict(max_q=2 ** 31), dict(q=q[..., :32]), dict(q=q.expand(1, 4, 64)[:, :1].expand(1, 4, 64)),
    ]
    for over in bad:
        args = dict(q=q, k_pages=k_pages, v_pages=v_pages, cu_q=cu, kv_len=kv, page_table=table, max_q=1)
        args.update(over)
        with pytest.raises((ValueError, B.RcError)):
            paged.paged_attention(**args)
    with pytest.raises(ValueError):
        paged.paged_attention(q.requires_grad_(True), k_pages, v_pages, cu, kv, table)
    q.requires_grad_(False)
    with pytest.raises(ValueError):
        paged.prefix_attention(q, k_pages, v_pages, table[0], 0, cu, kv, table)
    with pytest.raises(B.RcError):
        paged.prefix_attention(q, k_pages, v_pages, table[0][:1].contiguous(), 17, cu, kv, table)
    k = randn(bt.gen, 1, 2, 64)
    with pytest.raises(ValueError):
        paged.paged_append(q, k, k, k_pages, v_pages, cu, kv, table, pos=torch.zeros(1, 1, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        paged.paged_append(q, k, k.half(), k_pages, v_pages, cu, kv, table)
    with pytest.raises(ValueError):
        paged.paged_append(None, k, k, k_pages, v_pages, cu, kv, table, q_out=q)
    tables = paged.rope_tables((9,), (32,))
    pos = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    for args in [(q, pos.long(), tables), (q, pos[:0], tables), (q, pos, tables + tables), (q.long(), pos, tables),
                 (q[0], pos, tables), ((q, k, k), pos, tables), (q, pos, (tables[0].half(),))]:
        with pytest.raises((ValueError, B.RcError)):
            paged.rope_axes(*args)
    with pytest.raises(ValueError):
        paged.rope_axes(q, pos, tables, pairing="quarter")
    # a slice that starts off a 16-byte boundary
    with pytest.raises(B.RcError):
        paged.rope_axes(torch.zeros(1 * 4 * 64 + 1, dtype=BF16, device="cuda")[1:].view(1, 4, 64), pos, tables)


def test_an_empty_batch():
    bt = Batch(71, [(1, 30)], 4, 2, 64, 16)
    none = torch.empty((0, 4, 64), dtype=BF16, device="cuda")
    cu, kv, table = torch.zeros(1, dtype=torch.int32, device="cuda"), bt.kv_len[:0], bt.page_table[:0]
    assert paged.paged_attention(none, bt.k_pages, bt.v_pages, cu, kv, table).shape == (0, 4, 64)
    k = none[:, :2]
    assert paged.paged_append(none, k, k, bt.k_pages, bt.v_pages, cu, kv, table).shape == (0, 4, 64)
    # tokens, but no sequence: nothing is written
    out = torch.full((3, 4, 64), 7.0, dtype=BF16, device="cuda")
    paged.paged_attention(torch.zeros_like(out), bt.k_pages, bt.v_pages, cu, kv, table, out=out)
    assert bool((out == 7).all())


def test_a_pool_past_32_bit_offsets():
    """Pages whose offsets in bytes and in elements pass 2^32: the first and the last of 9 GB."""
    hk, d, page = 8, 128, 128
    n = (9 * 2 ** 30) // (hk * page * d * 2)
    pool = torch.empty((n, hk, page, d), dtype=BF16, device="cuda")
    g = generator(72)
    table = torch.tensor([[n - 1, 0, n - 2, 3]], dtype=torch.int32, device="cuda")
    for i in table[0].tolist():
        pool[i] = randn(g, hk, page, d)
    for a in (1, 60):
        bt = Batch.__new__(Batch)
        bt.lens, bt.hq, bt.hk, bt.d, bt.page, bt.dtype, bt.cu, bt.n_tok = [(a, 500)], 16, hk, d, page, BF16, [0, a], a
        bt.q, bt.k_pages, bt.v_pages, bt.page_table = randn(g, a, 16, d), pool, pool, table
        bt.cu_q = torch.tensor([0, a], dtype=torch.int32, device="cuda")
        bt.kv_len = torch.tensor([500], dtype=torch.int32, device="cuda")
        assert_attend(paged.paged_attention(*bt.args(), max_q=a, return_lse=True), bt)
    k, v = randn(g, 1, hk, d), randn(g, 1, hk, d)
    kv = torch.tensor([1], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    v_pool = torch.empty_like(pool)
    paged.paged_append(None, k, v, pool, v_pool, cu, kv, table)
    assert torch.equal(pool[n - 1, :, 0], k[0]) and torch.equal(v_pool[n - 1, :, 0], v[0])


@pytest.mark.parametrize("max_q", [1, 50])
def test_keys_of_one_stream_do_not_reach_another(max_q):
    """Infinities and NaN in one stream's pages leave the other's result as it was."""
    lens = [(max_q, 200), (max_q, 333)]
    a, b = (Batch(73, lens, 4, 2, 64, 16, fill=0.0) for _ in range(2))
    own = b.page_table[1][:21].long()
    b.k_pages[own] = float("inf")
    b.v_pages[own] = float("nan")
    x = paged.paged_attention(*a.args(), max_q=max_q)
    y = paged.paged_attention(*b.args(), max_q=max_q)
    assert torch.equal(x[:max_q], y[:max_q]) and bool(y[max_q:].isnan().any())


def test_thousands_of_sequences():
    """The most sequences of a call, in both kernels; more units than whole rounds are planned for in one of them."""
    lens = [(1 + i % 2, 1 + i * 7 % 30 + i % 2) for i in range(4096)]
    bt = Batch(74, lens, 24, 3, 64, 16)
    a, la = paged.paged_attention(*bt.args(), max_q=2, return_lse=True)
    b, lb = paged.paged_attention(*bt.args(), max_q=17, return_lse=True)
    sample = Batch.__new__(Batch)
    sample.__dict__.update(bt.__dict__)
    pick = [0, 1, 511, 512, 513, 2000, 4094, 4095]
    sample.lens = [lens[i] for i in pick]
    rows = [r for i in pick for r in range(bt.cu[i], bt.cu[i + 1])]
    sample.cu = [0]
    for q, _ in sample.lens:
        sample.cu.append(sample.cu[-1] + q)
    sample.n_tok, sample.q, sample.page_table = len(rows), bt.q[rows], bt.page_table[pick]
    for o, lse in ((a, la), (b, lb)):
        assert_attend((o[rows], lse[:, rows]), sample)
    # everywhere else the two differ by no more than both bounds allow a value of the largest magnitude
    most = float(bt.v_pages[~bt.v_pages.isnan()].abs().max())
    assert float((a.float() - b.float()).abs().max()) <= 4 * 2.0 ** -8 * 2 * most
    assert float((la - lb).abs().max()) <= 2.0 ** -10
    more = torch.zeros(4098, dtype=torch.int32, device="cuda")
    with pytest.raises(B.RcError):
        paged.paged_attention(bt.q[:1], bt.k_pages, bt.v_pages, more, more[:-1], bt.page_table[:1].expand(4097, -1))


@pytest.mark.parametrize("max_q", [1, 70])
def test_in_place_and_a_table_row_shared_by_all(max_q):
    bt = Batch(75, [(max_q, 300)] * 3, 8, 2, 128, 16)
    bt.page_table = bt.page_table[:1].expand(3, -1)  # stride 0
    want, wl = paged.paged_attention(*bt.args(), max_q=max_q, return_lse=True)
    assert_attend((want, wl), bt)
    q = bt.q.clone()
    got = paged.paged_attention(q, *bt.args()[1:], max_q=max_q, out=q)
    assert got is q and torch.equal(q, want)


def test_queries_that_see_only_the_prefix():
    """kv_len 0 and a table without columns: the sequences' own tokens are none."""
    for a, hq in ((1, 8), (300, 2), (30, 8)):
        bt = Batch(76, [(a, 0)] * 2, hq, 2, 64, 16, spare=9)
        bt.page_table = bt.page_table[:, :0]
        table = torch.tensor(bt.free[:8], dtype=torch.int32, device="cuda")
        j = torch.arange(120, device="cuda")
        for pool in (bt.k_pages, bt.v_pages):
            pool[table[j // 16].long(), :, j % 16] = randn(bt.gen, 120, 2, 64)
        got = paged.prefix_attention(*bt.args()[:3], table, 120, *bt.args()[3:], max_q=a, return_lse=True)
        bt.page_table = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
        assert_attend(got, bt, prefix=(table, 120))


def test_lengths_past_the_table_are_cut_and_reported():
    bt = Batch(77, [(1, 40), (1, 9)], 4, 2, 64, 16)
    bt.page_table = bt.page_table[:, :3].contiguous()
    want, wl = paged.paged_attention(*bt.args(), max_q=1, return_lse=True)
    bt.kv_len = torch.tensor([49, 9], dtype=torch.int32, device="cuda")  # 48 places
    long = torch.tensor([2 ** 31 - 1, -4], dtype=torch.int32, device="cuda")
    for kv in (bt.kv_len, long):
        for max_q in (1, 20):
            paged.paged_attention(bt.q, bt.k_pages, bt.v_pages, bt.cu_q, kv, bt.page_table, max_q=max_q)
            with pytest.raises(B.RcError) as e:
                paged.device_status()
            assert e.value.status == B.RC_ERANGE
    again, al = paged.paged_attention(bt.q, bt.k_pages, bt.v_pages, bt.cu_q,
                                      torch.tensor([40, 9], dtype=torch.int32, device="cuda"), bt.page_table, max_q=1,
                                      return_lse=True)
    assert torch.equal(again, want) and torch.equal(al, wl)


def test_rows_listed_out_of_order_fault_nothing():
    """cu_q that descends or passes the tokens: brought into range and reported."""
    bt = Batch(78, [(2, 40), (3, 30), (1, 9)], 4, 2, 64, 16)
    for cu in ([0, 5, 2, 6], [0, 2, 500, 6], [-3, 2, 5, 6], [4, 4, 4, 2 ** 31 - 1]):
        t = torch.tensor(cu, dtype=torch.int32, device="cuda")
        for max_q in (3, 20):
            paged.paged_attention(bt.q, bt.k_pages, bt.v_pages, t, bt.kv_len, bt.page_table, max_q=max_q)
            with pytest.raises(B.RcError) as e:
                paged.device_status()
            assert e.value.status == B.RC_ERANGE
        k = randn(bt.gen, bt.n_tok, 2, 64)
        paged.paged_append(None, k, k, bt.k_pages, bt.v_pages, t, bt.kv_len, bt.page_table)
        torch.cuda.synchronize()
    try:
        paged.device_status()  # some of these give a token a place that is none
    except B.RcError:
        pass


@pytest.mark.parametrize("pages", [190, 300])  # in clusters, in two passes
def test_a_nan_in_the_prefix_reaches_every_row_and_reads_no_part_that_is_none(pages):
    """Rows whose sum is NaN, with parts of unequal number on both sides of a pair of query tiles."""
    lens = [(1, 70)] + [(2, 40)] * 31 + [(1, 0)]  # 8 heads a key head: 32 queries a pair, the 16th of the twos in both
    bt = Batch(79, lens, 8, 1, 64, 16, spare=pages + 10)
    n = 16 * pages + 3
    table = torch.tensor(bt.free[:pages + 1], dtype=torch.int32, device="cuda")
    j = torch.arange(n, device="cuda")
    for pool in (bt.k_pages, bt.v_pages):
        pool[table[j // 16].long(), :, j % 16] = randn(bt.gen, n, 1, 64)
    call = lambda: paged.prefix_attention(*bt.args()[:3], table, n, *bt.args()[3:], max_q=2, return_lse=True)
    want = call()
    assert_attend(want, bt, prefix=(table, n))
    at = (int(table[100]), 0, 5)
    key = bt.k_pages[at].clone()
    bt.k_pages[at] = float("nan")
    o, lse = call()
    assert bool(o.isnan().all()) and bool(lse.isnan().all())
    bt.k_pages[at] = key
    again = call()
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


@pytest.mark.parametrize("a", [1, 40])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_key_that_is_no_number_makes_the_rows_that_see_it_nan(a, value):
    """A NaN score, and one of +inf (inf - inf in the softmax), wherever in a tile; other sequences keep their bits."""
    for at in (0, 3, 5, 118, 127, 130, 4001):
        bt = Batch(80, [(a, 5000), (a, 300), (a, 40)], 2, 1, 64, 16)
        want, wl = paged.paged_attention(*bt.args(), max_q=a, return_lse=True)
        row = bt.k_pages[int(bt.page_table[0, at // 16]), 0, at % 16]
        row.copy_(torch.full_like(row, value) if value != value else value * bt.q[a - 1, 0].sign())
        o, lse = paged.paged_attention(*bt.args(), max_q=a, return_lse=True)
        rows = slice(0, a) if value != value else slice(a - 1, a)
        heads = slice(0, 2) if value != value else slice(0, 1)
        assert bool(o[rows, heads].isnan().all()) and bool(lse[heads, rows].isnan().all()), at
        assert torch.equal(o[a:], want[a:]) and torch.equal(lse[:, a:], wl[:, a:])


@pytest.mark.parametrize("max_q", [1, 40])
def test_the_smallest_scale_and_scales_beyond_the_bounds(max_q):
    bt = Batch(81, [(max_q, 500), (max_q, 70)], 4, 2, 64, 16)
    assert_attend(paged.paged_attention(*bt.args(), max_q=max_q, scale=1e-30, return_lse=True), bt, scale=1e-30)
    for scale in (1e-31, 1e-46, 1.1e30, 1e300, float("nan"), float("inf")):
        with pytest.raises(ValueError):
            paged.paged_attention(*bt.args(), max_q=max_q, scale=scale)


def test_writes_into_tensors_that_autograd_saved_are_noticed():
    bt = Batch(82, [(2, 30), (1, 9)], 4, 2, 64, 16)
    q, k_pages, v_pages, cu, kv, table = bt.args()
    tables = paged.rope_tables((9,), (32,))
    pos = torch.zeros(3, 1, dtype=torch.int32, device="cuda")
    k = randn(bt.gen, 3, 2, 64)
    writes = [(q, lambda: paged.rope_axes(q, pos, tables, out=q)),
              (k, lambda: paged.rope_axes((q, k), pos, tables, out=(torch.empty_like(q), k))),
              (q, lambda: paged.paged_append(q, k, k, k_pages, v_pages, cu, kv, table, q_out=q)),
              (k_pages, lambda: paged.paged_append(None, k, k, k_pages, v_pages, cu, kv, table)),
              (v_pages, lambda: paged.paged_append(None, k, k, k_pages, v_pages, cu, kv, table)),
              (q, lambda: paged.paged_attention(q, k_pages, v_pages, cu, kv, table, max_q=2, out=q))]
    w = torch.ones((), dtype=BF16, device="cuda", requires_grad=True)
    for t, write in writes:
        y = (w * t).sum()  # saves t
        with torch.no_grad():
            write()
        with pytest.raises(RuntimeError, match="inplace"):
            y.backward()
    with torch.inference_mode():  # tensors without a version
        x = randn(bt.gen, 3, 2, 64)
        paged.rope_axes(x, pos, tables, out=x)


def test_capture_beside_a_living_eager_graph_is_refused():
    g = generator(83)
    tables = paged.rope_tables((50,), (64,))
    pos = _positions(g, 20, (50,))
    x = randn(g, 20, 3, 128, dtype=F32).requires_grad_(True)
    gy = randn(g, 20, 3, 128, dtype=F32)
    y = paged.rope_axes(x, pos, tables)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        z = gy + 1
        with pytest.raises(ValueError, match="graph of this tensor"):
            paged.rope_axes(x, pos, tables)
        with pytest.raises(ValueError, match="graph of this tensor"):
            paged.rope_axes((gy, x), pos, tables)
        paged.rope_axes(x.detach(), pos, tables)
    del y
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        (dx,) = torch.autograd.grad(paged.rope_axes(x, pos, tables), (x,), gy)
    gr.replay()
    torch.cuda.synchronize()
    assert_turned(dx, gy, pos, tables, False, inverse=True)


@pytest.mark.parametrize("max_q,prefix", [(3, 0), (30, 0), (3, 40), (30, 40), (300, 200)])
def test_rows_before_the_first_sequence_are_left_and_reported(max_q, prefix):
    """cu_q that begins above 0, as a slice of a larger batch's does."""
    bt = Batch(84, [(2, 2), (max_q, max_q + 40), (1, 9)], 4, 2, 64, 16, spare=14)
    table = torch.tensor(bt.free[:13], dtype=torch.int32, device="cuda")
    j = torch.arange(prefix, device="cuda")
    for pool in (bt.k_pages, bt.v_pages):
        pool[table[j // 16].long(), :, j % 16] = randn(bt.gen, prefix, 2, 64)
    attend = lambda *a, **k: (paged.prefix_attention(*a[:3], table, prefix, *a[3:], **k) if prefix
                              else paged.paged_attention(*a, **k))
    out = torch.full_like(bt.q, 7.0)
    _, lse = attend(bt.q, bt.k_pages, bt.v_pages, bt.cu_q[1:], bt.kv_len[1:], bt.page_table[1:], max_q=max_q, out=out,
                    return_lse=True)
    assert bool((out[:2] == 7).all())
    bt.lens, bt.cu, bt.q, bt.page_table = bt.lens[1:], [n - 2 for n in bt.cu[1:]], bt.q[2:], bt.page_table[1:]
    bt.n_tok -= 2
    assert_attend((out[2:], lse[:, 2:]), bt, prefix=(table, prefix) if prefix else None)
    with pytest.raises(B.RcError) as e:
        paged.device_status()
    assert e.value.status == B.RC_ERANGE


def test_cut_units_with_more_queries_than_max_q_says():
    """Few rows all the same: the kernel computes them, and the merge of parts does too."""
    for lens in ([(3, 9000)], [(4, 30), (3, 20000), (1, 5)]):
        bt = Batch(85, lens, 8, 2, 64, 16)
        assert_attend(paged.paged_attention(*bt.args(), max_q=1, return_lse=True), bt)


def test_rows_before_the_first_of_many_short_sequences():
    """As above, where two results are merged."""
    lens, prefix = [(2, 2)] + [(20, 20)] * 70, 500
    bt = Batch(86, lens, 12, 12, 64, 16, pad=3, spare=40)
    table = torch.tensor(bt.free[:32], dtype=torch.int32, device="cuda")
    j = torch.arange(prefix, device="cuda")
    for pool in (bt.k_pages, bt.v_pages):
        pool[table[j // 16].long(), :, j % 16] = randn(bt.gen, prefix, 12, 64)
    out = torch.full_like(bt.q, 7.0)
    _, lse = paged.prefix_attention(bt.q, bt.k_pages, bt.v_pages, table, prefix, bt.cu_q[1:], bt.kv_len[1:],
                                    bt.page_table[1:], max_q=20, out=out, return_lse=True)
    assert bool((out[:2] == 7).all()) and bool((out[-3:] == 7).all())
    bt.lens, bt.cu, bt.q, bt.page_table = bt.lens[1:], [n - 2 for n in bt.cu[1:]], bt.q[2:], bt.page_table[1:]
    bt.n_tok -= 2
    assert_attend((out[2:], lse[:, 2:]), bt, prefix=(table, prefix))
    with pytest.raises(B.RcError) as e:
        paged.device_status()
    assert e.value.status == B.RC_ERANGE
