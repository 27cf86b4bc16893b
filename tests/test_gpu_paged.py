"""Paged-cache operators against their 64-bit forms: rotary positions over
several axes, the append into pages, attention over pages and over a shared prefix."""
import pytest
import torch

from rolling_kv_cache_b200 import binding as B
from rolling_kv_cache_b200 import paged

from paged_util import Batch, assert_attend, assert_turned, generator, randn, turned

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
    # and those that do not, with the prefix in a pass of its own before a pass for many rows
    ([(30, 30)] * 12 + [(0, 9), (1, 77)], 6, 3, 128, 32, (1, 0, 0), 260),
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
