"""Paged-cache operators without a GPU: refusals of the C entries and of the Python functions, struct
layouts, and rotation tables."""
import ctypes

import numpy as np
import pytest
import torch

from rolling_kv_cache_b200 import binding as B
from rolling_kv_cache_b200 import paged

from test_abi import _header_layout

P = 1 << 20  # an aligned address that nothing reads: every call here is refused before a launch


def test_struct_layouts_match_header():
    structs = [B.rc_rope, B.rc_rows, B.rc_paged, B.rc_paged_mask]
    lay = _header_layout(structs)
    for st in structs:
        assert ctypes.sizeof(st) == lay[st.__name__], st.__name__
        for f, _ in st._fields_:
            assert getattr(st, f).offset == lay[f"{st.__name__}.{f}"], (st.__name__, f)


def _pool(**over):
    s = dict(k_pages=P, v_pages=P, k_stride=(2 * 16 * 64, 16 * 64, 64), v_stride=(2 * 16 * 64, 16 * 64, 64),
             n_pages=10, page_size=16, kv_heads=2, head_dim=64, dtype=B.RC_BF16, n_seqs=3, cu_q=P, kv_len=P,
             page_table=P, table_stride=5, max_pages=5)
    s.update(over)
    s["k_stride"], s["v_stride"] = ((ctypes.c_int64 * 3)(*s[n]) for n in ("k_stride", "v_stride"))
    return B.rc_paged(**s)


def _rope(**over):
    s = dict(pos=P, table=(P, P, 0), n_pos=(4, 4, 0), pairs=(16, 16, 0), n_axes=2, pairing=B.RC_PAIR_HALVES)
    s.update(over)
    return B.rc_rope(pos=s["pos"], table=(ctypes.c_void_p * 3)(*s["table"]), n_pos=(ctypes.c_int32 * 3)(*s["n_pos"]),
                     pairs=(ctypes.c_int32 * 3)(*s["pairs"]), n_axes=s["n_axes"], pairing=s["pairing"])


def _rows(heads=4, data=P, tok=None, head=64):
    return B.rc_rows(data, heads * 64 if tok is None else tok, head, heads)


def _refused(status, fn, *args):
    with pytest.raises(B.RcError) as e:
        fn(*args)
    assert e.value.status == status, str(e.value)
    assert B.lib().rc_last_error()


BAD_POOLS = [dict(dtype=B.RC_F32), dict(dtype=9), dict(head_dim=96), dict(page_size=8), dict(page_size=48),
             dict(page_size=256), dict(kv_heads=0), dict(kv_heads=2000), dict(n_pages=0), dict(k_pages=0),
             dict(v_pages=P + 8), dict(k_stride=(2048, 1024, 60)), dict(v_stride=(2048, 1024, 32)),
             dict(k_stride=(-2048, 1024, 64)), dict(v_stride=(1 << 39, 1024, 64)), dict(n_seqs=-1), dict(n_seqs=4097),
             dict(cu_q=0), dict(kv_len=0), dict(page_table=0), dict(max_pages=-1), dict(table_stride=4),
             dict(table_stride=-5)]


@pytest.mark.parametrize("over", BAD_POOLS, ids=lambda o: next(iter(o)) + str(next(iter(o.values()))))
def test_bad_pools_are_refused(over):
    p = _pool(**over)
    two = _rows(2)
    _refused(B.RC_EINVAL, B.rc_paged_append, p, None, 3, _rows(), two, two, _rows())
    _refused(B.RC_EINVAL, B.rc_paged_workspace, p, B.rc_paged_mask(frame_seqlen=1, max_q=1), 3, 4)
    _refused(B.RC_EINVAL, B.rc_paged_attention, p, B.rc_paged_mask(frame_seqlen=1, max_q=1), 3, _rows(), _rows(), 0,
             P, 1 << 30)


def test_bounds_of_a_call():
    big = _pool(max_pages=(1 << 26) + 1, table_stride=1 << 27)
    _refused(B.RC_ERANGE, B.rc_paged_workspace, big, B.rc_paged_mask(frame_seqlen=1, max_q=1), 3, 4)
    # 4096 sequences of up to 2^25 tokens: their key tiles pass 32 bits
    many = _pool(n_seqs=4096, max_pages=1 << 21, table_stride=1 << 21)
    for max_q in (1, 100):
        _refused(B.RC_ERANGE, B.rc_paged_workspace, many, B.rc_paged_mask(frame_seqlen=1, max_q=max_q), 4096, 4)
    for n in (-1, (1 << 30) + 1):
        _refused(B.RC_EINVAL, B.rc_paged_workspace, _pool(), B.rc_paged_mask(frame_seqlen=1, max_q=1), n, 4)


BAD_MASKS = [dict(frame_seqlen=0), dict(frame_seqlen=(1 << 30) + 1), dict(sink_frames=-1, window_frames=1),
             dict(window_frames=-1), dict(sink_frames=1), dict(max_q=-1), dict(scale=-1.0), dict(scale=float("nan")),
             dict(scale=float("inf")), dict(prefix_len=-1), dict(prefix_len=5), dict(prefix_len=17, prefix_table=P, prefix_pages=1),
             dict(prefix_len=5, prefix_table=P, prefix_pages=-1)]


@pytest.mark.parametrize("over", BAD_MASKS, ids=lambda o: "-".join(f"{k}{v}" for k, v in o.items()))
def test_bad_masks_are_refused(over):
    m = B.rc_paged_mask(**{**dict(frame_seqlen=1, max_q=1), **over})
    _refused(B.RC_EINVAL, B.rc_paged_workspace, _pool(), m, 3, 4)


@pytest.mark.parametrize("scale", [1e-44, 9e-31, 1.1e30, 3e38])
def test_scales_whose_reciprocal_or_product_overflows_are_refused(scale):
    m = B.rc_paged_mask(frame_seqlen=1, max_q=1, scale=scale)
    _refused(B.RC_EINVAL, B.rc_paged_workspace, _pool(), m, 3, 4)


def test_bad_heads_rows_and_workspaces_are_refused():
    m = B.rc_paged_mask(frame_seqlen=1, max_q=1)
    for heads in (0, 3, -2, 2 * 129):
        _refused(B.RC_EINVAL, B.rc_paged_workspace, _pool(), m, 3, heads)
    two = _rows(2)
    for q, k, v, out in [(_rows(data=0), two, two, _rows()), (_rows(data=P + 2), two, two, _rows()),
                         (_rows(), two, two, _rows(tok=0)), (_rows(), two, two, _rows(head=32)),
                         (_rows(), two, two, _rows(6)), (_rows(), _rows(4), two, _rows()),
                         (_rows(), two, _rows(1), _rows()), (_rows(tok=-256), two, two, _rows()),
                         (_rows(tok=260), two, two, _rows()), (_rows(-1), two, two, _rows(-1))]:
        _refused(B.RC_EINVAL, B.rc_paged_append, _pool(), None, 3, q, k, v, out)


@pytest.mark.parametrize("over", [dict(n_axes=0), dict(n_axes=4), dict(n_axes=-1), dict(pairing=2), dict(pos=0),
                                  dict(pos=P + 2), dict(pairs=(16, 17, 0)), dict(pairs=(-1, 33, 0)),
                                  dict(n_pos=(0, 4, 0)), dict(table=(0, P, 0)), dict(table=(P, P + 4, 0))],
                         ids=lambda o: next(iter(o)) + str(next(iter(o.values()))))
def test_bad_rotations_are_refused(over):
    two = (B.rc_rows * 2)(_rows(), B.rc_rows())
    _refused(B.RC_EINVAL, B.rc_rope_axes, _rope(**over), B.RC_BF16, 3, 64, 0, two, two)
    if over != dict(n_axes=0):  # the append takes that as no rotation
        k = _rows(2)
        _refused(B.RC_EINVAL, B.rc_paged_append, _pool(), _rope(**over), 3, _rows(), k, k, _rows())


def test_bad_rotated_tensors_are_refused():
    ok, none = _rows(), B.rc_rows()
    for dtype, d, x, y in [(3, 64, (ok, none), (ok, none)), (0, 96, (ok, none), (ok, none)),
                           (0, 64, (ok, none), (_rows(3), none)), (0, 64, (ok, ok), (ok, none)),
                           (0, 64, (_rows(data=0), none), (ok, none)), (0, 64, (ok, none), (_rows(tok=0), none)),
                           (2, 64, (_rows(data=P + 8), none), (ok, none)), (2, 64, (_rows(tok=258), none), (ok, none))]:
        _refused(B.RC_EINVAL, B.rc_rope_axes, _rope(), dtype, 3, d, 0, (B.rc_rows * 2)(*x), (B.rc_rows * 2)(*y))
    two = (B.rc_rows * 2)(ok, none)
    for n in (-1, (1 << 30) + 1):
        _refused(B.RC_EINVAL, B.rc_rope_axes, _rope(), 0, n, 64, 0, two, two)
    lib, row = B.lib(), _rows()
    assert lib.rc_rope_axes(None, 0, 3, 64, 0, two, two, None, None) == B.RC_EINVAL
    assert lib.rc_paged_append(None, None, 3, row, row, row, row, None, None) == B.RC_EINVAL
    assert lib.rc_paged_attention(None, None, 3, row, row, None, None, 0, None, None) == B.RC_EINVAL
    pool, mask = _pool(), B.rc_paged_mask(frame_seqlen=1)
    assert lib.rc_paged_workspace(pool, mask, 3, 4, None) == B.RC_EINVAL
    assert lib.rc_paged_attention(pool, mask, 3, None, row, None, None, 0, None, None) == B.RC_EINVAL


def test_python_functions_refuse_host_tensors():
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    pool = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    table = torch.zeros(1, 3, dtype=torch.int32)
    tables = paged.rope_tables((4,), (32,), device="cpu")
    with pytest.raises(ValueError):
        paged.rope_axes(x, torch.zeros(3, 1, dtype=torch.int32), tables)
    with pytest.raises(ValueError):
        paged.paged_append(x, x, x, pool, pool, i, i[:1], table)
    with pytest.raises(ValueError):
        paged.paged_attention(x, pool, pool, i, i[:1], table)
    with pytest.raises(ValueError):
        paged.prefix_attention(x, pool, pool, i, 0, i, i[:1], table)
    with pytest.raises(ValueError):
        paged.rope_tables((4, 4), (32,), device="cpu")


def test_rope_tables_match_the_librarys():
    cfg = B.rc_config_init(1, 2, 128, 1560, 1, 6)
    cfg.grid_h, cfg.grid_w, cfg.t_max = 30, 52, 400
    h = B.rc_cache_create(cfg, 0, 0)
    try:
        tables = paged.rope_tables((400, 30, 52), (22, 21, 21), device="cpu")
        for axis, t in enumerate(tables):
            assert np.max(np.abs(B.rc_rope_table(h, axis) - t.numpy().ravel())) <= 2.0 ** -24
    finally:
        B.rc_cache_destroy(h)


@pytest.mark.parametrize("name", ["cu_q", "kv_len", "page_table", "prefix_table", "status", "lse"])
def test_words_off_their_alignment_are_refused(name):
    p = _pool(**({name: P + 2} if name in ("cu_q", "kv_len", "page_table") else {}))
    m = B.rc_paged_mask(frame_seqlen=1, max_q=1)
    if name == "prefix_table":
        m = B.rc_paged_mask(frame_seqlen=1, max_q=1, prefix_len=5, prefix_table=P + 2, prefix_pages=1)
    status, lse = (P + 2 if name == n else 0 for n in ("status", "lse"))
    two = _rows(2)
    _refused(B.RC_EINVAL, B.rc_paged_attention, p, m, 3, _rows(), _rows(), lse, P, 1 << 30, status)
    if name not in ("prefix_table", "lse"):
        _refused(B.RC_EINVAL, B.rc_paged_append, p, None, 3, _rows(), two, two, _rows(), status)
    if name == "status":
        one = (B.rc_rows * 2)(_rows(), B.rc_rows())
        _refused(B.RC_EINVAL, B.rc_rope_axes, _rope(), B.RC_BF16, 3, 64, 0, one, one, status)


def test_written_rows_that_overlap_are_refused():
    """Also where each stride is at least a row: [3][4] rows of 64, a token's heads reaching into the next token's."""
    two, one = _rows(2), (B.rc_rows * 2)(_rows(), B.rc_rows())
    m = B.rc_paged_mask(frame_seqlen=1, max_q=1)
    for tok, head in ((64, 64), (128, 64), (192, 64), (64, 128), (64, 184), (200, 72)):
        r = B.rc_rows(P, tok, head, 4)
        _refused(B.RC_EINVAL, B.rc_paged_attention, _pool(), m, 3, _rows(), r, 0, P, 1 << 30)
        _refused(B.RC_EINVAL, B.rc_paged_append, _pool(), None, 3, _rows(), two, two, r)
        _refused(B.RC_EINVAL, B.rc_rope_axes, _rope(), B.RC_BF16, 3, 64, 0, one, (B.rc_rows * 2)(r, B.rc_rows()))
    # the pool an append writes: pages closer than a page, heads closer than 16 rows
    for st in ((1024, 1024, 64), (2048, 512, 64), (1088, 1024, 128)):
        for name in ("k_stride", "v_stride"):
            _refused(B.RC_EINVAL, B.rc_paged_append, _pool(**{name: st}), None, 3, _rows(), two, two, _rows())


def test_written_rows_in_every_nesting_pass_the_checks():
    """Refused only for the workspace, which is looked at after the rows (or, without a GPU, for that)."""
    m = B.rc_paged_mask(frame_seqlen=1, max_q=100)  # many rows: a workspace is needed
    for tok, head in ((256, 64), (64, 192), (320, 72), (512, 128), (72, 256)):
        with pytest.raises(B.RcError, match="workspace|device attribute"):
            B.rc_paged_attention(_pool(), m, 3, _rows(), B.rc_rows(P, tok, head, 4), 0, 0, 0)


def test_tangents_and_traces_are_refused_on_any_device():
    import torch.autograd.forward_ad as fw

    x = torch.zeros(3, 2, 64)
    pos, tables = torch.zeros(3, 1, dtype=torch.int32), paged.rope_tables((4,), (32,), device="cpu")
    pool, i, table = torch.zeros(4, 2, 16, 64), torch.zeros(2, dtype=torch.int32), torch.zeros(1, 3, dtype=torch.int32)
    calls = [lambda t: paged.rope_axes(t, pos, tables), lambda t: paged.paged_append(None, t, x, pool, pool, i, i[:1], table),
             lambda t: paged.paged_attention(t, pool, pool, i, i[:1], table)]
    for call in calls:
        with fw.dual_level(), pytest.raises(ValueError, match="forward-mode"):
            call(fw.make_dual(x, x))
        with pytest.raises(ValueError, match="trace"):
            torch.jit.trace(call, (x,), check_trace=False)
        with pytest.raises(ValueError, match="CUDA"):
            call(x)


def test_tables_that_ask_for_a_gradient_are_refused_on_any_device():
    x, pos = torch.zeros(3, 2, 64), torch.zeros(3, 1, dtype=torch.int32)
    learned = (paged.rope_tables((4,), (32,), device="cpu")[0].requires_grad_(True),)
    pool, i, table = torch.zeros(4, 2, 16, 64), torch.zeros(2, dtype=torch.int32), torch.zeros(1, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="tables"):
        paged.rope_axes(x, pos, learned)
    with pytest.raises(ValueError, match="tables"):
        paged.paged_append(None, x, x, pool, pool, i, i[:1], table, pos=pos, tables=learned)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        paged.rope_axes(x, pos, learned)


def test_negated_views_are_refused_on_any_device():
    x, pos = torch._neg_view(torch.zeros(3, 2, 64)), torch.zeros(3, 1, dtype=torch.int32)
    pool, i, table = torch.zeros(4, 2, 16, 64), torch.zeros(2, dtype=torch.int32), torch.zeros(1, 3, dtype=torch.int32)
    for call in (lambda: paged.rope_axes(x, pos, paged.rope_tables((4,), (32,), device="cpu")),
                 lambda: paged.paged_append(None, x, x, pool, pool, i, i[:1], table),
                 lambda: paged.paged_attention(x, pool, pool, i, i[:1], table)):
        with pytest.raises(ValueError, match="negated"):
            call()


def test_a_tensor_given_for_two_outputs_is_refused():
    one, two = _rows(), _rows(2)
    for fn, args in ((B.rc_rope_axes, (_rope(), B.RC_BF16, 3, 64, 0, (B.rc_rows * 2)(one, one), (B.rc_rows * 2)(one, one))),
                     (B.rc_paged_append, (_pool(), None, 3, one, two, two, one))):
        with pytest.raises(B.RcError, match="are one"):
            fn(*args)
