"""Many streams in one pool of pages: rotary positions over several axes, the
append that rotates keys into the pages, and attention over pages.

Where ``RollingKVCache`` holds one stream in a ring, these functions serve a
batch of streams whose keys and values live in pages of one pool,
``k_pages`` and ``v_pages`` ([n_pages, kv_heads, page_size, head_dim], any
strides with a contiguous last dimension). Token i of sequence b is row
``i % page_size`` of page ``page_table[b, i // page_size]``. Queries are packed:
sequence b owns rows ``cu_q[b]:cu_q[b + 1]``, its last tokens, and ``kv_len[b]``
counts its tokens in the pages, those among them. A decoding step is::

    q = paged_append(q, k, v, k_pages, v_pages, cu_q, kv_len, page_table, pos=pos, tables=tables)
    out = paged_attention(q, k_pages, v_pages, cu_q, kv_len, page_table, max_q=1)

Everything runs in librc.so's kernels on the current stream of the tensors'
device; a call allocates its outputs and its workspace from torch's caching allocator, so that calls on
several streams and captured graphs do not share scratch. Lengths, tables and
positions are int32 device tensors read when the kernels run. What they hold out of range
is never followed; ``device_status`` reports it.
"""
from __future__ import annotations

from typing import Optional, Sequence, Tuple, Union

import torch

from . import binding as B

_DTYPES = {torch.bfloat16: B.RC_BF16, torch.float16: B.RC_F16, torch.float32: B.RC_F32}
_PAIRING = {"adjacent": B.RC_PAIR_ADJACENT, "halves": B.RC_PAIR_HALVES}
_NO_ROWS = B.PACK_ROWS.pack(0, 0, 0, 0)
_status = {}  # device index -> (status word, its address), one per device for every call of this module
_work_bytes = {}  # sizes of a call -> bytes of workspace


def _word(index: int) -> int:
    """Address of the device's status word."""
    w = _status.get(index)
    if w is None:
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("run one paged call on this device before capturing one")
        t = torch.zeros(1, dtype=torch.int32, device=torch.device("cuda", index))
        torch.cuda.current_stream(index).synchronize()
        w = _status[index] = (t, t.data_ptr())
    return w[1]


def device_status(device: Union[torch.device, str, int, None] = None) -> None:
    """Waits for the device and raises RcError if a call of this module since
    the last check met a value out of range (RC_ERANGE) or a wait that gave up
    (RC_ETIMEOUT)."""
    device = torch.device("cuda" if device is None else device)
    index = torch.cuda.current_device() if device.index is None else device.index
    torch.cuda.synchronize(index)
    w = _status.get(index)
    code = int(w[0].item()) if w is not None else 0
    if code:
        w[0].zero_()
        torch.cuda.synchronize(index)
        what = {B.RC_ERANGE: "a position, page or length was out of range",
                B.RC_ETIMEOUT: "a device-side wait gave up"}.get(code, "unknown")
        raise B.RcError(code, what)


def _index_of(first: torch.Tensor, *others) -> int:
    """The one CUDA device that every tensor is on."""
    index = first.get_device()
    for t in others:
        if t is not None and t.get_device() != index:
            raise ValueError("tensors on more than one device")
    if index < 0:
        raise ValueError("paged operators take CUDA tensors")
    return index


def _launch(index: int, fn, *args) -> None:
    """fn(*args, status, stream) with the tensors' device current, on its current stream."""
    if index == torch._C._cuda_getDevice():
        fn(*args, _word(index), torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            fn(*args, _word(index), torch._C._cuda_getCurrentRawStream(index))


def _rows(t: torch.Tensor, what: str) -> bytes:
    a, h, e = t.stride()
    if e != 1:
        raise ValueError(f"{what} must have a contiguous last dimension")
    return B.PACK_ROWS.pack(t.data_ptr(), a, h, t.shape[1])


def rope_tables(max_pos: Sequence[int], pairs: Sequence[int], theta: float = 10000.0,
                device: Union[torch.device, str] = "cuda") -> Tuple[torch.Tensor, ...]:
    """(cos, sin) tables [max_pos[a], pairs[a], 2] fp32 of ``len(pairs)`` axes:
    position p of axis a turns pair j by p * theta^(-j / pairs[a]), as rc_step's
    tables do (angles in fp64, rounded once)."""
    if len(max_pos) != len(pairs) or not 1 <= len(pairs) <= 3:
        raise ValueError("one max_pos and one pairs entry for each of 1 to 3 axes")
    out = []
    for n, p in zip(max_pos, pairs):
        a = (torch.arange(n, dtype=torch.float64)[:, None]
             * theta ** (-torch.arange(p, dtype=torch.float64) / max(p, 1))[None])
        out.append(torch.stack((a.cos(), a.sin()), -1).float().to(device))
    return tuple(out)


def _rope(pos, tables, pairing, n_tok, head_dim) -> bytes:
    n = len(tables)
    if pairing not in _PAIRING:
        raise ValueError("pairing must be 'adjacent' or 'halves'")
    if not 1 <= n <= 3:
        raise ValueError("1 to 3 rotation tables")
    if pos.dtype is not torch.int32 or pos.shape != (n_tok, n) or not pos.is_contiguous():
        raise ValueError("pos must be a contiguous int32 tensor [tokens, axes]")
    ptr, rows, pairs = [0, 0, 0], [0, 0, 0], [0, 0, 0]
    for a, t in enumerate(tables):
        if t.dtype is not torch.float32 or t.dim() != 3 or not t.is_contiguous():
            raise ValueError("a rotation table is a contiguous fp32 tensor [positions, pairs, 2]")
        rows[a], pairs[a], two = t.shape
        if two != 2:
            raise ValueError("a rotation table is a contiguous fp32 tensor [positions, pairs, 2]")
        ptr[a] = t.data_ptr()
    if sum(pairs) * 2 != head_dim:
        raise ValueError("the tables' pairs must sum to head_dim / 2")
    return B.PACK_ROPE.pack(pos.data_ptr(), *ptr, *rows, *pairs, n, _PAIRING[pairing])


def _turn(xs, outs, pos, tables, pairing, inverse):
    x = xs[0]
    index = _index_of(*xs, *outs, pos, *tables)
    dt = x.dtype
    if dt not in _DTYPES:
        raise ValueError("rope_axes takes bf16, fp16 or fp32")
    if x.dim() != 3:
        raise ValueError("x must be [tokens, heads, head_dim]")
    n_tok, _, d = x.shape
    rx = ry = b""
    for a, o in zip(xs, outs):
        s = a.shape
        if a.dtype is not dt or o.dtype is not dt or len(s) != 3 or s[0] != n_tok or s[2] != d or o.shape != s:
            raise ValueError("tensors differ in type, tokens or head_dim")
        rx += _rows(a, "x")
        ry += _rows(o, "out")
    if len(xs) == 1:
        rx += _NO_ROWS
        ry += _NO_ROWS
    _launch(index, B.rc_rope_axes, _rope(pos, tables, pairing, n_tok, d), _DTYPES[dt], n_tok, d, inverse, rx, ry)


def _new_like(t: torch.Tensor) -> torch.Tensor:
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


def _readable(t: torch.Tensor) -> torch.Tensor:
    """The tensor itself where the kernels can read it, else a contiguous copy (an autograd gradient may be
    expanded or sliced at any offset)."""
    size = 16 // t.element_size()
    if (t.stride(2) == 1 and t.stride(0) % size == 0 and t.stride(1) % size == 0 and t.stride(0) >= 0
            and t.stride(1) >= 0 and t.data_ptr() % 16 == 0):
        return t
    return t.clone(memory_format=torch.contiguous_format)


class _RopeAxes(torch.autograd.Function):
    @staticmethod
    def forward(ctx, pos, tables, pairing, inverse, *xs):
        ctx.save_for_backward(pos, *tables)
        ctx.pairing, ctx.inverse = pairing, inverse
        ctx.set_materialize_grads(False)
        outs = tuple(_new_like(x) for x in xs)
        _turn(xs, outs, pos, tables, pairing, inverse)
        return outs

    @staticmethod
    def backward(ctx, *grads):
        pos, *tables = ctx.saved_tensors
        need = [i for i, g in enumerate(grads) if g is not None and ctx.needs_input_grad[4 + i]]
        out = [None] * len(grads)
        if need:
            gs = tuple(_readable(grads[i]) for i in need)
            for i, g in zip(need, _turned(gs, pos, tuple(tables), ctx.pairing, not ctx.inverse)):
                out[i] = g
        return (None, None, None, None, *out)


def _turned(xs, pos, tables, pairing, inverse):
    if torch.is_grad_enabled() and any(t.requires_grad for t in xs):
        return _RopeAxes.apply(pos, tables, pairing, inverse, *xs)
    outs = tuple(_new_like(t) for t in xs)
    _turn(xs, outs, pos, tables, pairing, inverse)
    return outs


def rope_axes(x, pos: torch.Tensor, tables: Sequence[torch.Tensor], *, pairing: str = "adjacent",
              inverse: bool = False, out=None):
    """Turns heads by rotary positions over 1 to 3 axes (time, height, width).

    x: [tokens, heads, head_dim] (head_dim 64 or 128; bf16, fp16 or fp32) or a
    pair of such tensors (queries and keys) for one launch. pos: [tokens, axes]
    int32; tables: one [positions, pairs, 2] table of (cos, sin) per axis (``rope_tables``), whose
    pairs sum to head_dim / 2. ``pairing``: pair m turns elements (2m, 2m + 1)
    ("adjacent") or (m, m + head_dim / 2) ("halves"). ``inverse`` turns back.
    Differentiable in x (the gradient is the turn back). With ``out`` (a tensor
    or a pair; x itself for in place) the result is written there, outside autograd.
    """
    pair = isinstance(x, (tuple, list))
    xs = tuple(x) if pair else (x,)
    if not 1 <= len(xs) <= 2:
        raise ValueError("one tensor or a pair")
    if out is not None:
        outs = tuple(out) if pair else (out,)
        if len(outs) != len(xs):
            raise ValueError("one out for each x")
        if torch.is_grad_enabled() and any(t.requires_grad for t in (*xs, *outs)):
            raise ValueError("out= takes no part in autograd; call it under torch.no_grad()")
        _turn(xs, outs, pos, tuple(tables), pairing, bool(inverse))
    else:
        outs = _turned(xs, pos, tuple(tables), pairing, bool(inverse))
    return outs if pair else outs[0]


def _paged(k_pages, v_pages, cu_q, kv_len, page_table) -> bytes:
    s = k_pages.shape
    dt = k_pages.dtype
    if len(s) != 4 or v_pages.shape != s or v_pages.dtype is not dt:
        raise ValueError("k_pages and v_pages must be [n_pages, kv_heads, page_size, head_dim] alike")
    if dt is not torch.bfloat16 and dt is not torch.float16:
        raise ValueError("pages are bf16 or fp16")
    if cu_q.dtype is not torch.int32 or kv_len.dtype is not torch.int32 or page_table.dtype is not torch.int32:
        raise ValueError("cu_q, kv_len and page_table must be int32")
    if cu_q.dim() != 1 or kv_len.dim() != 1 or page_table.dim() != 2:
        raise ValueError("cu_q [n + 1], kv_len [n] and page_table [n, pages]")
    n, width = page_table.shape
    if kv_len.shape[0] != n or cu_q.shape[0] != n + 1:
        raise ValueError("cu_q has one entry more than kv_len, page_table as many rows")
    ks, vs, (row, entry) = k_pages.stride(), v_pages.stride(), page_table.stride()
    if ks[3] != 1 or vs[3] != 1 or (entry != 1 and width > 1) or not (cu_q.is_contiguous() and kv_len.is_contiguous()):
        raise ValueError("pages must have a contiguous last dimension; cu_q, kv_len and rows of page_table too")
    return B.PACK_PAGED.pack(k_pages.data_ptr(), v_pages.data_ptr(), ks[0], ks[1], ks[2], vs[0], vs[1], vs[2], s[0],
                             s[2], s[1], s[3], _DTYPES[dt], n, cu_q.data_ptr(), kv_len.data_ptr(),
                             page_table.data_ptr(), row, width)


def _no_grad(*tensors) -> None:
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                raise ValueError("the paged cache serves; it has no gradient (call it under torch.no_grad())")


def paged_append(q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor,
                 v_pages: torch.Tensor, cu_q: torch.Tensor, kv_len: torch.Tensor, page_table: torch.Tensor, *,
                 pos: Optional[torch.Tensor] = None, tables: Optional[Sequence[torch.Tensor]] = None,
                 pairing: str = "adjacent", q_out: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """Appends a batch's new tokens to its pages, turning queries and keys by
    their rotary positions on the way (see ``rope_axes``; without ``pos`` and
    ``tables`` nothing turns).

    q [tokens, q_heads, d] (or None), k, v [tokens, kv_heads, d], strided as they
    come from a fused projection; ``kv_len`` counts the new tokens already.
    Returns the turned queries (``q_out`` if given; q itself for in place). Two
    tokens of one call must not share a place.
    """
    _no_grad(q, k, v, k_pages, v_pages, q_out)
    if (pos is None) != (tables is None):
        raise ValueError("pos and tables go together")
    index = _index_of(k, v, k_pages, v_pages, cu_q, kv_len, page_table, q, q_out, pos, *(tables or ()))
    shape, dt = k.shape, k_pages.dtype
    if len(shape) != 3 or v.shape != shape or shape[2] != k_pages.shape[-1]:
        raise ValueError("k and v must be [tokens, kv_heads, head_dim] alike, of the pages' head_dim")
    n_tok, _, d = shape
    paged = _paged(k_pages, v_pages, cu_q, kv_len, page_table)
    if k.dtype is not dt or v.dtype is not dt:
        raise ValueError("q, k, v and the pages must have one type")
    rq = ro = _NO_ROWS
    if q is not None:
        sq = q.shape
        if q.dtype is not dt or len(sq) != 3 or sq[0] != n_tok or sq[2] != d:
            raise ValueError("q must be [tokens, q_heads, head_dim] of k's type, tokens and head_dim")
        if q_out is None:
            q_out = _new_like(q)
        elif q_out.shape != sq or q_out.dtype is not dt:
            raise ValueError("q_out differs from q in shape or type")
        rq, ro = _rows(q, "q"), _rows(q_out, "q_out")
    elif q_out is not None:
        raise ValueError("q_out without q")
    rope = None if pos is None else _rope(pos, tables, pairing, n_tok, d)
    _launch(index, B.rc_paged_append, paged, rope, n_tok, rq, _rows(k, "k"), _rows(v, "v"), ro)
    return q_out


def _attend(q, k_pages, v_pages, cu_q, kv_len, page_table, max_q, frame_seqlen, sink_frames, window_frames, scale,
            out, return_lse, prefix_table, prefix_len):
    _no_grad(q, k_pages, v_pages, out)
    index = _index_of(q, k_pages, v_pages, cu_q, kv_len, page_table, prefix_table, out)
    shape, pool, dt = q.shape, k_pages.shape, q.dtype
    paged = _paged(k_pages, v_pages, cu_q, kv_len, page_table)
    if dt is not k_pages.dtype or len(shape) != 3 or shape[2] != pool[3]:
        raise ValueError("q must be [tokens, q_heads, head_dim] of the pages' type and head_dim")
    if scale is None:
        scale = 0.0
    elif not scale > 0:
        raise ValueError("scale must be positive")
    n_tok, heads, _ = shape
    if out is None:
        out = _new_like(q)
    elif out.shape != shape or out.dtype is not dt:
        raise ValueError("out differs from q in shape or type")
    lse = q.new_empty((heads, n_tok), dtype=torch.float32) if return_lse else None
    if max_q is None:
        max_q = n_tok
    table = pages = 0
    if prefix_table is not None:
        if prefix_table.dtype is not torch.int32 or prefix_table.dim() != 1 or not prefix_table.is_contiguous():
            raise ValueError("prefix_table must be a contiguous int32 tensor [pages]")
        table, pages = prefix_table.data_ptr(), prefix_table.shape[0]
    mask = B.PACK_MASK.pack(frame_seqlen, sink_frames, window_frames, max_q, scale, prefix_len, table, pages)
    # the workspace's size depends on these alone; a call's other checks are the library's
    key = (index, n_tok, heads, pool, max_q, prefix_len > 0)
    n = _work_bytes.get(key)
    if n is None:
        with torch.cuda.device(index):
            n = B.rc_paged_workspace(paged, mask, n_tok, heads)
        if len(_work_bytes) >= 4096:
            _work_bytes.clear()
        _work_bytes[key] = n
    work = q.new_empty((n + 1) // 2)  # 16-bit elements
    _launch(index, B.rc_paged_attention, paged, mask, n_tok, _rows(q, "q"), _rows(out, "out"),
            lse.data_ptr() if return_lse else 0, work.data_ptr(), n)
    return (out, lse) if return_lse else out


def paged_attention(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, cu_q: torch.Tensor,
                    kv_len: torch.Tensor, page_table: torch.Tensor, *, max_q: Optional[int] = None,
                    frame_seqlen: int = 1, sink_frames: int = 0, window_frames: int = 0,
                    scale: Optional[float] = None, out: Optional[torch.Tensor] = None, return_lse: bool = False):
    """Attention of a batch's queries over their sequences' pages.

    q: [tokens, q_heads, head_dim]; query head h reads key head
    h // (q_heads // kv_heads). With f = position // frame_seqlen, a query sees
    the keys of frames <= its own (frame_seqlen 1: causal; a frame beyond every
    length: full attention); with ``window_frames`` only the last that many, its own
    included, and the first ``sink_frames``. Entries of pages that no query sees
    may hold anything. ``max_q``: the most queries of a sequence, where the
    caller knows it (default: all tokens); it chooses the kernel and must not be
    too small. Rows behind the last sequence are left as they are (uninitialised without ``out``).
    Returns out, or (out, lse [q_heads, tokens] fp32). A query that sees
    nothing gets zeros and -inf.
    """
    return _attend(q, k_pages, v_pages, cu_q, kv_len, page_table, max_q, frame_seqlen, sink_frames, window_frames,
                   scale, out, return_lse, None, 0)


def prefix_attention(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, prefix_table: torch.Tensor,
                     prefix_len: int, cu_q: torch.Tensor, kv_len: torch.Tensor, page_table: torch.Tensor, *,
                     max_q: Optional[int] = None, frame_seqlen: int = 1, sink_frames: int = 0,
                     window_frames: int = 0, scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                     return_lse: bool = False):
    """``paged_attention`` of a batch that shares a prefix: ``prefix_len`` tokens
    in the pages ``prefix_table`` [pages] lists, which every query sees whole
    before its own sequence. The prefix is read once and multiplied with all
    queries of the batch, instead of once per sequence. ``kv_len``,
    ``page_table``, frames and window count the sequences' own tokens.
    """
    if prefix_len < 1:
        raise ValueError("prefix_len must be positive")
    return _attend(q, k_pages, v_pages, cu_q, kv_len, page_table, max_q, frame_seqlen, sink_frames, window_frames,
                   scale, out, return_lse, prefix_table, prefix_len)
