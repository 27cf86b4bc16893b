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

import ctypes
from typing import Optional, Sequence, Tuple, Union

import torch

from . import binding as B

_DTYPES = {torch.bfloat16: B.RC_BF16, torch.float16: B.RC_F16, torch.float32: B.RC_F32}
_PAIRING = {"adjacent": B.RC_PAIR_ADJACENT, "halves": B.RC_PAIR_HALVES}
_status = {}


def _word(device: torch.device) -> torch.Tensor:
    """The device's status word, shared by every call of this module."""
    w = _status.get(device.index)
    if w is None:
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("run one paged call on this device before capturing one")
        w = torch.zeros(1, dtype=torch.int32, device=device)
        torch.cuda.current_stream(device).synchronize()
        _status[device.index] = w
    return w


def device_status(device: Union[torch.device, str, int, None] = None) -> None:
    """Waits for the device and raises RcError if a call of this module since
    the last check met a value out of range (RC_ERANGE) or a wait that gave up
    (RC_ETIMEOUT)."""
    device = torch.device("cuda" if device is None else device)
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    torch.cuda.synchronize(device)
    w = _status.get(device.index)
    code = int(w.item()) if w is not None else 0
    if code:
        w.zero_()
        torch.cuda.synchronize(device)
        what = {B.RC_ERANGE: "a position, page or length was out of range",
                B.RC_ETIMEOUT: "a device-side wait gave up"}.get(code, "unknown")
        raise B.RcError(code, what)


def _device_of(*tensors) -> torch.device:
    dev = None
    for t in tensors:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("paged operators take CUDA tensors")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"tensors on {dev} and {t.device}")
    return dev


class _On:
    """Makes a device current for one call."""

    def __init__(self, device):
        self.index = device.index

    def __enter__(self):
        self.prev = torch.cuda.current_device()
        if self.prev != self.index:
            torch.cuda.set_device(self.index)

    def __exit__(self, *exc):
        if self.prev != self.index:
            torch.cuda.set_device(self.prev)


def _rows(t: torch.Tensor, what: str) -> B.rc_rows:
    if t.dim() != 3 or (t.stride(2) != 1 and t.shape[2] > 1):
        raise ValueError(f"{what} must be [tokens, heads, head_dim] with a contiguous last dimension")
    return B.rc_rows(t.data_ptr(), t.stride(0), t.stride(1), t.shape[1])


def _int32(t: torch.Tensor, dims: int, what: str) -> torch.Tensor:
    if t.dtype != torch.int32 or t.dim() != dims or (t.numel() > 1 and t.stride(-1) != 1 and t.shape[-1] > 1):
        raise ValueError(f"{what} must be an int32 tensor of {dims} dimension(s), contiguous in the last")
    return t


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


def _rope(pos, tables, pairing, n_tok, head_dim) -> B.rc_rope:
    if pairing not in _PAIRING:
        raise ValueError("pairing must be 'adjacent' or 'halves'")
    tables = tuple(tables)
    n = len(tables)
    if not 1 <= n <= 3:
        raise ValueError("1 to 3 rotation tables")
    if pos.dtype != torch.int32 or pos.shape != (n_tok, n) or not pos.is_contiguous():
        raise ValueError("pos must be a contiguous int32 tensor [tokens, axes]")
    r = B.rc_rope(pos=pos.data_ptr(), n_axes=n, pairing=_PAIRING[pairing])
    total = 0
    for a, t in enumerate(tables):
        if t.dtype != torch.float32 or t.dim() != 3 or t.shape[2] != 2 or not t.is_contiguous():
            raise ValueError("a rotation table is a contiguous fp32 tensor [positions, pairs, 2]")
        r.table[a], r.n_pos[a], r.pairs[a] = t.data_ptr(), t.shape[0], t.shape[1]
        total += t.shape[1]
    if total != head_dim // 2:
        raise ValueError("the tables' pairs must sum to head_dim / 2")
    return r


def _turn(xs, outs, pos, tables, pairing, inverse):
    x = xs[0]
    dev = _device_of(*xs, *outs, pos, *tables)
    if x.dtype not in _DTYPES:
        raise ValueError("rope_axes takes bf16, fp16 or fp32")
    n_tok, _, d = x.shape
    for t in (*xs, *outs):
        if t.dtype != x.dtype or t.dim() != 3 or t.shape[0] != n_tok or t.shape[2] != d:
            raise ValueError("tensors differ in type, tokens or head_dim")
    rope = _rope(pos, tables, pairing, n_tok, d)
    rx, ry = (B.rc_rows * 2)(), (B.rc_rows * 2)()
    for i, (a, o) in enumerate(zip(xs, outs)):
        if a.shape != o.shape:
            raise ValueError("an output differs in shape")
        rx[i], ry[i] = _rows(a, "x"), _rows(o, "out")
    with _On(dev):
        B.rc_rope_axes(rope, _DTYPES[x.dtype], n_tok, d, int(inverse), rx, ry, _word(dev).data_ptr(),
                       torch.cuda.current_stream(dev).cuda_stream)


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
        outs = tuple(torch.empty(x.shape, dtype=x.dtype, device=x.device) for x in xs)
        _turn(xs, outs, pos, tables, pairing, inverse)
        return outs

    @staticmethod
    def backward(ctx, *grads):
        pos, *tables = ctx.saved_tensors
        need = [i for i in range(len(grads)) if ctx.needs_input_grad[4 + i] and grads[i] is not None]
        out = [None] * len(grads)
        if need:
            turned = _RopeAxes.apply(pos, tuple(tables), ctx.pairing, not ctx.inverse,
                                     *(_readable(grads[i]) for i in need))
            for i, g in zip(need, turned):
                out[i] = g
        return (None, None, None, None, *out)


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
        _turn(xs, outs, pos, tuple(tables), pairing, inverse)
    elif torch.is_grad_enabled() and any(t.requires_grad for t in xs):
        outs = _RopeAxes.apply(pos, tuple(tables), pairing, inverse, *xs)
    else:
        outs = tuple(torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in xs)
        _turn(xs, outs, pos, tuple(tables), pairing, inverse)
    return outs if pair else outs[0]


def _paged(k_pages, v_pages, cu_q, kv_len, page_table) -> B.rc_paged:
    if k_pages.dim() != 4 or v_pages.shape != k_pages.shape or v_pages.dtype != k_pages.dtype:
        raise ValueError("k_pages and v_pages must be [n_pages, kv_heads, page_size, head_dim] alike")
    if k_pages.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("pages are bf16 or fp16")
    if k_pages.stride(3) != 1 or v_pages.stride(3) != 1:
        raise ValueError("the pages' last dimension must be contiguous")
    _int32(cu_q, 1, "cu_q")
    _int32(kv_len, 1, "kv_len")
    _int32(page_table, 2, "page_table")
    n = kv_len.shape[0]
    if cu_q.shape[0] != n + 1 or page_table.shape[0] != n:
        raise ValueError("cu_q has one entry more than kv_len, page_table as many rows")
    st = ctypes.c_int64 * 3
    s = k_pages.shape
    return B.rc_paged(k_pages.data_ptr(), v_pages.data_ptr(), st(*k_pages.stride()[:3]), st(*v_pages.stride()[:3]),
                      s[0], s[2], s[1], s[3], _DTYPES[k_pages.dtype], n, cu_q.data_ptr(), kv_len.data_ptr(),
                      page_table.data_ptr(), page_table.stride(0), page_table.shape[1])


def _no_grad(*tensors) -> None:
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
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
    dev = _device_of(q, k, v, k_pages, v_pages, cu_q, kv_len, page_table, pos, q_out, *(tables or ()))
    if (pos is None) != (tables is None):
        raise ValueError("pos and tables go together")
    if k.dim() != 3 or v.shape != k.shape:
        raise ValueError("k and v must be [tokens, kv_heads, head_dim] alike")
    n_tok, _, d = k.shape
    if d != k_pages.shape[-1]:
        raise ValueError("k and v differ from the pages in head_dim")
    paged = _paged(k_pages, v_pages, cu_q, kv_len, page_table)
    for t in (q, k, v, q_out):
        if t is not None and t.dtype != k_pages.dtype:
            raise ValueError("q, k, v and the pages must have one type")
    if q is not None:
        if q.dim() != 3 or q.shape[0] != n_tok or q.shape[2] != d:
            raise ValueError("q must be [tokens, q_heads, head_dim] of k's tokens and head_dim")
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        elif q_out.shape != q.shape:
            raise ValueError("q_out differs from q in shape")
        rq, ro = _rows(q, "q"), _rows(q_out, "q_out")
    else:
        if q_out is not None:
            raise ValueError("q_out without q")
        rq, ro = B.rc_rows(), B.rc_rows()
    rope = None if pos is None else _rope(pos, tables, pairing, n_tok, d)
    with _On(dev):
        B.rc_paged_append(paged, rope, n_tok, rq, _rows(k, "k"), _rows(v, "v"), ro, _word(dev).data_ptr(),
                          torch.cuda.current_stream(dev).cuda_stream)
    return q_out


def _attend(q, k_pages, v_pages, cu_q, kv_len, page_table, max_q, frame_seqlen, sink_frames, window_frames, scale,
            out, return_lse, prefix_table, prefix_len):
    _no_grad(q, k_pages, v_pages, out)
    dev = _device_of(q, k_pages, v_pages, cu_q, kv_len, page_table, prefix_table, out)
    paged = _paged(k_pages, v_pages, cu_q, kv_len, page_table)
    if q.dtype != k_pages.dtype or q.dim() != 3 or q.shape[2] != k_pages.shape[3]:
        raise ValueError("q must be [tokens, q_heads, head_dim] of the pages' type and head_dim")
    n_tok, heads, _ = q.shape
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=dev)
    elif out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("out differs from q in shape or type")
    lse = torch.empty((heads, n_tok), dtype=torch.float32, device=dev) if return_lse else None
    mask = B.rc_paged_mask(frame_seqlen, sink_frames, window_frames, n_tok if max_q is None else max_q,
                           0.0 if scale is None else scale)
    if prefix_table is not None:
        _int32(prefix_table, 1, "prefix_table")
        mask.prefix_len, mask.prefix_table = prefix_len, prefix_table.data_ptr()
        mask.prefix_pages = prefix_table.shape[0]
    if scale is not None and not scale > 0:
        raise ValueError("scale must be positive")
    with _On(dev):
        n = B.rc_paged_workspace(paged, mask, n_tok, heads)
        work = torch.empty(n, dtype=torch.uint8, device=dev)
        B.rc_paged_attention(paged, mask, n_tok, _rows(q, "q"), _rows(out, "out"),
                             lse.data_ptr() if return_lse else 0, work.data_ptr(), n, _word(dev).data_ptr(),
                             torch.cuda.current_stream(dev).cuda_stream)
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
