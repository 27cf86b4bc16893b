"""Many streams in one pool of pages: rotary positions over several axes, the
append that rotates keys into the pages, and attention over pages.

Where ``RollingKVCache`` holds one stream in a ring, these functions serve a
batch of streams whose keys and values live in pages of one pool,
``k_pages`` and ``v_pages`` ([n_pages, kv_heads, page_size, head_dim], any
strides with a contiguous last dimension). Token i of sequence b is row
``i % page_size`` of page ``page_table[b, i // page_size]``. Queries are packed:
sequence b owns rows ``cu_q[b]:cu_q[b + 1]``, its last tokens, and ``kv_len[b]``
counts its tokens in the pages, those among them. A call takes up to 4096 sequences. A decoding step is::

    q = paged_append(q, k, v, k_pages, v_pages, cu_q, kv_len, page_table, pos=pos, tables=tables)
    out = paged_attention(q, k_pages, v_pages, cu_q, kv_len, page_table, max_q=1)

Everything runs in librc.so's kernels on the current stream of the tensors'
device; a call allocates its outputs and its workspace from torch's caching
allocator, so that calls on several streams and captured graphs do not share scratch. Lengths, tables and
positions are int32 device tensors read when the kernels run. What they hold out of range
is never followed; ``device_status`` reports it. Tensors with a forward-mode tangent, and calls under
torch.jit.trace or make_fx, are refused.
"""
from __future__ import annotations

import importlib
from typing import Optional, Sequence, Tuple, Union

import torch

from . import binding as B

_HALVES = {"adjacent": False, "halves": True}
_module = None


def _ext():
    """The torch extension over librc.so. Raises if it is missing: there is no fallback."""
    global _module
    if _module is None:
        try:
            _module = importlib.import_module("._paged", __package__)
        except ImportError as e:
            raise RuntimeError("rolling_kv_cache_b200/_paged.so is missing or does not load; build it with "
                               "python -m rolling_kv_cache_b200.build") from e
    return _module


def device_status(device: Union[torch.device, str, int, None] = None) -> None:
    """Waits for the device and raises RcError if a call of this module since
    the last check met a value out of range (RC_ERANGE) or a wait that gave up
    (RC_ETIMEOUT)."""
    device = torch.device("cuda" if device is None else device)
    index = torch.cuda.current_device() if device.index is None else device.index
    torch.cuda.synchronize(index)
    word = _ext().status_word(index)
    code = int(word.item()) if word is not None else 0
    if code:
        word.zero_()
        torch.cuda.synchronize(index)
        what = {B.RC_ERANGE: "a position, page or length was out of range",
                B.RC_ETIMEOUT: "a device-side wait gave up"}.get(code, "unknown")
        raise B.RcError(code, what)


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


def rope_axes(x, pos: torch.Tensor, tables: Sequence[torch.Tensor], *, pairing: str = "adjacent",
              inverse: bool = False, out=None):
    """Turns heads by rotary positions over 1 to 3 axes (time, height, width).

    x: [tokens, heads, head_dim] (head_dim 64 or 128; bf16, fp16 or fp32) or a
    pair of such tensors (queries and keys) for one launch. pos: [tokens, axes]
    int32; tables: one [positions, pairs, 2] table of (cos, sin) per axis (``rope_tables``), whose
    pairs sum to head_dim / 2. ``pairing``: pair m turns elements (2m, 2m + 1)
    ("adjacent") or (m, m + head_dim / 2) ("halves"). ``inverse`` turns back.
    Differentiable in x by backward passes (the gradient is the turn back), not in the tables. With ``out`` (a tensor
    or a pair that do not overlap; x itself for in place) the result is written there, outside autograd.
    A leaf whose earlier graph, made on another stream, is alive is refused while
    a CUDA graph is captured.
    """
    if pairing not in _HALVES:
        raise ValueError("pairing must be 'adjacent' or 'halves'")
    pair = isinstance(x, (tuple, list))
    y = _ext().rope_axes(x if pair else (x,), pos, tables, _HALVES[pairing], inverse,
                         out if pair or out is None else (out,))
    if out is not None:
        return out
    return tuple(y) if pair else y[0]


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
    tokens of one call must not share a place: its rows would be a mix of theirs.
    """
    if pairing not in _HALVES:
        raise ValueError("pairing must be 'adjacent' or 'halves'")
    y = _ext().append(q, k, v, k_pages, v_pages, cu_q, kv_len, page_table, pos, tables, _HALVES[pairing], q_out)
    return y if q_out is None else q_out


def paged_attention(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, cu_q: torch.Tensor,
                    kv_len: torch.Tensor, page_table: torch.Tensor, *, max_q: Optional[int] = None,
                    frame_seqlen: int = 1, sink_frames: int = 0, window_frames: int = 0,
                    scale: Optional[float] = None, out: Optional[torch.Tensor] = None, return_lse: bool = False):
    """Attention of a batch's queries over their sequences' pages.

    q: [tokens, q_heads, head_dim]; query head h reads key head
    h // (q_heads // kv_heads). With f = position // frame_seqlen, a query sees
    the keys of frames <= its own (frame_seqlen 1: causal; a frame beyond every
    length: full attention); with ``window_frames`` only the last that many, its own
    included, and the first ``sink_frames`` (0 without a window). ``scale``
    (default 1 / sqrt(head_dim)) lies in [1e-30, 1e30]. Rows of pages that no query of the call sees
    may hold anything. ``max_q``: the most queries of a sequence, where the
    caller knows it (default: all tokens); it chooses the kernel and must not be
    too small. ``out`` may be q itself. Rows behind the last sequence are left as they are (uninitialised without ``out``).
    Returns out, or (out, lse [q_heads, tokens] fp32). A query that sees
    nothing gets zeros and -inf.
    """
    o, lse = _ext().attention(q, k_pages, v_pages, cu_q, kv_len, page_table, max_q, frame_seqlen, sink_frames,
                              window_frames, scale, out, return_lse, None, 0)
    o = o if out is None else out
    return (o, lse) if return_lse else o


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
    if prefix_table is None:
        raise ValueError("prefix_attention needs a prefix_table")
    o, lse = _ext().attention(q, k_pages, v_pages, cu_q, kv_len, page_table, max_q, frame_seqlen, sink_frames,
                              window_frames, scale, out, return_lse, prefix_table, prefix_len)
    o = o if out is None else out
    return (o, lse) if return_lse else o
