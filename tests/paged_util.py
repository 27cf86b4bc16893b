"""Plain 64-bit forms of the paged operators, batches for their tests, and the bounds that their
arithmetic allows."""
import math

import torch

F64 = torch.float64
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def randn(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def turned(x, pos, tables, halves, inverse=False):
    """(the turned rows, |a| + |b| of each element's pair) in 64 bits."""
    cs = torch.cat([t.to(F64)[pos[:, a].long().clamp(0, t.shape[0] - 1)] for a, t in enumerate(tables)], 1)
    c, s = cs[:, None, :, 0], cs[:, None, :, 1] * (-1 if inverse else 1)
    x = x.detach().to(F64)
    a, b = x.chunk(2, -1) if halves else (x[..., 0::2], x[..., 1::2])
    y = (a * c - b * s, a * s + b * c)
    mag = a.abs() + b.abs()
    if halves:
        return torch.cat(y, -1), torch.cat((mag, mag), -1)
    return torch.stack(y, -1).flatten(-2), torch.stack((mag, mag), -1).flatten(-2)


def assert_turned(got, x, pos, tables, halves, inverse=False):
    """One rounding to the type (UNIT of the value) after two fp32 products and
    a sum (three roundings, each at most 2^-24 of |a| + |b|)."""
    want, mag = turned(x, pos, tables, halves, inverse)
    bound = UNIT[got.dtype] * want.abs() * (1 + 2.0 ** -20) + 3 * 2.0 ** -24 * mag
    if got.dtype == torch.float16:
        bound = bound + 2.0 ** -25  # half a step of the denormals
    err = (got.to(F64) - want).abs()
    assert bool((err <= bound).all()), float((err - bound).max())


class Batch:
    """Sequences with (queries, tokens) lengths, their pages drawn in random
    order from a pool whose unused rows hold `fill`."""

    def __init__(self, seed, lens, hq, hk, d, page, dtype=torch.bfloat16, fill=float("nan"), spare=2, pad=0,
                 nhd=False):
        g = self.gen = generator(seed)
        self.lens, self.hq, self.hk, self.d, self.page, self.dtype = lens, hq, hk, d, page, dtype
        need = [(n + page - 1) // page for _, n in lens]
        total = sum(need) + spare
        order = torch.randperm(total, generator=g, device="cuda").int().cpu()
        wide = max(need + [1]) + 1
        table = torch.full((len(lens), wide), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        self.free = order[at:].tolist()
        self.page_table = table.cuda()
        cu = [0]
        for q, _ in lens:
            cu.append(cu[-1] + q)
        self.cu = cu
        self.cu_q = torch.tensor(cu, dtype=torch.int32, device="cuda")
        self.kv_len = torch.tensor([n for _, n in lens], dtype=torch.int32, device="cuda")
        self.n_tok = cu[-1] + pad
        self.q = randn(g, self.n_tok, hq, d, dtype=dtype)
        shape = (total, page, hk, d) if nhd else (total, hk, page, d)
        self.k_pages = torch.full(shape, fill, dtype=dtype, device="cuda")
        self.v_pages = torch.full(shape, fill, dtype=dtype, device="cuda")
        if nhd:
            self.k_pages, self.v_pages = self.k_pages.transpose(1, 2), self.v_pages.transpose(1, 2)
        for b, (_, n) in enumerate(lens):
            if n:
                j = torch.arange(n, device="cuda")
                pg, row = self.page_table[b][j // page].long(), j % page
                self.k_pages[pg, :, row] = randn(g, n, hk, d, dtype=dtype)
                self.v_pages[pg, :, row] = randn(g, n, hk, d, dtype=dtype)

    def args(self):
        return self.q, self.k_pages, self.v_pages, self.cu_q, self.kv_len, self.page_table

    def rows(self, pool, table, j):
        return pool[table[j // self.page].long(), :, j % self.page].to(F64)


def visible(first, a, n, f, sinks, window, device="cuda"):
    """[a queries from position first, n keys] truth values of the mask."""
    p = torch.arange(first, first + a, device=device)[:, None]
    j = torch.arange(n, device=device)[None]
    fp = torch.div(p, f, rounding_mode="floor")
    seen = (j // f <= fp) & (p >= 0)
    if window:
        seen &= (j < sinks * f) | (fp - j // f < window)
    return seen


def attend(bt, f=1, sinks=0, window=0, scale=None, prefix=None):
    """(out, lse, bound of out, bound of lse) in 64 bits, rows of sequences only.

    The bounds: a score is a sum of d exact products in fp32 (each addition off by at most
    2^-23 of the terms' sum of magnitudes) and the multiplication to base 2; its error dx is
    a relative error of its weight. The exponential is allowed 2^-13 (the hardware's is far
    within it; the stale maximum cancels), a weight's rounding to the type UNIT, the sums of n
    terms in fp32 n 2^-23, all relative to the sum of |weights values| A; the division
    and the merge of parts a few 2^-22; the output's rounding UNIT of the value."""
    hq, hk, d, dt = bt.hq, bt.hk, bt.d, bt.dtype
    out = torch.zeros((bt.n_tok, hq, d), dtype=F64, device="cuda")
    lse = torch.full((hq, bt.n_tok), -math.inf, dtype=F64, device="cuda")
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    sc = scale or d ** -0.5
    u = UNIT[dt]
    for b, (a, n) in enumerate(bt.lens):
        seen = visible(n - a, a, n, f, sinks, window)
        used = seen.any(0).nonzero().flatten()
        k, v = (bt.rows(x, bt.page_table[b], used) for x in (bt.k_pages, bt.v_pages))
        seen = seen[:, used]
        if prefix is not None:
            j = torch.arange(prefix[1], device="cuda")
            k = torch.cat((bt.rows(bt.k_pages, prefix[0], j), k))
            v = torch.cat((bt.rows(bt.v_pages, prefix[0], j), v))
            seen = torch.cat((seen.new_ones(a, prefix[1]), seen), 1)
        r = slice(bt.cu[b], bt.cu[b + 1])
        if not a or not k.shape[0]:
            continue
        for h in range(hq):
            q = bt.q[r, h].to(F64)
            kh, vh = k[:, h // (hq // hk)], v[:, h // (hq // hk)]
            x = (q @ kh.T * sc).masked_fill(~seen, -math.inf)
            some = seen.any(1)
            w = torch.softmax(x, -1).nan_to_num(0.0)
            o, A = w @ vh, w @ vh.abs()
            dx = ((q.abs() @ kh.abs().T).masked_fill(~seen, 0).amax(1) * sc * (d + 2) * 2.0 ** -23)[:, None]
            m = seen.sum(1, keepdim=True)
            rel = u + 2 * (dx + 2.0 ** -13 + m * 2.0 ** -23) + 2.0 ** -20
            out[r, h], tol[r, h] = o, rel * A + u * (o.abs() + rel * A) + (2.0 ** -25 if dt == torch.float16 else 0)
            ls = torch.logsumexp(x, -1)
            lse[h, r] = torch.where(some, ls, torch.full_like(ls, -math.inf))
            ltol[h, r] = (dx + 2.0 ** -13 + m * 2.0 ** -23)[:, 0] + 2.0 ** -21 * (ls.abs().nan_to_num(0, 0, 0) + 1)
    return out, lse, tol, ltol


def assert_attend(got, bt, **kw):
    out, lse = got
    want, wlse, tol, ltol = attend(bt, **kw)
    n = bt.cu[-1]
    err = (out[:n].to(F64) - want[:n]).abs()
    assert bool(torch.isfinite(out[:n]).all()), "not finite"
    assert bool((err <= tol[:n]).all()), ("out", float((err - tol[:n]).max()), float(err.max()))
    empty = wlse[:, :n] == -math.inf
    assert bool((lse[:, :n][empty] == -math.inf).all()) and bool((out[:n].transpose(0, 1)[empty] == 0).all())
    lerr = (lse[:, :n].to(F64) - wlse[:, :n]).abs()[~empty]
    if lerr.numel():
        assert bool((lerr <= ltol[:, :n][~empty]).all()), ("lse", float(lerr.max()))
