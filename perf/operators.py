"""Workloads of the paged-cache operators: multi-axis rotary positions, the append that rotates keys into
the pages of a cache, attention over such pages (sinks, sliding window, frame-causal), and attention
for a batch that shares a prefix.

``run`` computes a case in elementary torch operations, or, where ``own`` is true, by the library's
calls; ``exact`` gives its value from the definition in 64 bits. ``listed`` holds fixed cases, ``draw``
makes more of the same ranges.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one denoise call of the smallest test stream: four 4 x 4-token frames, where latency counts
        dict(name="rope_frames_tiny", op="rope", dtype="bf16", tokens=64, q_heads=2, kv_heads=2, head_dim=64,
             pairs_t=12, pairs_h=10, pairs_w=10, grid_h=4, grid_w=4, halves=False, train=False),
        # a training clip of twelve 30 x 52-token frames: queries and keys forward, their gradients back
        dict(name="rope_clip_train", op="rope", dtype="bf16", tokens=18720, q_heads=12, kv_heads=12, head_dim=128,
             pairs_t=22, pairs_h=21, pairs_w=21, grid_h=30, grid_w=52, halves=False, train=True),
        # a packed image with shared key heads, trained in 32 bits: two axes, pairs half a head apart, odd length
        dict(name="rope_image_fp32", op="rope", dtype="fp32", tokens=4097, q_heads=14, kv_heads=2, head_dim=64,
             pairs_t=0, pairs_h=16, pairs_w=16, grid_h=64, grid_w=65, halves=True, train=True),
        # one decoding step of 64 streams: one token each into its last page
        dict(name="append_tokens", op="append", dtype="fp16", seqs=64, q_min=1, q_max=1, kv_min=100, kv_max=8000,
             q_heads=32, kv_heads=8, head_dim=128, page=16, pairs_t=64, pairs_h=0, pairs_w=0, grid_h=1, grid_w=1,
             halves=True),
        # four video streams appending a chunk of three 30 x 52-token frames
        dict(name="append_chunks", op="append", dtype="bf16", seqs=4, q_min=4680, q_max=4680, kv_min=4680, kv_max=14040,
             q_heads=12, kv_heads=12, head_dim=128, page=64, pairs_t=22, pairs_h=21, pairs_w=21, grid_h=30, grid_w=52,
             halves=False),
        # one token of one short stream: latency
        dict(name="decode_one", op="attend", dtype="bf16", seqs=1, q_min=1, q_max=1, kv_min=777, kv_max=777, q_heads=12,
             kv_heads=12, head_dim=64, page=16, frame=1, sinks=0, window=0),
        # a decoding step of 64 streams of very different lengths
        dict(name="decode_batch", op="attend", dtype="bf16", seqs=64, q_min=1, q_max=1, kv_min=300, kv_max=16384,
             q_heads=32, kv_heads=8, head_dim=128, page=16, frame=1, sinks=0, window=0),
        # long streams under a window with four first tokens kept; the pages between are given back
        dict(name="decode_window", op="attend", dtype="fp16", seqs=32, q_min=1, q_max=1, kv_min=2000, kv_max=65536,
             q_heads=40, kv_heads=8, head_dim=128, page=32, frame=1, sinks=4, window=4096),
        # prompts of several lengths, causal token by token, seven query heads to a key head
        dict(name="prompts_ragged", op="attend", dtype="bf16", seqs=6, q_min=37, q_max=2900, kv_min=37, kv_max=2900,
             q_heads=28, kv_heads=4, head_dim=128, page=64, frame=1, sinks=0, window=0),
        # the 480p video chunk: 3 new frames of 1560 tokens, 1 sink frame and a window of 18 frames
        dict(name="chunk_video", op="attend", dtype="bf16", seqs=1, q_min=4680, q_max=4680, kv_min=37440, kv_max=37440,
             q_heads=12, kv_heads=12, head_dim=128, page=64, frame=1560, sinks=1, window=18),
        # 48 continuations of one long prompt, one token each
        dict(name="prefix_decode", op="prefix", dtype="bf16", seqs=48, q_min=1, q_max=1, kv_min=1, kv_max=600,
             prefix=7021, q_heads=32, kv_heads=8, head_dim=128, page=16, frame=1, sinks=0, window=0),
        # four continuations of the same six frames, a frame of 1560 tokens each
        dict(name="prefix_video", op="prefix", dtype="bf16", seqs=4, q_min=1560, q_max=1560, kv_min=1560, kv_max=4680,
             prefix=9360, q_heads=12, kv_heads=12, head_dim=128, page=64, frame=1560, sinks=0, window=0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "prefix"])
    d = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 3, 4, 8, 12])
    group = 1 if kv_heads == 12 else rng.choice([1, 2, 3, 4, 5, 7, 8])
    case = dict(op=op, q_heads=kv_heads * group, kv_heads=kv_heads, head_dim=d)
    if op in ("rope", "append"):
        axes = rng.choice([1, 2, 3])
        c = d // 6
        t, h, w = {1: (d // 2, 0, 0), 2: (0, d // 4, d // 4), 3: (d // 2 - 2 * c, c, c)}[axes]
        case.update(pairs_t=t, pairs_h=h, pairs_w=w, grid_h=_log_int(rng, 2, 64), grid_w=_log_int(rng, 2, 64),
                    halves=rng.random() < 0.5)
        if op == "rope":
            case.update(dtype=rng.choice(["bf16", "fp16", "fp32"]), tokens=_log_int(rng, 1, 18720),
                        train=rng.random() < 0.5)
            return case
    case.update(dtype=rng.choice(["bf16", "fp16"]), page=rng.choice([16, 32, 64, 128]))
    one = rng.random() < 0.5
    q = 1 if one else _log_int(rng, 2, 2900)
    seqs = _log_int(rng, 1, 64 if one else 6)
    kv = max(q, _log_int(rng, 20, 16384 if one else 9000))
    # no more keys and values than the largest listed case reads
    seqs = max(1, min(seqs, 2 * 10 ** 9 // (4 * d * kv_heads * kv)))
    case.update(seqs=seqs, q_min=max(1, q // rng.choice([1, 2, 9])), q_max=q, kv_min=max(1, kv // rng.choice([1, 3, 40])),
                kv_max=kv)
    if op == "append":
        return case
    frame = rng.choice([1, 1, 16, 1560])
    case.update(frame=frame, sinks=0, window=0)
    if rng.random() < 0.5:
        case.update(sinks=rng.choice([0, 1, 4]), window=max(1, _log_int(rng, 64, 4096) // frame))
    if op == "prefix":
        case.update(prefix=_log_int(rng, 64, 9360))
    return case


def _spread(lo, hi, n):
    """n whole numbers over [lo, hi], hi the first, the others by golden-ratio steps."""
    return [hi - int((hi - lo + 1) * ((i * 0.6180339887498949) % 1.0)) for i in range(n)]


def _lengths(case):
    """(queries, tokens in the pages) of each sequence; the queries are a sequence's last tokens."""
    nq = _spread(case["q_min"], case["q_max"], case["seqs"])
    kv = [max(a, b) for a, b in zip(nq, _spread(case["kv_min"], case["kv_max"], case["seqs"]))]
    return nq, kv


def _visible(case, first, last):
    """(sink end, window start) in tokens for the queries at positions [first, last] of a sequence."""
    f, w = case.get("frame", 1), case.get("window", 0)
    start = max(0, (first // f - w + 1) * f) if w else 0
    return (case.get("sinks", 0) * f if w else 0), start


def _dtype(case):
    return DTYPES[case["dtype"]]


def _tables(case, n_t, device):
    """(cos, sin) of position * theta^(-j / pairs) for each axis in use, 64-bit angles rounded to 32."""
    out = []
    for n, p in ((n_t, case["pairs_t"]), (case["grid_h"], case["pairs_h"]), (case["grid_w"], case["pairs_w"])):
        if p:
            a = (torch.arange(n, dtype=torch.float64, device=device)[:, None]
                 * 10000.0 ** (-torch.arange(p, dtype=torch.float64, device=device) / p)[None, :])
            out.append(torch.stack((a.cos(), a.sin()), -1).float().contiguous())
    return tuple(out)


def _positions(case, g):
    """Axis positions of the tokens at stream positions g: frames of grid_h x grid_w tokens."""
    per = case["grid_h"] * case["grid_w"]
    cols = []
    if case["pairs_t"]:
        cols.append(g // per)
    if case["pairs_h"]:
        cols.append(g // case["grid_w"] % case["grid_h"])
    if case["pairs_w"]:
        cols.append(g % case["grid_w"])
    return torch.stack(cols, -1).int().contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt, H, Hk, d = _dtype(case), case["q_heads"], case["kv_heads"], case["head_dim"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dt)

    s = dict(case=case)
    if case["op"] == "rope":
        T = case["tokens"]
        per = case["grid_h"] * case["grid_w"]
        s.update(q=normal(T, H, d), k=normal(T, Hk, d), pos=_positions(case, torch.arange(T, device=dev)),
                 tables=_tables(case, (T + per - 1) // per, dev))
        if case["train"]:
            s["q"].requires_grad_(True)
            s["k"].requires_grad_(True)
            s.update(gq=normal(T, H, d), gk=normal(T, Hk, d))
        return s
    nq, kv = _lengths(case)
    page, n = case["page"], case["seqs"]
    need = [(x + page - 1) // page for x in kv]
    # pages that no query sees any more are back with the pool: their entries are -1
    live = []
    for b in range(n):
        sink, start = _visible(case, kv[b] - nq[b], kv[b] - 1)
        live.append([p for p in range(need[b]) if p * page < sink or (p + 1) * page > start])
    pre = (case.get("prefix", 0) + page - 1) // page
    total = sum(len(x) for x in live) + pre
    order = torch.randperm(total + 3, generator=gen, device=dev).tolist()
    table = torch.full((n, max(need)), -1, dtype=torch.int32)
    at = 0
    for b in range(n):
        table[b, live[b]] = torch.tensor(order[at:at + len(live[b])], dtype=torch.int32)
        at += len(live[b])
    cu = [0]
    for x in nq:
        cu.append(cu[-1] + x)
    T = cu[-1]
    s.update(cu_q=torch.tensor(cu, dtype=torch.int32, device=dev), max_q=max(nq),
             kv_len=torch.tensor(kv, dtype=torch.int32, device=dev), page_table=table.to(dev),
             k_pages=normal(total + 3, Hk, page, d), v_pages=normal(total + 3, Hk, page, d), q=normal(T, H, d))
    if pre:
        s.update(prefix_table=torch.tensor(order[at:at + pre], dtype=torch.int32, device=dev))
    if case["op"] == "append":
        g = torch.cat([torch.arange(kv[b] - nq[b], kv[b], device=dev) for b in range(n)])
        per = case["grid_h"] * case["grid_w"]
        s.update(k=normal(T, Hk, d), v=normal(T, Hk, d), pos=_positions(case, g),
                 tables=_tables(case, (max(kv) + per - 1) // per, dev))
    return s


# ---------------------------------------------------------------------- plain form

def _angles(pos, tables):
    """cos and sin [tokens, 1, pairs] of every pair, axes in order."""
    cs = torch.cat([t[pos[:, a].long()] for a, t in enumerate(tables)], 1)
    return cs[:, None, :, 0], cs[:, None, :, 1]


def _rotate(x, cos, sin, halves):
    x32 = x.float()
    if halves:
        a, b = x32.chunk(2, -1)
        y = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    else:
        a, b = x32[..., 0::2], x32[..., 1::2]
        y = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    return y.to(x.dtype)


def _places(s):
    """Sequence and position of each token."""
    t = torch.arange(s["q"].shape[0], device=s["q"].device)
    b = torch.searchsorted(s["cu_q"], t, right=True) - 1
    i = t - s["cu_q"][b]
    return b, i, s["kv_len"][b] - (s["cu_q"][b + 1] - s["cu_q"][b]) + i


def _plain_rope(s):
    halves = s["case"]["halves"]
    cos, sin = _angles(s["pos"], s["tables"])
    out = [_rotate(s["q"].detach(), cos, sin, halves), _rotate(s["k"].detach(), cos, sin, halves)]
    if s["case"]["train"]:  # the rotation's transpose turns by the opposite angle
        out += [_rotate(s["gq"], cos, -sin, halves), _rotate(s["gk"], cos, -sin, halves)]
    return out


def _plain_append(s):
    halves, page = s["case"]["halves"], s["case"]["page"]
    cos, sin = _angles(s["pos"], s["tables"])
    b, _, p = _places(s)
    where, row = s["page_table"][b, p // page].long(), (p % page).long()
    s["k_pages"][where, :, row] = _rotate(s["k"], cos, sin, halves)
    s["v_pages"][where, :, row] = s["v"]
    return [_rotate(s["q"], cos, sin, halves), s["k_pages"], s["v_pages"]]


def _plain_attend(s):
    c = s["case"]
    H, Hk, d = c["q_heads"], c["kv_heads"], c["head_dim"]
    G, f, n = H // Hk, c["frame"], c["seqs"]
    q, dev = s["q"], s["q"].device
    keys = s["page_table"].shape[1] * c["page"]

    def pages(pool, table):  # [.., pages] -> [.., Hk, tokens, d]
        x = pool[table.clamp(min=0).long()].float()
        return x.transpose(-4, -3).flatten(-3, -2)

    i = torch.arange(s["max_q"], device=dev)
    nq = s["cu_q"][1:] - s["cu_q"][:-1]
    tok = (s["cu_q"][:-1, None] + torch.minimum(i[None], nq[:, None] - 1)).long()
    qp = q[tok].float().view(n, s["max_q"], Hk, G, d).permute(0, 2, 3, 1, 4).reshape(n, Hk, G * s["max_q"], d)
    sc = qp @ pages(s["k_pages"], s["page_table"]).transpose(-1, -2) / math.sqrt(d)
    at = (s["kv_len"] - nq)[:, None, None] + i[None, :, None]
    j = torch.arange(keys, device=dev)[None, None]
    seen = (j < s["kv_len"][:, None, None]) & (j // f <= at // f)
    if c["window"]:
        seen &= (j < c["sinks"] * f) | (j // f > at // f - c["window"])
    sc = sc.view(n, Hk, G, s["max_q"], keys).masked_fill_(~seen[:, None, None], -math.inf)
    v = pages(s["v_pages"], s["page_table"])
    if c["op"] == "prefix":
        kx, vx = pages(s["k_pages"], s["prefix_table"])[:, :c["prefix"]], pages(s["v_pages"], s["prefix_table"])[:, :c["prefix"]]
        sx = (qp @ kx.transpose(-1, -2) / math.sqrt(d)).view(n, Hk, G, s["max_q"], c["prefix"])
        top = torch.maximum(sc.amax(-1, keepdim=True), sx.amax(-1, keepdim=True))
        px = (sx - top).exp()
    else:
        top = sc.amax(-1, keepdim=True)
    p = sc.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = p.view(n, Hk, G * s["max_q"], keys) @ v
    if c["op"] == "prefix":
        total = total + px.sum(-1, keepdim=True)
        o = o + px.view(n, Hk, G * s["max_q"], c["prefix"]) @ vx
    o = o.view(n, Hk, G, s["max_q"], d) / total
    lse = (top + total.log()).reshape(n, H, s["max_q"])
    b, i, _ = _places(s)
    return [o.permute(0, 3, 1, 2, 4)[b, i].reshape(q.shape).to(q.dtype), lse.transpose(1, 2)[b, i].T.contiguous()]


# ---------------------------------------------------------------------- the library's calls

def _own_rope(s):
    from rolling_kv_cache_b200 import paged
    pairing = "halves" if s["case"]["halves"] else "adjacent"
    y = paged.rope_axes((s["q"], s["k"]), s["pos"], s["tables"], pairing=pairing)
    if not s["case"]["train"]:
        return list(y)
    grads = torch.autograd.grad(y, (s["q"], s["k"]), (s["gq"], s["gk"]))
    return [y[0].detach(), y[1].detach(), *grads]


def _own_append(s):
    from rolling_kv_cache_b200 import paged
    q = paged.paged_append(s["q"], s["k"], s["v"], s["k_pages"], s["v_pages"], s["cu_q"], s["kv_len"], s["page_table"],
                           pos=s["pos"], tables=s["tables"], pairing="halves" if s["case"]["halves"] else "adjacent")
    return [q, s["k_pages"], s["v_pages"]]


def _own_attend(s):
    from rolling_kv_cache_b200 import paged
    c = s["case"]
    mask = dict(max_q=s["max_q"], frame_seqlen=c["frame"], sink_frames=c["sinks"], window_frames=c["window"])
    if c["op"] == "prefix":
        out = paged.prefix_attention(s["q"], s["k_pages"], s["v_pages"], s["prefix_table"], c["prefix"], s["cu_q"],
                                     s["kv_len"], s["page_table"], return_lse=True, **mask)
    else:
        out = paged.paged_attention(s["q"], s["k_pages"], s["v_pages"], s["cu_q"], s["kv_len"], s["page_table"],
                                    return_lse=True, **mask)
    return list(out)


def run(state):
    op = state["case"]["op"]
    if own:
        call = {"rope": _own_rope, "append": _own_append}.get(op, _own_attend)
    else:
        call = {"rope": _plain_rope, "append": _plain_append}.get(op, _plain_attend)
    return call(state)


# ---------------------------------------------------------------------- work and exact values

def work(case):
    H, Hk, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    size = 4 if case["dtype"] == "fp32" else 2
    pairs = case.get("pairs_t", 0) + case.get("pairs_h", 0) + case.get("pairs_w", 0)
    axes = sum(1 for a in "thw" if case.get("pairs_" + a, 0))
    if case["op"] == "rope":
        turns = 2 if case["train"] else 1
        per = case["grid_h"] * case["grid_w"]
        rows = 0
        if case["pairs_t"]:
            rows += case["pairs_t"] * ((case["tokens"] + per - 1) // per)
        rows += case["pairs_h"] * min(case["grid_h"], case["tokens"]) + case["pairs_w"] * min(case["grid_w"], case["tokens"])
        return {"bytes": turns * (2 * case["tokens"] * (H + Hk) * d * size) + case["tokens"] * axes * 4 + rows * 8,
                "flops": turns * 6 * case["tokens"] * (H + Hk) * pairs}
    nq, kv = _lengths(case)
    T = sum(nq)
    if case["op"] == "append":
        return {"bytes": 2 * T * (H + 2 * Hk) * d * size + T * axes * 4, "flops": 6 * T * (H + Hk) * pairs}
    f, w, P = case["frame"], case["window"], case.get("prefix", 0)
    met = keys = 0
    for a, b in zip(nq, kv):
        sink, start = _visible(case, b - a, b - 1)
        keys += b - max(0, start - sink)
        for fr in range((b - a) // f, (b - 1) // f + 1):
            rows = min(b, (fr + 1) * f) - max(b - a, fr * f)
            end = min(b, (fr + 1) * f)
            sk, st = _visible(case, fr * f, fr * f)
            met += rows * (end - max(0, st - sk) + P)
    return {"bytes": 2 * T * H * d * size + 2 * (keys + P) * Hk * d * size + T * H * 4, "flops": 4 * d * H * met}


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] in ("rope", "append"):
        cs = torch.cat([tab.to(f64)[s["pos"][:, a].long()] for a, tab in enumerate(s["tables"])], 1)
        z = torch.complex(cs[..., 0], cs[..., 1])[:, None]

        def turn(x, unit):
            x = x.detach().to(f64)
            if case["halves"]:
                h = case["head_dim"] // 2
                y = torch.complex(x[..., :h].contiguous(), x[..., h:].contiguous()) * unit
                return torch.cat((y.real, y.imag), -1)
            y = torch.view_as_complex(x.reshape(*x.shape[:-1], -1, 2)) * unit
            return torch.view_as_real(y).flatten(-2)

        if case["op"] == "rope":
            out = [turn(s["q"], z), turn(s["k"], z)]
            return out + [turn(s["gq"], z.conj()), turn(s["gk"], z.conj())] if case["train"] else out
        kp, vp, rk = s["k_pages"].to(f64), s["v_pages"].to(f64), turn(s["k"], z)
    nq, kv = _lengths(case)
    page, table, at = case["page"], s["page_table"], 0
    H, Hk, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    out = torch.empty(s["q"].shape, dtype=f64, device=s["q"].device)
    lse = torch.empty((H, s["q"].shape[0]), dtype=f64, device=s["q"].device)
    for b, (a, n) in enumerate(zip(nq, kv)):
        p = torch.arange(n - a, n, device=out.device)
        if case["op"] == "append":
            where = table[b][p // page].long()
            kp[where, :, p % page], vp[where, :, p % page] = rk[at:at + a], s["v"][at:at + a].to(f64)
            at += a
            continue
        # every key that some query sees, by its position
        j = torch.arange(n, device=out.device)
        f, w = case["frame"], case["window"]
        sink, start = _visible(case, n - a, n - 1)
        j = j[(j < sink) | (j >= start)]
        where = table[b][j // page].long()
        seen = j[None] // f <= p[:, None] // f
        if w:
            seen &= (j[None] < case["sinks"] * f) | (p[:, None] // f - j[None] // f < w)
        for h in range(H):
            k, v = (x[where, h // (H // Hk), j % page].to(f64) for x in (s["k_pages"], s["v_pages"]))
            vis = seen
            if case["op"] == "prefix":
                i = torch.arange(case["prefix"], device=out.device)
                e = s["prefix_table"][i // page].long()
                k, v = (torch.cat((x[e, h // (H // Hk), i % page].to(f64), y))
                        for x, y in ((s["k_pages"], k), (s["v_pages"], v)))
                vis = torch.cat((seen.new_ones(a, case["prefix"]), seen), 1)
            x = s["q"][at:at + a, h].to(f64) @ k.T * d ** -0.5
            x = x.masked_fill(~vis, -math.inf)
            out[at:at + a, h] = torch.softmax(x, -1) @ v
            lse[h, at:at + a] = torch.logsumexp(x, -1)
        at += a
    if case["op"] == "append":
        return [turn(s["q"], z), kp, vp]
    return [out, lse]
