"""What is measured of the paged serving operators: their cases, inputs, plain
forms and definitions.

Five operators that let requests of different lengths share one pool of cache
pages:

  plan      block tables and slot maps of one step, from request lengths
  store     new raw tokens (RMSNorm, partial RoPE) into their pages
  compress  new blocks of m tokens pooled into FP8/BF16 entry pages, with the
            tail of each request's incomplete block
  chunk     attention of each request's new tokens over its paged entries and
            the sliding window of its paged tokens
  window    attention of each request's new tokens over a sliding window and
            the first tokens of the request, which stay visible

Lengths belong to the case (they decide the work); values, page numbers and
parameters are drawn from the seed.
"""
import math
import random

import torch

own = False

M_HCA = 128                                    # tokens per entry
LAYOUTS = {512: (512, 64, 64), 128: (128, 32, 32)}     # d -> (d, d_rope, scale group)
EPS = 1e-6
DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step's tables for 32 requests of up to 256K tokens
        dict(name="plan_decode_b32", op="plan", B=32, T=1, ctx=262143, ragged=False, P=64, m=1, lens=1),
        # a prefill step's tables: 192 requests, up to 512 new tokens each, some with none
        dict(name="plan_prefill_b192", op="plan", B=192, T=512, ctx=65535, ragged=True, P=64, m=1, lens=2),
        # one decode step's tokens into their pages, one layer
        dict(name="store_decode_b32", op="store", B=32, T=1, ctx=262143, ragged=False, P=64, d=512, extras=True, lens=3),
        # prefill: about 16K tokens of 23 requests into their pages, normalised and rotated
        dict(name="store_prefill_16k", op="store", B=23, T=1400, ctx=131072, ragged=True, P=64, d=512, extras=True, lens=4),
        # decode: one token each, one request in 128 finishes a block; the small layout
        dict(name="compress_decode_d128", op="compress", B=40, T=1, ctx=1023, ragged=True, P=16, m=128, d=128,
             extras=False, lens=5),
        # prefill: blocks of 128 across ragged chunks, entries normalised and rotated
        dict(name="compress_prefill_16k", op="compress", B=21, T=1500, ctx=131072, ragged=True, P=64, m=128, d=512,
             extras=True, lens=6),
        # decode over 1M tokens: 8192 entries for each of 4 requests
        dict(name="chunk_decode_b4_1m", op="chunk", B=4, T=1, ctx=1048575, ragged=False, P=64, m=128, d=512, H=64, W=128,
             extras=False, lens=7),
        # decode of a batch of short and long requests in the small layout
        dict(name="chunk_decode_b33_d128", op="chunk", B=33, T=1, ctx=65535, ragged=True, P=16, m=128, d=128, H=8, W=128,
             extras=False, lens=8),
        # one 4096-token prefill chunk after 131072 tokens
        dict(name="chunk_prefill_4096_131k", op="chunk", B=1, T=4096, ctx=131072, ragged=False, P=64, m=128, d=512, H=64,
             W=128, extras=False, lens=9),
        # a step of chunks, single tokens and idle requests together, with query RMSNorm, RoPE and sink
        dict(name="chunk_mixed_b13", op="chunk", B=13, T=257, ctx=65535, ragged=True, P=64, m=128, d=512, H=64, W=128,
             extras=True, lens=10),
        # a window-only layer's decode step, 4 first tokens visible
        dict(name="window_decode_b32", op="window", B=32, T=1, ctx=262143, ragged=False, P=64, d=512, H=64, W=128, first=4,
             extras=False, lens=11),
        # a window-only layer's prefill chunks, with query RMSNorm, RoPE and sink
        dict(name="window_prefill_b3", op="window", B=3, T=2048, ctx=65535, ragged=True, P=64, d=512, H=64, W=128, first=4,
             extras=True, lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "store", "compress", "chunk", "chunk", "chunk", "window", "window"])
    c = dict(op=op, lens=rng.randrange(1 << 30), ragged=rng.random() < 0.8, P=rng.choice([16, 32, 48, 64, 128]))
    if op == "plan":
        c.update(B=_log(rng, 1, 512), T=_log(rng, 1, 512), ctx=_log(rng, 1, 262143), m=rng.choice([1, 1, 4, 128]))
        return c
    c.update(d=rng.choice([512, 512, 128]), extras=rng.random() < 0.5, ctx=_log(rng, 1, 262143))
    if op in ("store", "compress"):
        c.update(B=_log(rng, 1, 64), T=_log(rng, 1, 2048))
        c["T"] = max(1, min(c["T"], 16384 // c["B"]))
        if op == "compress":
            c["m"] = rng.choice([4, 128])
        return c
    decode = rng.random() < 0.4
    c.update(B=_log(rng, 1, 64), T=1 if decode else _log(rng, 2, 2048), W=rng.choice([1, 17, 64, 128, 128, 128]))
    c["T"] = max(1, min(c["T"], 4096 // c["B"]))
    c["H"] = 64 if c["d"] == 512 else rng.choice([1, 5, 8, 8, 16, 64])
    if op == "chunk":
        c["m"] = 128
        c["ctx"] = min(c["ctx"], 131072 * 32 // max(32, c["B"] * c["T"] // 128))
    else:
        c["first"] = rng.choice([0, 1, 4, 4, 64])
    return c


def lengths(case):
    """(tokens cached before the step, new tokens) of each request."""
    r = random.Random(case["lens"])
    ctx, new = [], []
    for b in range(case["B"]):
        if case["ragged"]:
            ctx.append(r.choice([0, r.randint(0, case["ctx"]), r.randint(case["ctx"] // 2, case["ctx"]), case["ctx"]]))
            new.append(r.choice([0, r.randint(0, case["T"]), r.randint(0, case["T"]), r.randint((case["T"] + 1) // 2, case["T"])]))
        else:
            ctx.append(case["ctx"])
            new.append(case["T"])
    if sum(new) == 0:
        new[0] = case["T"]
    return ctx, new


def _items(case, m):
    """Per request (first item, one past the last) for items of m tokens."""
    return [(c // m, (c + n) // m) for c, n in zip(*lengths(case))]


def _pages(n, P):
    return -(-n // P)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _normal(shape, g, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(torch.bfloat16)


def _starts(counts):
    s = [0]
    for c in counts:
        s.append(s[-1] + c)
    return s


def _table(spans, P, g, spare=3):
    """Block table whose pages hold rows [0, end) of every request but only
    for the pages that `spans` names ([(lo, hi)] row ranges per request);
    pages that no span touches are -1.  Returns (table, number of pages)."""
    width = max(1, max(_pages(max((hi for _, hi in sp), default=0), P) for sp in spans))
    need = [sorted({p for lo, hi in sp if hi > lo for p in range(lo // P, _pages(hi, P))}) for sp in spans]
    total = sum(len(n) for n in need)
    ids = torch.randperm(total + spare, generator=g, device=DEV)[:total].to(torch.int32)
    table = torch.full((len(spans), width), -1, dtype=torch.int32, device=DEV)
    if total:
        rows = torch.tensor([b for b, n in enumerate(need) for _ in n], device=DEV)
        cols = torch.tensor([p for n in need for p in n], device=DEV)
        table[rows, cols] = ids
    return table, total + spare


def _rows(spans, table, P):
    """(row_start, row_req, row_pos, slot) of the items in `spans`, one range per request."""
    req = torch.tensor([b for b, (lo, hi) in enumerate(spans) for _ in range(lo, hi)], dtype=torch.int64, device=DEV)
    pos = torch.tensor([e for lo, hi in spans for e in range(lo, hi)], dtype=torch.int64, device=DEV)
    slot = table[req, pos // P].long() * P + pos % P
    return (_i32(_starts([hi - lo for lo, hi in spans])), req.to(torch.int32), pos.to(torch.int32), slot)


def _params(case, g):
    d, dr, _ = LAYOUTS[case["d"]]
    s = {}
    if case["extras"]:
        s["norm_w"] = 1.0 + 0.1 * torch.randn(d, generator=g, device=DEV)
        s["inv_freq"] = (10000.0 ** (-torch.arange(0, dr, 2, dtype=torch.float64, device=DEV) / dr)).float()
        if "H" in case:
            s["sink"] = torch.randn(case["H"], generator=g, device=DEV)
    return s


def _entry_pool(n_pages, P, d, g):
    """Entries as compression leaves them: FP8 codes with amax / 448 scales, bf16 RoPE dims."""
    _, dr, grp = LAYOUTS[d]
    y = torch.randn((n_pages, P, (d - dr) // grp, grp), generator=g, device=DEV) * 0.25
    scales = y.abs().amax(-1) / 448.0
    codes = (y / scales[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).reshape(n_pages, P, d - dr)
    return codes.contiguous(), scales.contiguous(), _normal((n_pages, P, dr), g, 0.25)


def prepare(case, seed):
    g = _gen(seed)
    op, P = case["op"], case["P"]
    ctx, new = lengths(case)
    s = dict(case=case, ctx=_i32(ctx), new=_i32(new), N=sum(new), max_new=max(new))
    if op == "plan":
        m = case["m"]
        items = _items(case, m)
        held = [_pages(lo, P) for lo, _ in items]
        want = [_pages(hi, P) for _, hi in items]
        total = sum(held) + sum(w - h for w, h in zip(want, held) if w > h)
        ids = torch.randperm(total + 5, generator=g, device=DEV).to(torch.int32)
        table = torch.full((case["B"], max(1, max(want))), -1, dtype=torch.int32, device=DEV)
        if sum(held):
            req = torch.repeat_interleave(torch.arange(case["B"], device=DEV), torch.tensor(held, device=DEV))
            col = torch.arange(sum(held), device=DEV) - torch.tensor(_starts(held)[:-1], device=DEV)[req]
            table[req, col] = ids[:sum(held)]
        rows = sum(hi - lo for lo, hi in items) + 7
        s.update(table=table, free_pages=ids[sum(held):].contiguous(), free_count=_i32([total + 5 - sum(held)]),
                 row_start=_i32([0] * (case["B"] + 1)), row_req=_i32([-1] * rows), row_pos=_i32([-1] * rows),
                 slot=torch.full((rows,), -1, dtype=torch.int64, device=DEV), missing=_i32([0]), free_left=_i32([0]))
        return s
    d = case["d"]
    _, dr, grp = LAYOUTS[d]
    s.update(_params(case, g))
    s["starts"] = _i32(_starts(new))
    if op == "store":
        spans = [(c, c + n) for c, n in zip(ctx, new)]
        table, n_pages = _table([[sp] for sp in spans], P, g)
        s["row_start"], s["row_req"], s["row_pos"], s["slot"] = _rows(spans, table, P)
        s["x"] = _normal((s["N"], d), g)
        s["pages"] = torch.zeros((n_pages, P, d), dtype=torch.bfloat16, device=DEV)
        return s
    if op == "compress":
        m = case["m"]
        spans = _items(case, m)
        table, n_pages = _table([[sp] for sp in spans], P, g)
        s["row_start"], s["row_req"], s["row_pos"], s["slot"] = _rows(spans, table, P)
        s["x"], s["gate"] = _normal((s["N"], d), g), _normal((s["N"], d), g)
        s["bias"] = torch.randn((m, d), generator=g, device=DEV) * 0.5
        s["tail_x"], s["tail_gate"] = _normal((case["B"], m, d), g), _normal((case["B"], m, d), g)
        s["codes"] = torch.zeros((n_pages, P, d - dr), dtype=torch.uint8, device=DEV)
        s["scales"] = torch.zeros((n_pages, P, (d - dr) // grp), device=DEV)
        s["rope"] = torch.zeros((n_pages, P, dr), dtype=torch.bfloat16, device=DEV)
        return s
    W, first = case["W"], case.get("first", 0)
    s["q"] = _normal((s["N"], case["H"], d), g)
    s["scale"] = float(d) ** -0.5
    tspans = [[(0, min(first, c + n)), (max(0, c - W + 1), c + n)] if n else [] for c, n in zip(ctx, new)]
    s["token_table"], n_tp = _table(tspans, P, g)
    s["pages"] = _normal((n_tp, P, d), g)
    if op == "chunk":
        s["entry_table"], n_ep = _table([[(0, (c + n) // case["m"])] for c, n in zip(ctx, new)], P, g)
        s["codes"], s["scales"], s["rope"] = _entry_pool(n_ep, P, d, g)
    return s


# ------------------------------------------------------------------ plain forms
def run(s):
    return (_own if own else _plain)(s)


def _plain(s):
    return {"plan": _plain_plan, "store": _plain_store, "compress": _plain_compress, "chunk": _plain_attn,
            "window": _plain_attn}[s["case"]["op"]](s)


def _plain_plan(s):
    m, P = s["case"]["m"], s["case"]["P"]
    zero = torch.zeros(1, dtype=torch.int64, device=DEV)
    ctx, new = s["ctx"].long(), s["new"].long()
    lo, hi = ctx // m, (ctx + new) // m
    start = torch.cat([zero, (hi - lo).cumsum(0)])
    have, want = (lo + P - 1) // P, (hi + P - 1) // P
    page0 = torch.cat([zero, (want - have).cumsum(0)])
    # new pages come off the top of the free stack, in request order
    table, F = s["table"], s["free_count"].long()
    col = torch.arange(table.shape[1], device=DEV)[None]
    k = F - 1 - (page0[:-1, None] + col - have[:, None])
    fresh = (col >= have[:, None]) & (col < want[:, None])
    got = torch.where(k >= 0, s["free_pages"][torch.where(fresh, k.clamp(min=0), 0)], -1)
    table = torch.where(fresh, got, table)
    rows = torch.arange(s["row_req"].numel(), device=DEV)
    live = rows < start[-1]
    req = torch.searchsorted(start[1:], rows, right=True).clamp(max=table.shape[0] - 1)
    pos = rows - start[req] + lo[req]
    page = table[req, (pos // P).clamp(max=table.shape[1] - 1)].long()
    slot = torch.where(page >= 0, page * P + pos % P, -1)
    return {"table": table, "row_start": start.to(torch.int32),
            "row_req": torch.where(live, req, s["row_req"]).to(torch.int32),
            "row_pos": torch.where(live, pos, s["row_pos"]).to(torch.int32), "slot": torch.where(live, slot, s["slot"]),
            "missing": (page0[-1:] - F).clamp(min=0).to(torch.int32), "free_left": (F - page0[-1:]).clamp(min=0).to(torch.int32)}


def _angles(pos, s):
    a = pos.double()[:, None] * s["inv_freq"].double()[None]
    return a.cos().float(), a.sin().float()


def _rope(y, cos, sin, back=False):
    """Rotates the last 2 * cos.shape[-1] channels, pairs (2i, 2i + 1)."""
    k = 2 * cos.shape[-1]
    a, b = y[..., -k::2], y[..., y.shape[-1] - k + 1::2]
    sin = -sin if back else sin
    r = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([y[..., :-k], r], -1)


def _norm(y, w):
    return y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS) * w


def _plain_store(s):
    y = s["x"].float()
    if s["case"]["extras"]:
        y = _rope(_norm(y, s["norm_w"]), *_angles(s["row_pos"], s))
    pages = s["pages"]
    pages.view(-1, pages.shape[-1])[s["slot"]] = y.to(torch.bfloat16)
    return pages


def _plain_compress(s):
    case = s["case"]
    m, d = case["m"], case["d"]
    _, dr, grp = LAYOUTS[d]
    ctx, start = s["ctx"].long(), s["starts"].long()
    req, ent = s["row_req"].long(), s["row_pos"].long()
    t = ent[:, None] * m + torch.arange(m, device=DEV)
    N = s["x"].shape[0]
    row = torch.where(t < ctx[req][:, None], N + req[:, None] * m + t % m, start[req][:, None] + t - ctx[req][:, None])
    x = torch.cat([s["x"], s["tail_x"].view(-1, d)])[row].float()
    z = torch.cat([s["gate"], s["tail_gate"].view(-1, d)])[row].float() + s["bias"]
    e = torch.exp(z - z.amax(1, keepdim=True))
    y = (e * x).sum(1) / e.sum(1)
    if case["extras"]:
        y = _rope(_norm(y, s["norm_w"]), *_angles(ent * m, s))
    k = y[:, :d - dr].view(-1, (d - dr) // grp, grp)
    scales = k.abs().amax(-1) / 448.0
    codes = (k / scales[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8).view(-1, d - dr)
    s["codes"].view(-1, d - dr)[s["slot"]] = codes
    s["scales"].view(-1, (d - dr) // grp)[s["slot"]] = scales
    s["rope"].view(-1, dr)[s["slot"]] = y[:, d - dr:].to(torch.bfloat16)
    # the tail: the new tokens of each request's incomplete block (a copy, so that a pass can be repeated)
    rows = torch.arange(N, device=DEV)
    b = torch.searchsorted(start[1:], rows, right=True)
    t = rows - start[b] + ctx[b]
    end = ctx + start[1:] - start[:-1]
    at = torch.where(t >= end[b] // m * m, b * m + t % m, case["B"] * m)
    tails = []
    for src, old in ((s["x"], s["tail_x"]), (s["gate"], s["tail_gate"])):
        new = torch.cat([old.view(-1, d), old.view(-1, d)[:1]])
        new[at] = src
        tails.append(new[:-1].view_as(old))
    return {"codes": s["codes"].view(torch.float8_e4m3fn), "scales": s["scales"], "rope": s["rope"], "tail_x": tails[0],
            "tail_gate": tails[1]}


def _plain_attn(s):
    case = s["case"]
    d, H, W, P, N, T = case["d"], case["H"], case["W"], case["P"], s["N"], s["max_new"]
    first = case.get("first", 0)
    start, ctx = s["starts"].long(), s["ctx"].long()
    rows = torch.arange(N, device=DEV)
    req = torch.searchsorted(start[1:], rows, right=True)
    i = rows - start[req]
    p = ctx[req] + i
    q = s["q"].float()
    if case["extras"]:
        cos, sin = _angles(p, s)
        cos, sin = cos[:, None], sin[:, None]
        q = _rope(_norm(q, s["norm_w"]), cos, sin)
    # the first tokens that the window has left, then the window
    t = torch.cat([torch.arange(first, device=DEV).expand(N, first), p[:, None] - W + 1 + torch.arange(W, device=DEV)], 1)
    seen = torch.cat([t[:, :first] < (p - W + 1)[:, None], t[:, first:] >= 0], 1)
    table = s["token_table"]
    page = table[req[:, None], (t.clamp(min=0) // P).clamp(max=table.shape[1] - 1)].long()
    keys = s["pages"].view(-1, d)[torch.where(seen, page * P + t % P, 0)].float()
    logits = [torch.where(seen[:, None], torch.matmul(q, keys.transpose(1, 2)) * s["scale"], -math.inf)]
    if case["op"] == "chunk":
        m, B = case["m"], case["B"]
        _, dr, grp = LAYOUTS[d]
        table = s["entry_table"]
        E = table.shape[1] * P
        k = s["codes"].view(torch.float8_e4m3fn).float().view(-1, P, (d - dr) // grp, grp) * s["scales"][..., None]
        k = torch.cat([k.flatten(2), s["rope"].float()], -1)
        ent = k[table.long().clamp(min=0)].view(B, E, d)
        qp = torch.zeros((B, T, H, d), device=DEV)
        qp[req, i] = q
        le = torch.matmul(qp.view(B, T * H, d), ent.transpose(1, 2)).view(B, T, H, E)[req, i] * s["scale"]
        vis = torch.arange(E, device=DEV)[None] < ((p + 1) // m)[:, None]
        logits.append(torch.where(vis[:, None], le, -math.inf))
        del le, qp
    if case["extras"]:
        logits.append(s["sink"].expand(N, H)[..., None])
    w = torch.softmax(torch.cat(logits, -1), -1)
    del logits
    n = first + W
    out = torch.matmul(w[..., :n], keys)
    if case["op"] == "chunk":
        wp = torch.zeros((B, T, H, E), device=DEV)
        wp[req, i] = w[..., n:n + E]
        out += torch.matmul(wp.view(B, T * H, E), ent).view(B, T, H, d)[req, i]
    if case["extras"]:
        out = _rope(out, cos, sin, back=True)
    return out.to(torch.bfloat16)


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    import long_context_attention_hca_b200 as hca
    case = s["case"]
    op = case["op"]
    if op == "plan":
        plan = hca.PagePlan(s["row_start"], s["row_req"], s["row_pos"], s["slot"], s["missing"], s["free_left"])
        hca.kv_page_plan(s["ctx"], s["new"], case["m"], case["P"], s["table"], s["free_pages"], s["free_count"], plan=plan)
        return {"table": s["table"], "row_start": plan.row_start, "row_req": plan.row_req, "row_pos": plan.row_pos,
                "slot": plan.slot, "missing": plan.missing, "free_left": plan.free_left}
    layout = LAYOUTS[case["d"]]
    if op in ("store", "compress"):
        ee = hca.EntryExtras(s["norm_w"], EPS, s["inv_freq"]) if case["extras"] else None
        plan = hca.PagePlan(s["row_start"], s["row_req"], s["row_pos"], s["slot"])
        if op == "store":
            return hca.kv_page_store(s["x"], plan, s["pages"], layout, extras=ee)
        cache = hca.KVCache.of(s["codes"], s["scales"], s["rope"])
        tail_x, tail_gate = s["tail_x"].clone(), s["tail_gate"].clone()     # a pass can be repeated
        hca.kv_page_compress(s["x"], s["gate"], s["bias"], s["starts"], s["ctx"], plan, tail_x, tail_gate, cache, extras=ee)
        return {"codes": s["codes"].view(torch.float8_e4m3fn), "scales": s["scales"], "rope": s["rope"], "tail_x": tail_x,
                "tail_gate": tail_gate}
    ex = hca.AttnExtras(s["norm_w"], EPS, s["sink"], s["inv_freq"]) if case["extras"] else None
    if op == "window":
        return hca.paged_attn_window(s["q"], s["starts"], s["ctx"], s["pages"], s["token_table"], case["W"], case["first"],
                                     s["scale"], max_new=s["max_new"], extras=ex)
    cache = hca.KVCache.of(s["codes"], s["scales"], s["rope"])
    return hca.paged_attn_chunk(s["q"], s["starts"], s["ctx"], case["m"], cache, s["entry_table"], s["pages"],
                                s["token_table"], case["W"], s["scale"], max_new=s["max_new"], extras=ex)


# ------------------------------------------------------------------ work
def work(case):
    ctx, new = lengths(case)
    B, N, P = case["B"], sum(new), case["P"]
    if case["op"] == "plan":
        items = _items(case, case["m"])
        n = sum(hi - lo for lo, hi in items)
        fresh = sum(_pages(hi, P) - _pages(lo, P) for lo, hi in items)
        # lengths in, starts out; 16 bytes a row out; a fresh page is read once and written once
        return {"bytes": 12 * B + 16 * n + 8 * fresh, "flops": 0}
    d = case["d"]
    _, dr, grp = LAYOUTS[d]
    entry = (d - dr) + 4 * ((d - dr) // grp) + 2 * dr
    if case["op"] == "store":
        return {"bytes": N * (4 * d + 12), "flops": 6 * N * d if case["extras"] else 0}
    if case["op"] == "compress":
        m = case["m"]
        blocks = [(c, c + n, c // m, (c + n) // m) for c, n in zip(ctx, new)]
        ents = sum(hi - lo for _, _, lo, hi in blocks)
        old = sum(c - lo * m for c, _, lo, hi in blocks if hi > lo)
        tail = sum(e - max(c, hi * m) for c, e, _, hi in blocks)
        return {"bytes": 4 * d * (N + old + tail) + 4 * m * d + ents * entry, "flops": 6 * ents * m * d}
    W, first, H = case["W"], case.get("first", 0), case["H"]
    keys = toks = ents = 0
    for c, n in zip(ctx, new):
        if n == 0:
            continue
        w0 = max(0, c - W + 1)
        toks += c + n - w0 + min(first, w0)
        for p in range(c, c + n):
            lo = max(0, p - W + 1)
            keys += p - lo + 1 + min(first, lo)
            if case["op"] == "chunk":
                keys += (p + 1) // case["m"]
        if case["op"] == "chunk":
            ents += (c + n) // case["m"]
    return {"bytes": 4 * N * H * d + 2 * d * toks + entry * ents, "flops": 4 * H * d * keys}


# ------------------------------------------------------------------ the definition in 64 bits
def _e4m3_values():
    v = []
    for c in range(256):
        s, e, f = c >> 7, (c >> 3) & 15, c & 7
        x = f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        v.append(math.nan if (c & 127) == 127 else (-x if s else x))
    return torch.tensor(v, dtype=torch.float64, device=DEV)


def _rot64(v, ang):
    """Complex rotation of the trailing pairs by `ang` (one row of angles per row of v's first axis)."""
    k = 2 * ang.shape[-1]
    z = torch.view_as_complex(v[..., -k:].unflatten(-1, (-1, 2)).contiguous())
    turn = torch.polar(torch.ones_like(ang), ang).view(ang.shape[0], *([1] * (v.dim() - 2)), ang.shape[1])
    out = v.clone()
    out[..., -k:] = torch.view_as_real(z * turn).flatten(-2)
    return out


def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    d = case["d"]
    _, dr, grp = LAYOUTS[d]
    if "norm_w" in s:
        nw, fr = s["norm_w"].double(), s["inv_freq"].double()

    def unit(v):
        return v * (v.square().mean(-1, keepdim=True) + EPS).rsqrt() * nw

    if case["op"] == "store":
        y = s["x"].double()
        if case["extras"]:
            y = _rot64(unit(y), s["row_pos"].double()[:, None] * fr)
        out = torch.zeros(s["pages"].shape, dtype=torch.float64, device=DEV).view(-1, d)
        out[s["slot"]] = y
        return out.view(s["pages"].shape)
    ctx, new = lengths(case)
    start = _starts(new)
    if case["op"] == "compress":
        m, P = case["m"], case["P"]
        outs = {k: torch.zeros(s[k].shape, dtype=torch.float64, device=DEV) for k in ("codes", "scales", "rope")}
        tails = {k: s[k].double() for k in ("tail_x", "tail_gate")}
        slots, at = s["slot"].tolist(), 0
        for b, (c, n) in enumerate(zip(ctx, new)):
            lo = c // m * m
            x = torch.cat([s["tail_x"][b, :c - lo], s["x"][start[b]:start[b] + n]]).double()
            z = torch.cat([s["tail_gate"][b, :c - lo], s["gate"][start[b]:start[b] + n]]).double()
            k = x.shape[0] // m
            if k:
                wgt = torch.softmax(z[:k * m].view(k, m, d) + s["bias"].double(), 1)
                y = (wgt * x[:k * m].view(k, m, d)).sum(1)
                if case["extras"]:
                    first = torch.arange(lo // m, lo // m + k, device=DEV).double() * m
                    y = _rot64(unit(y), first[:, None] * fr)
                to = slots[at:at + k]
                at += k
                v = y[:, :d - dr].reshape(k, -1, grp)
                sc = v.abs().amax(-1) / 448
                outs["codes"].view(-1, d - dr)[to] = (v / sc[..., None]).reshape(k, -1)
                outs["scales"].view(-1, (d - dr) // grp)[to] = sc
                outs["rope"].view(-1, dr)[to] = y[:, d - dr:]
            rest = x.shape[0] - k * m
            tails["tail_x"][b, :rest] = x[k * m:]
            tails["tail_gate"][b, :rest] = z[k * m:]
        return {**outs, **tails}
    H, W, P, first = case["H"], case["W"], case["P"], case.get("first", 0)
    val = _e4m3_values()
    out = torch.zeros((s["N"], H, d), dtype=torch.float64, device=DEV)
    toks = s["pages"].reshape(-1, d)
    for b, (c, n) in enumerate(zip(ctx, new)):
        if n == 0:
            continue
        w0 = max(0, c - W + 1)
        tpos = torch.cat([torch.arange(min(first, w0), device=DEV), torch.arange(w0, c + n, device=DEV)])
        keys = toks[s["token_table"][b, tpos // P].long() * P + tpos % P].double()
        ne = (c + n) // case["m"] if case["op"] == "chunk" else 0
        if ne:
            e = torch.arange(ne, device=DEV)
            at = s["entry_table"][b, e // P].long() * P + e % P
            f8 = val[s["codes"].view(-1, d - dr)[at].long()].view(ne, -1, grp) * s["scales"].view(-1, (d - dr) // grp)[at].double()[..., None]
            keys = torch.cat([keys, torch.cat([f8.reshape(ne, -1), s["rope"].view(-1, dr)[at].double()], 1)])
        for i0 in range(0, n, 256):
            p = torch.arange(c + i0, c + min(n, i0 + 256), device=DEV)
            q = s["q"][start[b] + i0:start[b] + i0 + p.numel()].double()
            if case["extras"]:
                q = _rot64(unit(q), p.double()[:, None] * fr)
            see = (tpos[None] <= p[:, None]) & ((tpos[None] > p[:, None] - W) | (tpos[None] < first))
            if ne:
                see = torch.cat([see, (e[None] + 1) * case["m"] - 1 <= p[:, None]], 1)
            lg = torch.einsum("nhd,kd->nhk", q, keys) * s["scale"]
            lg.masked_fill_(~see[:, None], -math.inf)
            top = lg.amax(-1, keepdim=True)
            if case["extras"]:
                top = torch.maximum(top, s["sink"].double()[None, :, None])
            w = torch.exp(lg - top)
            den = w.sum(-1, keepdim=True)
            if case["extras"]:
                den = den + torch.exp(s["sink"].double()[None, :, None] - top)
            o = torch.einsum("nhk,kd->nhd", w / den, keys)
            if case["extras"]:
                o = _rot64(o, -p.double()[:, None] * fr)
            out[start[b] + i0:start[b] + i0 + p.numel()] = o
    return out
