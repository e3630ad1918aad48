"""Paged serving calls against the oracle and plain restatements: block tables
and slot maps, token and entry stores (bit for bit), attention of ragged chunks
and single tokens over pages, and steps of all of them together.

Attention tolerance, per output element, from the roundings on the way (u16 =
2^-11, half a step of fp16; ub = 2^-8, half a step of bf16): an entry's scale is
rounded to fp16 and each product with a code once more, the query once, so a
logit is off by at most dl = scale * sum_i |q_i| |k_i| * (3 u16 + 2^-14), the
last term covering the fp32 sum of d <= 512 products (512 * 2^-23 = 2^-14 where
every addition truncates), plus 2^-12 for values below fp16's normal range
(2^-25 off each); a weight is then off by a factor within e^(+-2 dl) and P by
u16 more, the values by 2 u16, a split's partial by u16: |error| <= (e^(2 dl) -
1 + 4 u16) * sum_j p_j |v_j| + ub |o|.  That is a worst case; the mean is held
to what the workloads are held to: sum |a - b| / sum |b| <= 1e-3 for the
arithmetic plus 2^-9, the mean of a bf16 rounding (half of its largest).
"""
import numpy as np
import pytest
import torch

import hca_inputs as inp
import oracle
from gpu_util import host

pytestmark = pytest.mark.gpu

hca = pytest.importorskip("long_context_attention_hca_b200")

DEV = "cuda"
LAYOUTS = {512: (512, 64, 64), 128: (128, 32, 32)}
U16, UB = 2.0 ** -11, 2.0 ** -8


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def bf(shape, g, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(torch.bfloat16)


def f64(t):
    return t.detach().double().cpu().numpy()


# ------------------------------------------------------------------ plan
def plan_ref(ctx, new, m, P, table, free, n_free):
    """Request by request, item by item."""
    table = table.copy()
    free = list(free[:n_free])
    width = table.shape[1]
    start, req, pos, slot, missing = [0], [], [], [], 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        c, n = max(c, 0), max(n, 0)
        lo, hi = c // m, (c + n) // m
        for p in range(-(-lo // P), -(-hi // P)):
            if p >= width:
                missing += 1
            elif free:
                table[b, p] = free.pop()
            else:
                table[b, p] = -1
                missing += 1
        for i in range(lo, hi):
            pg = table[b, i // P] if i // P < width else -1
            req.append(b)
            pos.append(i)
            slot.append(int(pg) * P + i % P if pg >= 0 else -1)
        start.append(len(req))
    return table, start, req, pos, slot, missing, len(free)


@pytest.mark.parametrize("B,m,P,maxc,maxn,short", [
    (1, 1, 1, 0, 1, 0), (1, 1, 64, 1000, 1, 0), (5, 1, 16, 300, 40, 0), (33, 128, 16, 70000, 1500, 0),
    (700, 1, 48, 500, 90, 0), (1500, 4, 64, 3000, 64, 0), (16384, 1, 64, 40, 2, 0), (9, 1, 16, 200, 100, 7), (40, 4, 8, 900, 400, 1000)])
def test_plan(B, m, P, maxc, maxn, short):
    r = np.random.default_rng(B * 7 + m)
    ctx = r.integers(0, maxc + 1, B)
    new = np.where(r.random(B) < 0.3, 0, r.integers(0, maxn + 1, B))
    new[0] = maxn
    held = -(-(ctx // m) // P)
    want = -(-((ctx + new) // m) // P)
    width = max(1, int(want.max()) - (1 if short else 0))
    table = np.full((B, width), -7, np.int32)
    nid = 0
    for b in range(B):
        for p in range(min(int(held[b]), width)):
            table[b, p] = nid
            nid += 1
    free = r.permutation(np.arange(nid, nid + int((want - held).sum()) + 3)).astype(np.int32)
    n_free = max(0, len(free) - short)
    total = int(((ctx + new) // m - ctx // m).sum())
    plan = hca.PagePlan.empty(B, total + 5)
    t, f = i32(table), i32(free)
    got = hca.kv_page_plan(i32(ctx), i32(new), m, P, t, f, i32([n_free]), plan=plan)
    rt, start, req, pos, slot, missing, left = plan_ref(ctx.tolist(), new.tolist(), m, P, table, free.tolist(), n_free)
    assert got is plan
    assert plan.row_start.tolist() == start
    assert plan.row_req.tolist() == req + [-1] * 5
    assert plan.row_pos.tolist() == pos + [-1] * 5
    assert plan.slot.tolist() == slot + [-1] * 5
    assert plan.missing.tolist() == [missing] and plan.free_left.tolist() == [left]
    assert np.array_equal(t.cpu().numpy(), rt) and np.array_equal(f.cpu().numpy(), free)


def test_plan_fewer_rows_than_items_negative_lengths_and_no_requests():
    t = torch.full((3, 4), -1, dtype=torch.int32, device=DEV)
    plan = hca.PagePlan.empty(3, 5)
    hca.kv_page_plan(i32([-4, 3, 0]), i32([6, -2, 4]), 1, 4, t, i32([5, 6, 7, 8]), i32([99]), plan=plan)
    assert plan.row_start.tolist() == [0, 6, 6, 10]
    assert plan.slot.tolist() == [32, 33, 34, 35, 28] and plan.row_req.tolist() == [0] * 5
    assert t.tolist() == [[8, 7, -1, -1], [-1] * 4, [6, -1, -1, -1]] and plan.free_left.tolist() == [1]
    none = hca.kv_page_plan(i32([]), i32([]), 1, 4, torch.zeros((0, 2), dtype=torch.int32, device=DEV), i32([1, 2]),
                            i32([2]), max_rows=3)
    assert none.row_start.tolist() == [0] and none.free_left.tolist() == [2] and none.slot.tolist() == [-1] * 3


def test_plans_of_many_requests_from_two_threads():
    """Beyond 6000 requests a plan asks for more shared memory than a launch has
    by itself: calls of different B at once, each with the same answer as alone."""
    import threading
    jobs, errors = [], []
    for B in (16384, 6500):
        ctx, new = i32(np.arange(B) % 50), i32(np.arange(B) % 3)
        plan = lambda n=3 * B: hca.PagePlan.empty(B, n)
        table = torch.full((B, 1), -1, dtype=torch.int32, device=DEV)
        jobs.append((ctx, new, table, i32(np.arange(B)), i32([B]), plan(), plan(), torch.cuda.Stream()))
    for ctx, new, table, free, count, want, _, _ in jobs:
        hca.kv_page_plan(ctx, new, 1, 64, table, free, count, plan=want)
    torch.cuda.synchronize()
    for job in jobs:
        job[2].fill_(-1)
    torch.cuda.synchronize()

    def work(ctx, new, table, free, count, want, got, stream):
        try:
            for _ in range(200):
                hca.kv_page_plan(ctx, new, 1, 64, table, free, count, plan=got, stream=stream)
        except Exception as e:                          # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    assert not errors
    for *_, want, got, _ in jobs:
        assert torch.equal(want.slot, got.slot) and torch.equal(want.row_start, got.row_start)
        assert torch.equal(want.free_left, got.free_left)


# ------------------------------------------------------------------ stores
@pytest.mark.parametrize("d", [128, 512])
@pytest.mark.parametrize("extras", ["none", "norm", "rope", "both"])
def test_store_bits(d, extras):
    layout = LAYOUTS[d]
    g = gen(d + len(extras))
    n, P, pages = 37, 6, 11
    x = bf((n + 2, d), g)
    pos = torch.randint(0, 1 << 20, (n + 2,), generator=g, device=DEV).to(torch.int32)
    slot = torch.randperm(P * pages, generator=g, device=DEV)[:n + 2]
    slot[3], slot[8] = -1, P * pages
    nw = 1.0 + 0.1 * torch.randn(d, generator=g, device=DEV) if extras in ("norm", "both") else None
    fr = inp.rope_inv_freq(layout[1], device=DEV) if extras in ("rope", "both") else None
    ee = None if extras == "none" else hca.EntryExtras(nw, 1e-6, fr)
    plan = hca.PagePlan(i32([0, 20, n]), i32([0] * (n + 2)), pos, slot)
    pool = torch.full((pages, P, d), 7.0, dtype=torch.bfloat16, device=DEV)
    assert hca.kv_page_store(x, plan, pool, layout, extras=ee) is pool
    kw = {} if ee is None else dict(norm_w=None if nw is None else host(nw), eps=1e-6,
                                    inv_freq=None if fr is None else host(fr))
    want = host(torch.full((pages * P, d), 7.0, dtype=torch.bfloat16))
    y = host(x) if ee is None else oracle.token_prep(host(x), pos.cpu().numpy(), layout[1], **kw)
    for t in range(n):
        s = int(slot[t])
        if 0 <= s < pages * P:
            want[s] = y[t]
    assert np.array_equal(host(pool).reshape(-1, d), want)


class Pool:
    """Pages, block tables and free stack of one kind of item for B requests."""

    def __init__(self, B, max_items, P, seed, spare=2):
        self.P, self.width = P, max(1, -(-max_items // P))
        n = B * self.width + spare
        self.pages = n
        self.table = torch.full((B, self.width), -1, dtype=torch.int32, device=DEV)
        self.free = torch.randperm(n, generator=gen(seed), device=DEV).to(torch.int32)
        self.count = i32([n])

    def plan(self, ctx, new, m, max_rows):
        p = hca.kv_page_plan(ctx, new, m, self.P, self.table, self.free, self.count, max_rows=max_rows)
        self.count = p.free_left
        return p

    def rows(self, b, n):
        t = self.table[b].cpu().numpy().astype(np.int64)
        i = np.arange(n)
        return t[i // self.P] * self.P + i % self.P


@pytest.mark.parametrize("d,m,extras,P", [(128, 4, False, 5), (128, 128, True, 2), (512, 4, True, 16), (512, 128, False, 3),
                                          (512, 128, True, 16)])
def test_compress_bits_over_ragged_steps(d, m, extras, P):
    """Random step lengths (none, one, many): every entry equals the oracle's
    pooling of the whole sequence, whatever the steps cut its block into."""
    layout = LAYOUTS[d]
    g = gen(d + m)
    B, T = 5, 700 if m == 128 else 90
    x, gate = bf((B, T, d), g), bf((B, T, d), g)
    bias = torch.randn((m, d), generator=g, device=DEV) * 0.5
    nw = 1.0 + 0.1 * torch.randn(d, generator=g, device=DEV)
    fr = inp.rope_inv_freq(layout[1], device=DEV)
    ee = hca.EntryExtras(nw, 1e-6, fr) if extras else None
    kw = dict(norm_w=host(nw), eps=1e-6, inv_freq=host(fr)) if extras else {}
    rc, rs, rr = oracle.compress(host(x), host(gate), host(bias), m, T // m, layout[1], layout[2], **kw)[:3]
    pool = Pool(B, T // m + 1, P, 1)
    cache = hca.KVCache(pool.pages, P, layout, zero=True)
    tx, tg = torch.zeros((B, m, d), dtype=torch.bfloat16, device=DEV), torch.zeros((B, m, d), dtype=torch.bfloat16, device=DEV)
    r = np.random.default_rng(3)
    ctx = np.zeros(B, np.int64)
    for step in range(14):
        top = {0: 1, 1: m, 2: 3 * m + 1}[step % 3]
        new = np.minimum(np.where(r.random(B) < 0.2, 0, r.integers(0, top + 1, B)), T - ctx)
        if new.sum() == 0:
            continue
        xs = torch.cat([x[b, ctx[b]:ctx[b] + new[b]] for b in range(B)])
        gs = torch.cat([gate[b, ctx[b]:ctx[b] + new[b]] for b in range(B)])
        starts = i32(np.concatenate([[0], np.cumsum(new)]))
        plan = pool.plan(i32(ctx), i32(new), m, int(((ctx + new) // m - ctx // m).sum()) + 2)
        hca.kv_page_compress(xs, gs, bias, starts, i32(ctx), plan, tx, tg, cache, extras=ee)
        ctx = ctx + new
        for b in range(B):
            n = int(ctx[b]) % m
            assert torch.equal(tx[b, :n], x[b, ctx[b] - n:ctx[b]]) and torch.equal(tg[b, :n], gate[b, ctx[b] - n:ctx[b]])
    dn = layout[0] - layout[1]
    for b in range(B):
        k = int(ctx[b]) // m
        at = pool.rows(b, k)
        assert np.array_equal(host(cache.codes).reshape(-1, dn)[at], rc[b, :k])
        assert np.array_equal(host(cache.scales).view(np.uint32).reshape(-1, dn // layout[2])[at], rs[b, :k].view(np.uint32))
        assert np.array_equal(host(cache.rope).reshape(-1, layout[1])[at], rr[b, :k])
    assert (ctx // m).sum() > B
    untouched = np.ones(pool.pages * P, bool)
    for b in range(B):
        untouched[pool.rows(b, int(ctx[b]) // m)] = False
    assert not host(cache.codes).reshape(-1, dn)[untouched].any()


def test_plan_accepts_slices_and_repeats():
    """Integer arrays may be slices of longer ones; the same call twice gives the same plan (nothing is consumed)."""
    big = torch.arange(100, dtype=torch.int32, device=DEV)
    lens = i32([9, 7, 20, 1, 30])
    t = torch.full((3, 9), -1, dtype=torch.int32, device=DEV)
    t[0, :2], t[1, :3] = i32([91, 92]), i32([93, 94, 95])
    a = hca.kv_page_plan(lens[1:4], lens[:3], 1, 4, t, big[7:50], big[37:38], max_rows=40)
    first = (t.clone(), a.slot.clone(), a.free_left.clone())
    b = hca.kv_page_plan(lens[1:4], lens[:3], 1, 4, t, big[7:50], big[37:38], max_rows=40)
    assert torch.equal(t, first[0]) and torch.equal(b.slot, first[1]) and torch.equal(b.free_left, first[2])
    assert a.row_start.tolist() == [0, 9, 16, 36] and a.slot[:3].tolist() == [92 * 4 + 3, 43 * 4, 43 * 4 + 1]


@pytest.mark.parametrize("m", [4, 128])
def test_compress_without_a_page(m):
    """Entries that got no page are not stored, the others are, and the tails move on all the same."""
    d, B = 128, 3
    g = gen(m)
    new = [2 * m + 3, m + 1, m - 1]
    x, gate = bf((sum(new), d), g), bf((sum(new), d), g)
    bias = torch.randn((m, d), generator=g, device=DEV) * 0.5
    table = torch.full((B, 4), -1, dtype=torch.int32, device=DEV)
    ctx, nl = i32([0] * B), i32(new)
    plan = hca.kv_page_plan(ctx, nl, m, 1, table, i32([5, 2]), i32([2]), max_rows=6)
    assert plan.missing.tolist() == [1] and plan.slot.tolist() == [2, 5, -1, -1, -1, -1]
    cache = hca.KVCache(8, 1, LAYOUTS[d], zero=True)
    tx, tg = torch.zeros((B, m, d), dtype=torch.bfloat16, device=DEV), torch.zeros((B, m, d), dtype=torch.bfloat16, device=DEV)
    starts = i32(np.concatenate([[0], np.cumsum(new)]))
    hca.kv_page_compress(x, gate, bias, starts, ctx, plan, tx, tg, cache)
    ref = oracle.compress(host(x[None, :2 * m]), host(gate[None, :2 * m]), host(bias), m, 2, 32, 32)[0]
    codes = host(cache.codes).reshape(8, -1)
    assert np.array_equal(codes[[2, 5]], ref[0])
    assert not np.delete(codes, [2, 5], 0).any()
    assert torch.equal(tx[0, :3], x[2 * m:2 * m + 3]) and torch.equal(tx[1, 0], x[2 * m + 3 + m]) and torch.equal(tx[2, :m - 1], x[-(m - 1):])


# ------------------------------------------------------------------ attention
def entry_cache(pages, P, layout, g):
    d, dr, grp = layout
    y = torch.randn((pages, P, (d - dr) // grp, grp), generator=g, device=DEV) * 0.5
    sc = y.abs().amax(-1) / 448.0
    codes = (y / sc[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).reshape(pages, P, d - dr)
    return hca.KVCache.of(codes.contiguous(), sc.contiguous(), bf((pages, P, dr), g, 0.5))


class Case:
    def __init__(self, d, H, ctx, new, W, m=0, n_first=0, PE=16, PT=16, extras=False, seed=0, pad=3):
        self.__dict__.update(d=d, H=H, ctx=list(ctx), new=list(new), W=W, m=m, n_first=n_first, extras=extras)
        layout = self.layout = LAYOUTS[d]
        g = gen(1000 + seed)
        B, N = len(ctx), sum(new)
        self.N, self.starts = N, np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
        end = [c + n for c, n in zip(ctx, new)]
        self.PT, self.PE = PT, PE
        self.tw = max(1, max(-(-e // PT) for e in end))
        npt = B * self.tw + 1
        self.ttab = torch.randperm(npt, generator=g, device=DEV)[:B * self.tw].view(B, self.tw).to(torch.int32).contiguous()
        self.pages = bf((npt, PT, d), g)
        self.cache = self.etab = None
        if m:
            self.ew = max(1, max(-(-(e // m) // PE) for e in end))
            npe = B * self.ew + 1
            self.etab = torch.randperm(npe, generator=g, device=DEV)[:B * self.ew].view(B, self.ew).to(torch.int32).contiguous()
            self.cache = entry_cache(npe, PE, layout, g)
        self.q = bf((N + pad, H, d), g)
        self.scale = d ** -0.5
        self.ex, self.kw, self.lens = None, {}, None
        if extras:
            nw, sink = 1.0 + 0.1 * torch.randn(d, generator=g, device=DEV), torch.randn(H, generator=g, device=DEV)
            fr = inp.rope_inv_freq(layout[1], device=DEV)
            self.ex = hca.AttnExtras(nw, 1e-6, sink, fr)
            self.kw = dict(q_norm_w=host(nw), eps=1e-6, sink=host(sink), inv_freq=host(fr))

    def run(self, max_new=None, out=None, ws=None, stream=None, q=None):
        if self.lens is None or self.lens[0] != self.ctx:
            # kept: a call on another stream still reads them after run() has returned
            self.lens = (list(self.ctx), i32(self.starts), i32(self.ctx))
            torch.cuda.synchronize()
        a = (self.q if q is None else q, *self.lens[1:])
        kw = dict(max_new=max_new, out=out, ws=ws, stream=stream, extras=self.ex)
        if self.m:
            return hca.paged_attn_chunk(*a, self.m, self.cache, self.etab, self.pages, self.ttab, self.W, self.scale, **kw)
        return hca.paged_attn_window(*a, self.pages, self.ttab, self.W, self.n_first, self.scale, **kw)

    def keys(self, b, p):
        """(pool rows of the entries, pool rows of the tokens) that the query at position p of request b sees."""
        ents, first, end = oracle.causal_keys(p, self.m, self.W)
        toks = np.array(sorted(set(range(first, end)) | set(range(min(self.n_first, p + 1)))))
        tt = self.ttab[b].cpu().numpy().astype(np.int64)
        rows_t = tt[toks // self.PT] * self.PT + toks % self.PT
        rows_e = np.zeros(0, np.int64)
        if len(ents):
            et = self.etab[b].cpu().numpy().astype(np.int64)
            rows_e = et[ents // self.PE] * self.PE + ents % self.PE
        return rows_e, rows_t

    def pools(self):
        d, dr, g = self.layout
        if self.cache is None:
            e = (np.zeros((1, d - dr), np.uint8), np.zeros((1, (d - dr) // g), np.float32), np.zeros((1, dr), np.uint16))
        else:
            e = (host(self.cache.codes).reshape(-1, d - dr), host(self.cache.scales).reshape(-1, (d - dr) // g),
                 host(self.cache.rope).reshape(-1, dr))
        return e, host(self.pages).reshape(-1, d)

    def reference(self, rows=None):
        """{row: (fp64 output [H][d], bound of the error)}"""
        (c, s, r), toks = self.pools()
        d, dr, g = self.layout
        qh = host(self.q)
        val = torch.from_numpy(np.arange(256, dtype=np.uint8)).view(torch.float8_e4m3fn).double().numpy()
        out = {}
        for b in range(len(self.ctx)):
            for i in range(self.new[b]):
                n = int(self.starts[b]) + i
                if rows is not None and n not in rows:
                    continue
                p = self.ctx[b] + i
                re, rt = self.keys(b, p)
                o, _ = oracle.attend(qh[n], c, s, r, re, toks[rt], self.scale, g, q_pos=p, **self.kw)
                # the bound: prepared query, keys in fp64, the softmax's own weights
                q = oracle.bf16_to_f32(qh[n]).astype(np.float64)
                if self.extras:
                    q = q / np.sqrt((q * q).mean(-1, keepdims=True) + 1e-6) * self.kw["q_norm_w"]
                    q[:, d - dr:] = np.stack([oracle.rope_f64(v, p, self.kw["inv_freq"]) for v in q[:, d - dr:]])
                k = oracle.bf16_to_f32(toks[rt]).astype(np.float64)
                if len(re):
                    e = np.concatenate([val[c[re]] * np.repeat(s[re].astype(np.float64), g, 1),
                                        oracle.bf16_to_f32(r[re]).astype(np.float64)], 1)
                    k = np.concatenate([e, k])
                lg = q @ k.T * self.scale
                top = lg.max(1, keepdims=True)
                if self.extras:
                    top = np.maximum(top, self.kw["sink"][:, None])
                w = np.exp(lg - top)
                w /= w.sum(1, keepdims=True) + (np.exp(self.kw["sink"][:, None] - top) if self.extras else 0)
                dl = self.scale * (np.abs(q) @ np.abs(k).T).max(1, keepdims=True) * (3 * U16 + 2.0 ** -14) + 2.0 ** -12
                pv = w @ np.abs(k)
                if self.extras:                          # the rotation back mixes a pair's errors
                    pr = pv[:, d - dr:]
                    pr[:, 0::2] = pr[:, 1::2] = pr[:, 0::2] + pr[:, 1::2]
                out[n] = (o, (np.exp(2 * dl) - 1 + 4 * U16) * pv + UB * np.abs(o) + 1e-6)
        return out

    def check(self, got, rows=None, mean=True):
        ref = self.reference(rows)
        g = f64(got)
        num = den = 0.0
        for n, (o, tol) in ref.items():
            err = np.abs(g[n] - o)
            assert np.all(err <= tol), (n, float((err - tol).max()), float(err.max()))
            num += err.sum()
            den += np.abs(o).sum()
        assert not mean or num <= (1e-3 + 2.0 ** -9) * den, num / den
        assert hca.take_device_error() == 0


CASES = [
    # single tokens
    dict(d=512, H=64, ctx=[1000, 5, 0, 4095], new=[1, 1, 1, 1], W=128, m=128),
    dict(d=512, H=64, ctx=[30000], new=[1], W=128, m=4, PE=32),
    dict(d=128, H=8, ctx=[1000, 127, 0, 64, 255], new=[1, 1, 1, 0, 1], W=128, m=128),
    dict(d=128, H=1, ctx=[17, 300], new=[1, 1], W=7, n_first=3),
    # chunks
    dict(d=512, H=64, ctx=[0, 500, 127, 9], new=[5, 0, 3, 1], W=128, m=128, PE=1, PT=5),
    dict(d=512, H=64, ctx=[2000, 383], new=[17, 2], W=100, m=128, extras=True),
    dict(d=512, H=64, ctx=[2000, 0, 130], new=[3, 9, 6], W=128, n_first=4, extras=True),
    dict(d=512, H=64, ctx=[77], new=[130], W=64, m=4, PE=48, PT=48),
    dict(d=512, H=5, ctx=[600, 3], new=[30, 7], W=33, m=128, extras=True, PT=1),
    dict(d=512, H=128, ctx=[300], new=[3], W=128, m=4),
    dict(d=128, H=8, ctx=[1023, 0, 200], new=[40, 21, 1], W=128, m=128, extras=True),
    dict(d=128, H=64, ctx=[90, 91], new=[2, 66], W=17, m=4, PE=7, PT=9),
    dict(d=128, H=3, ctx=[500, 1, 60], new=[50, 3, 1], W=16, n_first=64, extras=True),
    dict(d=128, H=16, ctx=[0], new=[1], W=1),
    dict(d=512, H=64, ctx=[5, 0], new=[4, 70], W=1, n_first=1),
    dict(d=512, H=64, ctx=[100, 4000], new=[70, 65], W=128, n_first=200),
    dict(d=512, H=64, ctx=[0], new=[4], W=1, n_first=0),
    dict(d=512, H=64, ctx=[63, 1, 700, 0], new=[64, 5, 1, 4], W=64, m=4, PE=64, PT=64),
    dict(d=512, H=7, ctx=[3000, 10, 0], new=[41, 60, 2], W=128, m=4, PE=5, PT=3, extras=True),
    dict(d=512, H=1, ctx=[900], new=[300], W=70, n_first=5, extras=True),
    dict(d=512, H=64, ctx=[20000, 9000], new=[6, 8], W=128, m=4, extras=True),
]


@pytest.mark.parametrize("k", range(len(CASES)))
def test_attention(k):
    c = Case(seed=k, **CASES[k])
    out = torch.full_like(c.q, 7.0)
    got = c.run(out=out, max_new=max(c.new))
    assert torch.all(got[c.N:] == 7.0)                   # rows behind the last request
    c.check(got)


@pytest.mark.parametrize("k", [4, 7, 12])
def test_attention_without_the_bound(k):
    """max_new only chooses kernels: none, too large and too small give results of the same tolerance."""
    c = Case(seed=k, **CASES[k])
    for mn in (None, 1, 10 ** 6):
        c.check(c.run(max_new=mn))


def test_attention_many_splits_and_long_offsets():
    """One decode request over 20000 entries (every SM takes a split), pages far into a large pool."""
    c = Case(512, 64, [20000 * 4 - 1], [1], 128, m=4, PE=64, PT=64)
    c.check(c.run(max_new=1))


@pytest.mark.parametrize("k", [0, 6, 8])
def test_tables_too_wide_to_stage(k):
    """Tables whose entries would take more workspace than is staged: the row kernel serves d = 512 as well."""
    c = Case(seed=k, **{**CASES[k], "m": CASES[k].get("m") or 4, "n_first": 0})
    wide = torch.full((len(c.ctx), (3 << 20) // c.PE), -1, dtype=torch.int32, device=DEV)
    wide[:, :c.ew] = c.etab
    narrow, c.etab = c.etab, wide
    got = c.run(max_new=max(c.new))
    assert hca.paged_attn_workspace_size(c.q.shape[0], len(c.ctx), c.H, c.layout, max(c.new), wide.shape[1] * c.PE, c.W) < 1 << 29
    c.etab = narrow
    c.check(got)


def test_no_new_tokens_and_padded_rows():
    """Requests without new tokens only, and a padded batch: nothing but the live rows is written."""
    for d, H in ((512, 64), (128, 8)):
        c = Case(d, H, [300, 20, 5], [2, 0, 3], 64, m=4, pad=200)
        want = c.run()
        out = torch.full_like(c.q, 7.0)
        got = c.run(out=out)
        assert torch.equal(got[:5], want[:5]) and torch.all(got[5:] == 7.0)
        c.starts, c.lens = np.zeros(4, np.int64), None
        assert torch.all(c.run(out=torch.full_like(c.q, 7.0)) == 7.0)


def test_outputs_on_a_16_byte_boundary():
    """out, q and ws need 16-byte alignment only (no wider store is assumed)."""
    for kw in (CASES[4], CASES[8], CASES[1]):
        c = Case(seed=3, **kw)
        want = c.run()
        n = c.q.numel()
        flat = torch.zeros(n + 8, dtype=torch.bfloat16, device=DEV)
        q = torch.empty(n + 8, dtype=torch.bfloat16, device=DEV)[8:].view_as(c.q)
        q.copy_(c.q)
        need = hca.paged_attn_workspace_size(c.q.shape[0], len(c.ctx), c.H, c.layout, 0, c.ew * c.PE if c.m else 0, c.W, c.n_first)
        ws = torch.empty(need + 16, dtype=torch.uint8, device=DEV)[16:]
        got = c.run(q=q, out=flat[8:].view_as(c.q), ws=ws)
        assert torch.equal(got[:c.N], want[:c.N]) and torch.all(flat[:8] == 0)


def test_a_query_that_is_not_finite_stays_alone():
    for d, H in ((512, 64), (128, 8)):
        c = Case(d, H, [500, 40], [6, 3], 64, m=4)
        clean = c.run()
        c.q[2, 1, 7] = float("inf")
        c.q[4, 3, 0] = float("nan")
        got = c.run()
        assert torch.isnan(got[2, 1]).all() and torch.isnan(got[4, 3]).all()
        keep = torch.ones((9, H), dtype=torch.bool, device=DEV)
        keep[2, 1] = keep[4, 3] = False
        assert torch.equal(got[:9][keep], clean[:9][keep])


def test_many_requests_of_mixed_lengths():
    """More requests than a search round has lanes, most without new tokens; sampled rows against the oracle."""
    r = np.random.default_rng(5)
    for d, H in ((512, 64), (128, 8)):
        ctx = r.integers(0, 700, 130).tolist()
        new = np.where(r.random(130) < 0.6, 0, r.integers(1, 9, 130)).tolist()
        c = Case(d, H, ctx, new, 40, m=4, PE=8, PT=8, extras=True)
        c.check(c.run(max_new=8), rows=set(r.integers(0, c.N, 25).tolist()))


def test_token_rows_beyond_32_bits():
    """A pool of more than 2^32 elements: the last pages are the request's."""
    c = Case(512, 64, [200], [3], 128, n_first=4, PT=64)
    n = (1 << 32) // (64 * 512) + 8
    big = torch.empty((n, 64, 512), dtype=torch.bfloat16, device=DEV)
    last = torch.arange(n - c.pages.shape[0], n, device=DEV)
    big[last] = c.pages
    small, table = c.pages, c.ttab
    c.pages, c.ttab = big, (table + (n - small.shape[0])).to(torch.int32)
    got = c.run()
    c.pages, c.ttab = small, table
    c.check(got)


def test_unused_page_rows_may_hold_anything():
    """NaN, infinities and garbage everywhere but in the visible keys' rows change nothing."""
    for k in (0, 4, 6, 12):
        c = Case(seed=k, **CASES[k])
        clean = c.run()
        used_t, used_e = set(), set()
        for b in range(len(c.ctx)):
            for i in range(c.new[b]):
                re, rt = c.keys(b, c.ctx[b] + i)
                used_t |= set(rt.tolist())
                used_e |= set(re.tolist())
        free_t = [r for r in range(c.pages.shape[0] * c.PT) if r not in used_t]
        c.pages.view(-1, c.d)[free_t] = float("nan")
        if c.cache is not None:
            free_e = [r for r in range(c.cache.B * c.PE) if r not in used_e]
            c.cache.codes.view(-1, c.cache.codes.shape[2])[free_e] = 0x7F
            c.cache.scales.view(-1, c.cache.scales.shape[2])[free_e] = float("inf")
            c.cache.rope.view(-1, c.cache.rope.shape[2])[free_e] = float("-inf")
        assert torch.equal(c.run()[:c.N], clean[:c.N])


@pytest.mark.parametrize("d,H", [(512, 64), (128, 8)])
def test_non_finite_key_reaches_only_the_queries_that_see_it(d, H):
    c = Case(d, H, [300], [12], 20, m=4, PT=8)
    clean = c.run()
    p_bad = 306                                          # a token of the step itself
    row = int(c.ttab[0, p_bad // 8]) * 8 + p_bad % 8
    c.pages.view(-1, d)[row, 3] = float("inf")
    e_bad = 76                                           # visible from position 307 on
    er = int(c.etab[0, e_bad // 16]) * 16 + e_bad % 16
    c.cache.codes.view(-1, c.cache.codes.shape[2])[er, 5] = 0x7F
    got = c.run()
    for i in range(12):
        if 300 + i >= p_bad:
            assert torch.isnan(got[i]).all()
        else:
            assert torch.equal(got[i], clean[i])


def test_pages_outside_the_pool_are_not_visible():
    c = Case(512, 64, [100, 40, 900], [2, 3, 2], 32, m=4, PT=16, PE=4)
    ref = Case(512, 64, [100, 40, 900], [2, 3, 2], 32, m=4, PT=16, PE=4)
    c.etab[0, 3], c.etab[2, 0] = -1, c.cache.B           # entries 12..15 of request 0, 0..3 of request 2
    c.ttab[1, :] = c.pages.shape[0] + 5                  # request 1 has no token at all ...
    c.etab[1, :] = -(1 << 31)                            # ... and no entry: nothing is visible
    got = c.run()
    keys = ref.keys

    def without(b, p):
        re, rt = keys(b, p)
        if b == 0:
            re = np.delete(re, np.arange(12, 16))
        if b == 2:
            re = re[4:]
        return re, rt
    ref.keys = without
    ref.check(got, rows=[0, 1, 5, 6])
    assert torch.all(got[2:5] == 0)


def test_sink_without_keys_and_large_sinks():
    c = Case(128, 8, [10], [2], 8, m=4, extras=True)
    c.ttab[:] = -1
    c.etab[:] = -1
    assert torch.all(c.run()[:2] == 0)
    c = Case(512, 64, [10], [3], 8, m=4, extras=True)
    c.ex.sink[:] = 80.0
    assert torch.all(c.run()[:3].abs() < 1e-20)


@pytest.mark.parametrize("new", [[1], [40]])
def test_maxima_that_keep_growing(new):
    """Later keys give larger and larger logits (the running maximum moves, O is
    rescaled again and again); worst-case bound only, since such logits amplify
    the operands' roundings."""
    c = Case(512, 64, [1500], new, 128, m=4, PE=64, PT=64)
    e = c.etab[0].long()
    c.cache.scales[e] *= torch.linspace(0.2, 12.0, c.ew * 64, device=DEV).view(c.ew, 64, 1)
    t = c.ttab[0].long()
    c.pages[t] = (c.pages[t].float() * torch.linspace(0.5, 20.0, c.tw * 64, device=DEV).view(c.tw, 64, 1)).to(torch.bfloat16)
    c.check(c.run(), mean=False)


def test_queries_of_zero_give_the_mean():
    c = Case(512, 64, [700], [4], 128, m=128)
    c.q.zero_()
    c.check(c.run())


def test_streams_graphs_and_two_calls_at_once():
    c = Case(seed=4, **CASES[4])
    e = Case(seed=1, **CASES[1])
    want, wante = c.run(max_new=5), e.run(max_new=1)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        a, b = c.run(max_new=5, stream=s1), e.run(max_new=1, stream=s2)
        torch.cuda.synchronize()
        assert torch.equal(a[:c.N], want[:c.N]) and torch.equal(b[:e.N], wante[:e.N])
    # two captured steps, each with its own buffers, replayed side by side; new lengths between replays
    cap = torch.cuda.Stream()
    cap.wait_stream(torch.cuda.current_stream())
    starts, ctx = i32(c.starts), i32(c.ctx)
    out, oute = torch.zeros_like(c.q), torch.zeros_like(e.q)
    st_e, ctx_e = i32(e.starts), i32(e.ctx)
    with torch.cuda.stream(cap):
        g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g1, stream=cap):
            hca.paged_attn_chunk(c.q, starts, ctx, c.m, c.cache, c.etab, c.pages, c.ttab, c.W, c.scale, max_new=5, out=out)
        with torch.cuda.graph(g2, stream=cap):
            hca.paged_attn_chunk(e.q, st_e, ctx_e, e.m, e.cache, e.etab, e.pages, e.ttab, e.W, e.scale, max_new=1, out=oute)
    torch.cuda.synchronize()
    for _ in range(3):
        out.zero_(), oute.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            g1.replay()
        with torch.cuda.stream(s2):
            g2.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[:c.N], want[:c.N]) and torch.equal(oute[:e.N], wante[:e.N])
    ctx_e.fill_(29000)
    g2.replay()
    torch.cuda.synchronize()
    e.ctx = [29000]
    assert torch.equal(oute[:1], e.run(max_new=1)[:1])


def test_same_call_same_bytes():
    for k in (1, 5, 7):
        c = Case(seed=k, **CASES[k])
        a = c.run()
        assert all(torch.equal(a[:c.N], c.run()[:c.N]) for _ in range(3))


def test_refusals_of_the_binding():
    c = Case(128, 8, [10], [2], 8, m=4)
    with pytest.raises(TypeError):
        c.run(q=c.q.float())
    with pytest.raises(ValueError):
        c.run(q=c.q.transpose(0, 1))
    with pytest.raises(ValueError):
        c.run(out=c.q[:1])
    with pytest.raises(ValueError):
        hca.paged_attn_window(c.q.cpu(), i32(c.starts), i32(c.ctx), c.pages, c.ttab, 8, 0, c.scale)
    with pytest.raises(ValueError):
        hca.paged_attn_window(c.q, i32(c.starts)[:-1], i32(c.ctx), c.pages, c.ttab, 8, 0, c.scale)
    for W, first, scale in ((0, 0, 1.0), (5000, 0, 1.0), (8, -1, 1.0), (8, 0, 0.0), (8, 0, float("nan"))):
        with pytest.raises(hca.HCAError):
            hca.paged_attn_window(c.q, i32(c.starts), i32(c.ctx), c.pages, c.ttab, W, first, scale)
    big = Case(512, 64, [30000], [1], 128, m=4)
    assert hca.paged_attn_workspace_size(big.q.shape[0], 1, 64, big.layout, 1, big.ew * 16, 128) > 16
    with pytest.raises(hca.HCAError):
        big.run(max_new=1, ws=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        hca.KVCache.of(big.cache.codes, big.cache.scales[:, :, :3].contiguous(), big.cache.rope)
    with pytest.raises(ValueError):
        hca.kv_page_plan(i32([1]), i32([1]), 1, 4, i32([[0]]), i32([1]), i32([1]))


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("d,H,section9", [(128, 8, False), (128, 8, True), (512, 64, True)])
def test_steps_of_a_ragged_batch(d, H, section9):
    """Requests join, prefill in chunks, decode and idle together over a window
    layer (ratio 0, first tokens visible) and an HCA layer (ratio 128): plan,
    store, compress and attention of every step against the oracle's own
    pooling and attention over the whole sequences."""
    from long_context_attention_hca_b200.pipeline import PagedLoop
    layout = LAYOUTS[d]
    dr, grp = layout[1], layout[2]
    W, first, B, T, m = 64, 3, 4, 420, 128
    g = gen(900 + d + section9)
    ratios = [0, m]
    x = [bf((B, T, d), g) for _ in ratios]
    gate = [bf((B, T, d), g) for _ in ratios]
    bias = torch.randn((m, d), generator=g, device=DEV) * 0.5
    s9 = None
    if section9:
        s9 = [{"kv_norm_w": 1.0 + 0.1 * torch.randn((d,), generator=g, device=DEV),
               "q_norm_w": 1.0 + 0.1 * torch.randn((d,), generator=g, device=DEV),
               "sink": torch.randn((H,), generator=g, device=DEV),
               "inv_freq": inp.rope_inv_freq(dr, device=DEV), "eps": 1e-6} for _ in ratios]
    loop = PagedLoop(B, H, layout, ratios, W, first, max_tokens=T, max_rows=260, softmax_scale=d ** -0.5,
                     token_page=16, entry_page=2, s9=s9)
    loop.set_bias(1, bias)
    kw = {} if not section9 else dict(norm_w=host(s9[1]["kv_norm_w"]), eps=1e-6, inv_freq=host(s9[1]["inv_freq"]))
    ent = oracle.compress(host(x[1]), host(gate[1]), host(bias), m, T // m, dr, grp, **kw)[:3]
    steps = [[130, 0, 3, 0], [1, 0, 1, 60], [127, 40, 1, 1], [1, 1, 0, 1], [0, 88, 90, 67], [60, 1, 33, 1], [1, 1, 1, 0]]
    ctx = np.zeros(B, np.int64)
    for new in steps:
        new = np.array(new)
        N = int(new.sum())
        cat = lambda t: torch.cat([t[b, ctx[b]:ctx[b] + new[b]] for b in range(B)])
        q = [bf((N, H, d), g) for _ in ratios]
        out = loop.step(i32(new), [cat(t) for t in x], [cat(t) for t in gate], q, max_new=int(new.max()))
        torch.cuda.synchronize()
        starts = np.concatenate([[0], np.cumsum(new)])
        for li, r in enumerate(ratios):
            for b in range(B):
                for i in range(int(new[b])):
                    if i % 11 and i != new[b] - 1:
                        continue
                    p = int(ctx[b] + i)
                    ents, w0, w1 = oracle.causal_keys(p, r, W)
                    tk = sorted(set(range(w0, w1)) | (set(range(min(first, p + 1))) if r == 0 else set()))
                    win = host(x[li])[b, tk]
                    akw = {}
                    if section9:
                        P = s9[li]
                        win = oracle.token_prep(win, np.array(tk), dr, norm_w=host(P["kv_norm_w"]), eps=1e-6,
                                                inv_freq=host(P["inv_freq"]))
                        akw = dict(q_norm_w=host(P["q_norm_w"]), eps=1e-6, sink=host(P["sink"]),
                                   inv_freq=host(P["inv_freq"]), q_pos=p)
                    n = int(starts[b]) + i
                    e = [a[b] for a in ent]
                    ref, _ = oracle.attend(host(q[li])[n], *e, ents, win, d ** -0.5, grp, **akw)
                    err = np.abs(f64(out[li])[n] - ref)
                    assert err.max() <= 1e-2 + UB * np.abs(ref).max(), (li, b, p, err.max())
                    assert err.sum() <= (1e-3 + 2.0 ** -9) * np.abs(ref).sum() + 1e-4 * ref.size, (li, b, p)
        ctx += new
        assert loop.ctx.tolist() == ctx.tolist() and loop.missing() == 0


def test_released_requests_give_their_pages_back():
    from long_context_attention_hca_b200.pipeline import PagedLoop
    d, H, B, T = 128, 8, 2, 300
    g = gen(31)
    x, gate = bf((T, d), g), bf((T, d), g)
    bias = torch.randn((128, d), generator=g, device=DEV) * 0.5
    q = bf((T, H, d), g)
    loop = PagedLoop(B, H, LAYOUTS[d], [128], 32, 0, max_tokens=T, max_rows=T, softmax_scale=d ** -0.5, token_page=16,
                     entry_page=1, token_pages=20, entry_pages=2)
    loop.set_bias(0, bias)
    outs = []
    for who in ([T, 0], [0, T], [T, 0]):
        outs.append(loop.step(i32(who), [x], [gate], [q])[0])
        assert loop.missing() == 0
        loop.release(0 if who[0] else 1)
        assert loop.n_free_tokens.item() == 20 and loop.n_free_entries.item() == 2
        assert sorted(loop.free_tokens.tolist()) == list(range(20))
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    loop.step(i32([T, T]), [torch.cat([x, x])[:T]], [torch.cat([gate, gate])[:T]], [q])
    assert loop.missing() > 0                            # two requests do not fit: reported, not written elsewhere


@pytest.mark.parametrize("d,H", [(128, 8), (512, 64)])
def test_a_captured_step_replays_with_other_lengths(d, H):
    """One captured step (padded to 70 rows) replayed with each step's lengths:
    the bytes of the steps run one by one; rows past the last stay as they were."""
    from long_context_attention_hca_b200.pipeline import PagedLoop
    g = gen(77 + d)
    B, N = 3, 70
    bias = torch.randn((128, d), generator=g, device=DEV) * 0.5

    def make():
        loop = PagedLoop(B, H, LAYOUTS[d], [128, 0], 32, 2, max_tokens=400, max_rows=N, softmax_scale=d ** -0.5,
                         token_page=16, entry_page=1)
        loop.set_bias(0, bias)
        return loop

    x, gate, q = ([torch.zeros(s, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
                  for s in ((N, d), (N, d), (N, H, d)))
    new = torch.zeros((B,), dtype=torch.int32, device=DEV)
    eager, replayed = make(), make()
    torch.cuda.synchronize()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        outs = replayed.step(new, x, gate, q)
    torch.cuda.synchronize()
    for lens in ([70, 0, 0], [0, 60, 10], [57, 9, 1], [1, 1, 1], [0, 0, 0], [3, 66, 1], [1, 0, 1]):
        for t in x + gate + q:
            t.copy_(bf(tuple(t.shape), g))
        new.copy_(i32(lens))
        for o in outs:
            o.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = eager.step(new, x, gate, q)
        n = sum(lens)
        for a, b in zip(want, outs):
            assert torch.equal(a[:n], b[:n]) and bool((b[n:] == 7.0).all())
    assert replayed.ctx.tolist() == eager.ctx.tolist() and replayed.missing() == eager.missing() == 0
    assert torch.equal(replayed.token_table, eager.token_table)
    assert torch.equal(replayed.layers[0].cache.codes, eager.layers[0].cache.codes)


def test_a_negative_length_adds_nothing():
    from long_context_attention_hca_b200.pipeline import PagedLoop
    d, H = 128, 8
    g = gen(3)
    loop = PagedLoop(2, H, LAYOUTS[d], [0], 32, 0, max_tokens=64, max_rows=64, softmax_scale=d ** -0.5, token_page=16)
    for lens, ctx in (([5, 2], [5, 2]), ([-3, 4], [5, 6])):
        n = sum(max(v, 0) for v in lens)
        loop.step(i32(lens), [bf((n, d), g)], [None], [bf((n, H, d), g)])
        assert loop.ctx.tolist() == ctx


# ------------------------------------------------------------------ d = 128, steps of many rows (tiles of 128)
MANY_ROWS = [
    dict(d=128, H=128, ctx=[90, 700, 0], new=[150, 170, 21], W=17, m=4, PE=7, PT=9),
    dict(d=128, H=128, ctx=[500, 1, 60], new=[200, 111, 1], W=100, n_first=64, extras=True),
    dict(d=128, H=100, ctx=[2000, 3], new=[370, 40], W=128, m=128, extras=True, PE=5),
    dict(d=128, H=128, ctx=[0], new=[310], W=1, m=4),
]


@pytest.mark.parametrize("k", range(len(MANY_ROWS)))
def test_many_rows(k):
    c = Case(seed=40 + k, **MANY_ROWS[k])
    out = torch.full_like(c.q, 7.0)
    got = c.run(out=out, max_new=max(c.new))
    assert torch.all(got[c.N:] == 7.0)
    c.check(got, rows=[n for n in range(c.N) if n % 7 == 0 or n in (c.N - 1, 150, 149, 200, 201)])


def test_many_rows_non_finite_keys_and_missing_pages():
    a = dict(d=128, H=128, ctx=[300, 200], new=[290, 30], W=20, m=4, PT=8)
    c, ref = Case(seed=50, **a), Case(seed=50, **a)
    clean = c.run()
    c.etab[0, 2] = -1                                    # entries 32..47 of request 0
    c.ttab[1, :], c.etab[1, :] = -1, c.cache.B           # request 1 sees nothing
    got = c.run()
    keys = ref.keys
    ref.keys = lambda b, p: (np.delete(keys(b, p)[0], np.arange(32, 48)), keys(b, p)[1])
    ref.check(got, rows=[0, 1, 63, 64, 200, 289])
    assert torch.all(got[290:320] == 0)
    c = Case(seed=50, **a)
    c.pages.view(-1, 128)[int(c.ttab[0, 400 // 8]) * 8 + 400 % 8, 3] = float("inf")     # seen at 400 .. 419
    got = c.run()
    for i in range(320):
        if 100 <= i < 120:
            assert torch.isnan(got[i]).all()
        else:
            assert torch.equal(got[i], clean[i])


# ------------------------------------------------------------------ positions up to 2^31
TOP = 1 << 31


@pytest.mark.parametrize("d,H,extras,m", [(512, 64, False, 0), (512, 64, True, 0), (128, 8, True, 0), (128, 8, True, 128),
                                          (512, 64, True, 128)])
def test_attention_at_the_last_positions(d, H, extras, m):
    """Positions right below 2^31: the first column and the last ones of a wide table hold pages, all others none."""
    PT, PE, W, new = 256, 16, 64, 7
    c = Case(d, H, [300], [new], W, m=m, n_first=0 if m else 4, PT=PT, PE=PE, extras=extras, seed=60)
    pages = c.ttab[0].clone()
    c.ttab = torch.full((1, TOP // PT), -1, dtype=torch.int32, device=DEV)
    c.ttab[0, 0] = pages[0]
    c.ttab[0, -2:] = pages[:2]
    c.ctx = [TOP - new - 1]                              # the last query at 2^31 - 2
    if m:
        cols = TOP // m // PE
        c.etab = torch.full((1, cols), -1, dtype=torch.int32, device=DEV)
        c.etab[0, 3] = 0
        c.etab[0, cols - 1] = c.cache.B - 1
        keys = c.keys

        def present(b, p):
            c.m = 0                                      # the tokens alone; entries by hand
            rt = keys(b, p)[1]
            c.m = m
            n_e = (p + 1) // m
            return np.array([i for i in range(PE)] + [(c.cache.B - 1) * PE + i for i in range(PE)
                                                      if (cols - 1) * PE + i < n_e]), rt
        c.keys = present
    c.check(c.run(max_new=new))


def test_plan_and_store_at_the_last_positions():
    d, P, new = 128, 256, 300
    g = gen(8)
    width = TOP // P
    ctx = TOP - 1 - new
    table = torch.full((1, width), -1, dtype=torch.int32, device=DEV)
    table[0, ctx // P] = 2
    plan = hca.kv_page_plan(i32([ctx]), i32([new]), 1, P, table, i32([0, 1]), i32([2]), max_rows=new)
    pos = np.arange(ctx, ctx + new)
    page = np.where(pos // P == ctx // P, 2, 1 - (pos // P - ctx // P - 1))
    assert plan.row_pos.tolist() == pos.tolist() and plan.slot.tolist() == (page * P + pos % P).tolist()
    assert plan.missing.item() == 0 and plan.free_left.item() == 2 - ((ctx + new - 1) // P - ctx // P)
    x = bf((new, d), g)
    fr = inp.rope_inv_freq(32, device=DEV)
    pool = torch.zeros((3, P, d), dtype=torch.bfloat16, device=DEV)
    hca.kv_page_store(x, plan, pool, LAYOUTS[d], extras=hca.EntryExtras(None, 0.0, fr))
    want = oracle.token_prep(host(x), pos, 32, inv_freq=host(fr))
    assert np.array_equal(host(pool).reshape(-1, d)[plan.slot.cpu().numpy()], want)


# ------------------------------------------------------------------ d = 128, steps padded far beyond their live rows
PADDED = [                                               # (case, rows of q, max_new)
    (dict(H=64, ctx=[32766, 9000, 0, 20000, 511, 32766, 100, 16000], new=[1, 1, 1, 1, 0, 1, 1, 1], W=128, m=4, PE=64), 512, 1),
    (dict(H=64, ctx=[32765, 9000, 0, 20000, 511, 32766, 100, 16000], new=[2, 1, 2, 0, 2, 1, 1, 2], W=128, m=4, PE=64), 512, 2),
    (dict(H=64, ctx=[55 * b for b in range(74)], new=[1 + b % 2 for b in range(74)], W=128, m=4, extras=True), 296, 2),
    (dict(H=128, ctx=[3800], new=[200], W=128, m=4), 200, 1),       # (a bound that is too small)
    (dict(H=64, ctx=[5000, 2, 700, 0, 1023, 1024, 40, 3000], new=[2, 2, 1, 2, 0, 1, 2, 1], W=1024, n_first=4, extras=True), 512, 2),
]


@pytest.mark.parametrize("k", range(len(PADDED)))
def test_padded_steps_write_every_live_row(k):
    """Many rows of q, few of them live: every live row is written, whatever tiles and splits are chosen."""
    kw, n, mn = PADDED[k]
    c = Case(128, seed=70 + k, pad=n - sum(kw["new"]), **kw)
    out = torch.full_like(c.q, 7.0)
    got = c.run(out=out, max_new=mn)
    assert torch.all(got[c.N:] == 7.0) and got.shape[0] == n
    c.check(got, rows=[r for r in range(c.N) if r < 40 or r % 9 == 0 or r == c.N - 1])


# ------------------------------------------------------------------ d = 512, many short items of few rows
@pytest.mark.parametrize("H,new", [(5, 1), (64, 1), (7, 9)])
def test_many_items_of_one_key_tile(H, new):
    """Hundreds of items of fewer than 64 rows a CTA and one key tile each, so
    that a pair's next item starts while parts of the last one are still being
    written: the same bytes every time, and every request's rows in its place."""
    r = np.random.default_rng(11)
    ctx = r.integers(0, 60, 700).tolist()
    c = Case(512, H, ctx, [new] * 700, 33, n_first=4, PT=8, extras=True, seed=80)
    want = c.run(max_new=new)
    c.check(want, rows=set(r.integers(0, c.N, 60).tolist()))
    for _ in range(30):
        out = torch.full_like(c.q, 7.0)
        c.run(max_new=new, out=out)
        assert torch.equal(out[:c.N], want[:c.N]) and torch.all(out[c.N:] == 7.0)


# ------------------------------------------------------------------ steps after a shortage of pages
@pytest.mark.parametrize("m", [1, 4])
def test_a_page_still_missing_is_counted_in_every_step_that_needs_it(m):
    """Items whose page an earlier step could not get have no slot, and the plan says so: 0 missing means that every
    row has a slot."""
    P, width = 4, 3
    t = torch.full((4, width), -1, dtype=torch.int32, device=DEV)
    t[3] = i32([0, 1, 2])
    free, ctx = i32([7, 9]), np.array([0, 0, 0, 10])
    #        first items of three pages, one of them without; inside them; inside and on; none; past the table's width
    steps = [([2, 1, 3, 1], [9, 7, -1], 1, 0), ([1, 2, 0, 0], [9, 7, -1], 0, 0), ([0, 0, 1, 0], [9, 7, -1], 1, 0),
             ([1, 1, 1, 1], [9, 7, -1], 1, 0), ([1, 0, 0, 1], [9, 7, -1], 2, 0), ([0, 0, 1, 1], [9, 7, -1], 2, 0)]
    count = i32([2])
    for new, first, missing, left in steps:
        new = np.array(new)
        plan = hca.kv_page_plan(i32(ctx * m), i32(new * m), m, P, t, free, count, max_rows=16)
        assert t[:3, 0].tolist() == first and plan.missing.item() == missing and plan.free_left.item() == left
        n = int(new.sum())
        assert (missing == 0) == bool((plan.slot[:n] >= 0).all())
        count, ctx = plan.free_left, ctx + new


def test_many_requests_with_pages_missing():
    """Every request stands in a page: of 3000, those whose page is gone and that have an item this step are counted."""
    B, P = 3000, 16
    r = np.random.default_rng(2)
    ctx, new = r.integers(1, 64, B), r.integers(0, 3, B)
    ctx[ctx % P == 0] += 1
    table = np.arange(B * 6).reshape(B, 6).astype(np.int32)
    gone = r.random(B) < 0.3
    table[gone, ctx[gone] // P] = -1 - r.integers(0, 5, int(gone.sum()))
    plan = hca.kv_page_plan(i32(ctx), i32(new), 1, P, i32(table), i32(np.arange(B) + B * 6), i32([B]), max_rows=2 * B)
    assert plan.missing.item() == int((gone & (new > 0)).sum()) > 300


def test_a_plan_with_pages_missing_can_be_made_again():
    """Nothing is consumed by a plan: the same lengths again, once pages are free, give every row its slot."""
    t = torch.full((2, 3), -1, dtype=torch.int32, device=DEV)
    free, ctx, new = torch.zeros(8, dtype=torch.int32, device=DEV), i32([0, 0]), i32([6, 3])
    free[0] = 5
    a = hca.kv_page_plan(ctx, new, 1, 4, t, free, i32([1]), max_rows=9)
    assert a.missing.item() == 2 and t.tolist() == [[5, -1, -1], [-1, -1, -1]]
    free[1:3] = i32([2, 3])
    b = hca.kv_page_plan(ctx, new, 1, 4, t, free, i32([3]), max_rows=9)
    assert b.missing.item() == 0 and b.free_left.item() == 0 and t.tolist() == [[3, 2, -1], [5, -1, -1]]
    assert b.slot.tolist() == [12, 13, 14, 15, 8, 9, 20, 21, 22]


def test_the_loop_reports_every_step_that_loses_tokens():
    from long_context_attention_hca_b200.pipeline import PagedLoop
    d, H = 128, 8
    g = gen(5)
    loop = PagedLoop(2, H, LAYOUTS[d], [0], 32, 0, max_tokens=64, max_rows=64, softmax_scale=d ** -0.5, token_page=16,
                     token_pages=1)
    seen = []
    for lens in ([3, 2], [1, 0], [0, 1], [1, 1]):
        n = sum(lens)
        loop.step(i32(lens), [bf((n, d), g)], [None], [bf((n, H, d), g)])
        seen.append(loop.missing())
    assert seen == [1, 1, 2, 3]


# ------------------------------------------------------------------ queries beyond fp16's range
FAR = [(dict(d=512, H=64, ctx=[400, 0, 30], new=[3, 1, 2], W=20, m=4), 6), (dict(d=512, H=5, ctx=[400, 0, 30], new=[30, 1, 2], W=20), 0),
       (dict(d=512, H=64, ctx=[30000, 100], new=[1, 1], W=128, m=4, PE=32), 1),
       (dict(d=128, H=8, ctx=[400, 0, 30], new=[1, 1, 1], W=20, m=4), 1), (dict(d=128, H=64, ctx=[400, 0, 30], new=[3, 1, 2], W=20, m=4), 3),
       (dict(d=128, H=64, ctx=[9000, 100], new=[1, 1], W=128, m=4), 1), (dict(d=128, H=128, ctx=[90, 700], new=[150, 170], W=17, m=4), 0)]


@pytest.mark.parametrize("value", [float("inf"), 1e5, float("nan")])
@pytest.mark.parametrize("sink", [False, True])
@pytest.mark.parametrize("k,wide", [(k, False) for k in range(len(FAR))] + [(0, True), (2, True)])     # (wide: not staged)
def test_a_query_beyond_fp16_is_nan_whatever_its_keys(k, wide, value, sink):
    """Every visible key's product with the far element is negative: no logit is
    finite, and none is +inf.  The row is NaN, not the 0 of a row without keys,
    and the others' bytes do not change; a row that sees no key is 0."""
    kw, mn = FAR[k]
    c = Case(seed=90, **kw)
    if sink:
        c.ex = hca.AttnExtras(None, 1e-6, torch.zeros(c.H, device=DEV), None)
    at = c.d - 1                                         # a dim that entries hold in bf16
    c.pages[..., at] = -c.pages[..., at].abs() - 2.0 ** -14
    if c.cache is not None:
        c.cache.rope[..., -1] = -c.cache.rope[..., -1].abs() - 2.0 ** -14
    if wide:
        t = torch.full((len(c.ctx), (3 << 20) // c.PE), -1, dtype=torch.int32, device=DEV)
        t[:, :c.ew] = c.etab
        c.etab = t
    clean = c.run(max_new=mn)
    hit = torch.zeros((c.N, c.H), dtype=torch.bool, device=DEV)
    for b in range(len(c.ctx)):
        for n in {int(c.starts[b]), int(c.starts[b + 1]) - 1}:
            hit[n, (3 * n + 1) % c.H] = True
    c.q[:c.N, :, at][hit] = value
    got = c.run(max_new=mn)
    assert torch.isnan(got[:c.N][hit]).all()
    assert torch.equal(got[:c.N][~hit], clean[:c.N][~hit])
    c.ttab[:] = -1
    if c.cache is not None:
        c.etab[:] = c.cache.B
    assert torch.all(c.run(max_new=mn)[:c.N] == 0)
    assert hca.take_device_error() == 0
