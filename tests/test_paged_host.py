"""CPU tests of the paged calls' C ABI: workspace sizes and refusals, all
decided on the host before any CUDA call."""
import ctypes

import pytest

from test_abi_host import Cache, Layout, _build_lib

V, I32, I64, F, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
A = 0x10000                          # an aligned address that is never read
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 4
L512, L128 = Layout(512, 64, 64), Layout(128, 32, 32)


class PageMap(ctypes.Structure):
    _fields_ = [("table", V), ("width", I32), ("page_size", I32), ("pages", I64)]


class AttnExtras(ctypes.Structure):
    _fields_ = [("q_norm_w", V), ("norm_eps", F), ("sink", V), ("inv_freq", V), ("q_pos", V), ("win_len", V)]


@pytest.fixture(scope="module")
def lib():
    lb = ctypes.CDLL(_build_lib())
    lb.kv_page_plan.argtypes = [V, V, I32, I32, I32, V, I32, V, V, I32, I64, V, V, V, V, V, V, V]
    lb.kv_page_store.argtypes = [V, I64, V, V, V, Layout, V, V, I64, V]
    lb.kv_page_compress.argtypes = [I32, V, V, I64, V, V, I32, V, V, V, V, V, I64, V, V, Layout, Cache, I64, V, V]
    lb.paged_attn_workspace_size.argtypes = [I64, I32, I32, Layout, I64, I64, I32, I32]
    lb.paged_attn_workspace_size.restype = SZ
    lb.paged_attn_chunk.argtypes = [V, I64, I32, I32, V, V, I64, I32, Layout, Cache, PageMap, V, PageMap, I32, F, V, V, V,
                                    SZ, V]
    lb.paged_attn_window.argtypes = [V, I64, I32, I32, V, V, I64, Layout, V, PageMap, I32, I32, F, V, V, V, SZ, V]
    return lb


def plan(lib, **kw):
    a = dict(ctx=A, new=A, B=4, m=1, P=16, table=A, width=8, free=A, count=A, cap=4, rows=10, start=A, req=A, pos=A,
             slot=A, missing=A, left=A + 16)
    a.update(kw)
    return lib.kv_page_plan(*a.values(), None)


@pytest.mark.parametrize("bad", [dict(B=-1), dict(m=0), dict(P=0), dict(width=-1), dict(pos=A + 1), dict(cap=-1), dict(rows=-1),
                                 dict(ctx=None), dict(new=A + 2), dict(table=None), dict(free=None), dict(count=None),
                                 dict(start=None), dict(req=None), dict(slot=A + 4), dict(missing=None), dict(left=None),
                                 dict(left=A)])
def test_plan_refusals(lib, bad):
    assert plan(lib, **bad) == INVALID


def test_plan_limit(lib):
    assert plan(lib, B=16385) == UNSUPPORTED


def store(lib, **kw):
    a = dict(x=A, n=3, live=A + 4, pos=A, slot=A, layout=L512, ex=None, pages=A, n_slots=10)
    a.update(kw)
    return lib.kv_page_store(*a.values(), None)


def test_store_refusals(lib):
    for bad in (dict(n=-1), dict(n_slots=-1), dict(x=None), dict(live=None), dict(live=A + 2), dict(pos=None),
                dict(slot=A + 4), dict(pages=A + 2)):
        assert store(lib, **bad) == INVALID, bad
    assert store(lib, layout=Layout(256, 64, 64)) == UNSUPPORTED
    assert store(lib, n=0, x=None) == OK and store(lib, n_slots=0, pages=None) == OK


def compress(lib, **kw):
    a = dict(m=128, x=A, gate=A, n=3, start=A, ctx=A, B=2, bias=A, es=A, er=A, ep=A, eslot=A, me=4, tx=A, tg=A, layout=L512,
             pool=Cache(A, A, A, 16), n_slots=64, ex=None)
    a.update(kw)
    return lib.kv_page_compress(*a.values(), None)


def test_compress_refusals(lib):
    for bad in (dict(n=-1), dict(B=-1), dict(me=-1), dict(n_slots=-1), dict(x=None), dict(gate=A + 2), dict(start=None),
                dict(ctx=None), dict(bias=None), dict(es=None), dict(er=None), dict(eslot=None), dict(tx=None), dict(tg=None),
                dict(pool=Cache(None, A, A, 16))):
        assert compress(lib, **bad) == INVALID, bad
    assert compress(lib, m=8) == UNSUPPORTED and compress(lib, layout=Layout(512, 32, 64)) == UNSUPPORTED
    assert compress(lib, n=0, x=None) == OK and compress(lib, B=0, ctx=None) == OK


def chunk(lib, **kw):
    a = dict(q=A, n=5, H=64, B=2, start=A, ctx=A, max_new=0, m=128, layout=L512, pool=Cache(A, A, A, 16),
             em=PageMap(A, 4, 16, 8), pages=A, tm=PageMap(A, 4, 16, 8), W=128, scale=0.05, ex=None, out=A, ws=None, wb=0)
    a.update(kw)
    return lib.paged_attn_chunk(*a.values(), None)


def test_attention_refusals(lib):
    for bad in (dict(n=-1), dict(B=-1), dict(max_new=-1), dict(q=None), dict(out=A + 8), dict(start=None), dict(ctx=None),
                dict(m=0), dict(pool=Cache(None, A, A, 16)), dict(em=PageMap(None, 4, 16, 8)), dict(em=PageMap(A, 4, 0, 8)),
                dict(em=PageMap(A, -1, 16, 8)), dict(tm=PageMap(A, 4, 16, -8)), dict(tm=PageMap(A + 2, 4, 16, 8)),
                dict(pages=None), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan")),
                dict(em=PageMap(A, 1 << 20, 1 << 20, 8)), dict(ws=A + 4)):
        assert chunk(lib, **bad) == INVALID, bad
    for bad in (dict(H=0), dict(H=129), dict(W=0), dict(W=4097), dict(layout=Layout(256, 64, 64)), dict(n=1 << 27)):
        assert chunk(lib, **bad) == UNSUPPORTED, bad
    for name in ("q_pos", "win_len"):
        ex = AttnExtras(norm_eps=1e-6, **{name: A})
        assert chunk(lib, ex=ctypes.addressof(ex)) == INVALID
    ex = AttnExtras(norm_eps=-1.0)
    assert chunk(lib, ex=ctypes.addressof(ex)) == INVALID
    assert chunk(lib, n=0, q=None) == OK and chunk(lib, B=0, start=None) == OK

    def window(**kw):
        a = dict(q=A, n=5, H=8, B=2, start=A, ctx=A, max_new=0, layout=L128, pages=A, tm=PageMap(A, 4, 16, 8), W=8, first=4,
                 scale=0.1, ex=None, out=A, ws=None, wb=0)
        a.update(kw)
        return lib.paged_attn_window(*a.values(), None)
    assert window(first=-1) == UNSUPPORTED and window(first=4097) == UNSUPPORTED and window(pages=A + 8) == INVALID
    assert window(n=0) == OK


def test_workspace_sizes(lib):
    size = lib.paged_attn_workspace_size
    # one decode request over many entries is split; a missing or small workspace is refused before any launch
    need = size(1, 1, 64, L512, 1, 4 * 4096, 128, 0)
    assert need > 0
    long = dict(n=1, B=1, max_new=1, em=PageMap(A, 4, 4096, 8))
    assert chunk(lib, **long) == WORKSPACE
    assert chunk(lib, ws=A, wb=need - 1, **long) == WORKSPACE
    assert size(0, 1, 64, L512, 0, 0, 128, 0) == 0
    assert size(5, 1, 0, L512, 0, 0, 128, 0) == 0 and size(5, 1, 64, Layout(1, 1, 1), 0, 0, 128, 0) == 0


def test_every_split_has_rows_of_a_joined_tile(lib):
    """d = 128: tiles of 128 rows are never split (nothing joins their splits).
    Without staged keys the workspace is tiles x splits x rows x (128 fp16 + 2
    fp32) and 256 bytes, so that its size tells the tile: nothing, or a whole
    number of splits of 16- or 64-row tiles.  The first four: steps padded far
    beyond their live rows, and a bound that is too small."""
    size = lib.paged_attn_workspace_size
    steps = [(512, 8, 64, 1, 8192, 128, 0), (296, 74, 64, 2, 1024, 128, 0), (200, 1, 128, 1, 1024, 128, 0),
             (512, 8, 64, 2, 0, 1024, 4)]
    steps += [(n, B, H, mn, e, W, 0) for n in (1, 33, 200, 296, 512, 1000, 4096) for B in (1, 8, 74, 200) for H in (1, 8, 64, 128)
              for mn in (0, 1, 2, 7, 64) for e in (0, 1024, 65536) for W in (1, 128, 1024)]
    split = 0
    for n, B, H, mn, e, W, first in steps:
        got = size(n, B, H, L128, mn, e, W, first)
        if got == 0:
            continue
        split += 1
        one = [(n * H // R + B) * R * (128 * 2 + 8) for R in (16, 64)]
        assert any((got - 256) % o == 0 and 2 <= (got - 256) // o <= 64 for o in one), (n, B, H, mn, e, W, first)
    assert split > 100


def test_a_plan_without_row_starts_is_refused():
    """row_start holds B + 1 offsets, one at least: with none, the count of live
    rows would be read in front of it."""
    import torch

    hca = pytest.importorskip("long_context_attention_hca_b200")
    cpu = torch.device("cpu")
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)
    rows = (i32(3), i32(3), torch.zeros(3, dtype=torch.int64))
    hca.PagePlan(i32(1), *rows).check(cpu)
    hca.PagePlan(i32(5), *rows).check(cpu, 4)
    for starts, B in ((i32(0), None), (i32(0), 0), (i32(4), 4), (i32(0).long(), None)):
        with pytest.raises((ValueError, TypeError)):
            hca.PagePlan(starts, *rows).check(cpu, B)


def test_a_plan_to_be_made_needs_its_totals():
    """What a PagePlan lacks is named before anything runs."""
    import torch

    hca = pytest.importorskip("long_context_attention_hca_b200")
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)
    plan = hca.PagePlan(i32(3), i32(3), i32(3), torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="missing"):
        plan.check(torch.device("cpu"), 2, totals=True)
    plan.check(torch.device("cpu"), 2)
    with pytest.raises(TypeError, match="free_left"):
        hca.PagePlan(plan.row_start, plan.row_req, plan.row_pos, plan.slot, i32(1), i32(1).long()).check(
            torch.device("cpu"), 2, totals=True)


def test_the_loop_refuses_before_anything_is_launched():
    """A step's arguments are all looked at before its first call."""
    import torch

    pytest.importorskip("long_context_attention_hca_b200")
    from long_context_attention_hca_b200.pipeline import PagedLoop
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)
    loop = PagedLoop(2, 8, (128, 32, 32), [0, 128], 16, 0, max_tokens=64, max_rows=8, softmax_scale=0.1, token_page=16,
                     device="cpu")
    x = torch.zeros((2, 128), dtype=torch.bfloat16)
    q = torch.zeros((2, 8, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="set_bias"):
        loop.step(i32(2), [x, x], [None, x], [q, q])
    loop.set_bias(1, torch.zeros((128, 128)))
    with pytest.raises(ValueError, match="gate_new"):
        loop.step(i32(2), [x, x], [None, None], [q, q])
    for bad in (dict(x_new=[x]), dict(q=[q]), dict(gate_new=[None]), dict(gate_new=None)):
        with pytest.raises(ValueError, match="layer"):
            loop.step(**{**dict(new_len=i32(2), x_new=[x, x], gate_new=[None, x], q=[q, q]), **bad})
    for bad in (dict(new_len=i32(3)), dict(x_new=[x, x.float()]), dict(x_new=[x, x[:, :64]]), dict(gate_new=[None, x[:1]]),
                dict(q=[q, q[:, :4]]), dict(max_new=-1), dict(x_new=[torch.zeros((9, 128), dtype=torch.bfloat16), x])):
        with pytest.raises((ValueError, TypeError)):
            loop.step(**{**dict(new_len=i32(2), x_new=[x, x], gate_new=[None, x], q=[q, q]), **bad})
    assert loop.ctx.tolist() == [0, 0] and loop.token_table.eq(-1).all()
    # gates are asked for HCA layers only
    first = PagedLoop(2, 8, (128, 32, 32), [128, 0], 16, 0, max_tokens=64, max_rows=8, softmax_scale=0.1, device="cpu")
    first.set_bias(0, torch.zeros((128, 128)))
    first._check(i32(2), [x, x], [x], [q, q], None)
    window = PagedLoop(2, 8, (128, 32, 32), [0], 16, 0, max_tokens=64, max_rows=8, softmax_scale=0.1, device="cpu")
    for gates in (None, [], [None]):
        window._check(i32(2), [x], gates, [q], 1)
