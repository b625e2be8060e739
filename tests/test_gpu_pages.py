"""Page management against its plain restatement: tables, counts and moved bytes are equal."""
import numpy as np
import pytest
import torch

import _kv
from oracle import kv as o
from sparse_attention_indexer_spin_gb300 import spin

pytestmark = pytest.mark.gpu
B = spin.STATUS_BITS


def state(rng, lens, n_pages, width=None):
    table = _kv.make_table(rng, lens, n_pages, width)
    ref = np.bincount(table[table >= 0], minlength=n_pages).astype(np.int32)
    return table, ref


def make_pools(rng, n_pages, shapes):
    return [rng.integers(0, 256, (n_pages,) + s, dtype=np.uint8) for s in shapes]


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


SHAPES = [(64, 2, 16), (8,), (64, 1, 80), (12,), (4,), (70000,)]   # bytes of a page: aligned or not, small, large


@pytest.mark.parametrize("seed", range(4))
def test_fork_out_of_place(seed):
    rng = np.random.default_rng(seed)
    R = [1, 7, 40, 300][seed]
    lens = rng.integers(0, 1000, R)
    table, ref = state(rng, lens, int(sum(-(-n // 64) for n in lens)) + 5, 16)
    parent = rng.integers(-1, R, R).astype(np.int32)
    out = torch.full((R, 16), 77, dtype=torch.int32, device="cuda")
    dref, st = _kv.dev(ref), status()
    dt = _kv.dev(table)
    spin.pages_fork(dt, _kv.dev(parent), out, dref, st)
    want, wref = o.fork(table, parent, ref)
    assert np.array_equal(out.cpu().numpy(), want) and np.array_equal(dref.cpu().numpy(), wref)
    assert int(st.item()) == 0 and np.array_equal(dt.cpu().numpy(), table)


def test_fork_in_place():
    rng = np.random.default_rng(1)
    table, ref = state(rng, [300, 10, 0, 64, 500, 65], 30, 9)
    parent = np.array([0, 0, 4, -1, 4, 0], np.int32)   # 0 and 4 stay; 1, 5 continue 0; 2 continues 4; 3 leaves
    dt, dref, st = _kv.dev(table), _kv.dev(ref), status()
    spin.pages_fork(dt, _kv.dev(parent), dt, dref, st)
    want, wref = o.fork(table, parent, ref)
    assert np.array_equal(dt.cpu().numpy(), want) and np.array_equal(dref.cpu().numpy(), wref)
    assert int(st.item()) == 0
    # a row may not continue one that changes: it stays, with a report
    parent = np.array([1, 1, 0, 3, 9, 5], np.int32)
    before, bref = dt.cpu().numpy(), dref.cpu().numpy()
    spin.pages_fork(dt, _kv.dev(parent), dt, dref, st)
    ok = np.array([1, 1, 2, 3, 4, 5])
    want, wref = o.fork(before, ok, bref)
    assert np.array_equal(dt.cpu().numpy(), want) and np.array_equal(dref.cpu().numpy(), wref)
    assert int(st.item()) == B["BAD_PARENT"]


def test_fork_bad_parents_and_entries():
    rng = np.random.default_rng(1)
    table, ref = state(rng, [300, 10, 70], 12, 5)
    out, dref, st = torch.zeros((3, 5), dtype=torch.int32, device="cuda"), _kv.dev(ref), status()
    spin.pages_fork(_kv.dev(table), _kv.dev(np.array([0, 3, -2], np.int32)), out, dref, st)
    want, wref = o.fork(table, [0, -1, -1], ref)
    assert np.array_equal(out.cpu().numpy(), want) and np.array_equal(dref.cpu().numpy(), wref)
    assert int(st.item()) == B["BAD_PARENT"]
    broken = table.copy()
    broken[0, 1], broken[2, 0] = 12, -7
    keep = np.where((broken >= 0) & (broken < 12), broken, -1)
    ref = np.bincount(keep[keep >= 0], minlength=12).astype(np.int32)
    out, dref, st = torch.zeros((3, 5), dtype=torch.int32, device="cuda"), _kv.dev(ref), status()
    spin.pages_fork(_kv.dev(broken), _kv.dev(np.array([0, 0, 2], np.int32)), out, dref, st)
    want, wref = o.fork(keep, [0, 0, 2], ref)
    assert np.array_equal(out.cpu().numpy(), want) and np.array_equal(dref.cpu().numpy(), wref)
    assert int(st.item()) == B["BAD_PAGE"]


@pytest.mark.parametrize("seed", range(3))
def test_free(seed):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, 900, 50)
    table, ref = state(rng, lens, int(sum(-(-n // 64) for n in lens)) + 5, 15)
    table, ref = o.fork(table, rng.integers(-1, 50, 50), ref)       # shared pages
    keep = rng.integers(-1, 900, 50).astype(np.int32)
    keep[:4] = [0, 1, 64, 2 ** 31 - 1]
    dt, dref, st = _kv.dev(table), _kv.dev(ref), status()
    spin.pages_free(dt, _kv.dev(keep), dref, st)
    want, wref = o.free(table, keep, ref)
    assert np.array_equal(dt.cpu().numpy(), want) and np.array_equal(dref.cpu().numpy(), wref)
    assert int(st.item()) == 0


def test_free_reports_counts_that_do_not_match():
    rng = np.random.default_rng(0)
    table, ref = state(rng, [100, 30], 6)
    ref[table[0, 0]] = 0
    dt, dref, st = _kv.dev(table), _kv.dev(ref), status()
    spin.pages_free(dt, _kv.dev(np.array([0, 0], np.int32)), dref, st)
    assert (dt.cpu().numpy() == -1).all() and (dref.cpu().numpy() == 0).all()
    assert int(st.item()) == B["BAD_REF"]


def run_reserve(table, ref, n, add, pools):
    dt, dref, st = _kv.dev(table), _kv.dev(ref), status()
    dp = [_kv.dev(p) for p in pools]
    granted = torch.full((len(table),), 9, dtype=torch.int32, device="cuda")
    ws = spin.pages_workspace(len(table), len(ref))
    ws.fill_(255)
    spin.pages_reserve(dt, _kv.dev(np.asarray(n, np.int32)), _kv.dev(np.asarray(add, np.int32)), dref,
                       spin.PagePools(*dp), granted, ws, st)
    torch.cuda.synchronize()
    return (dt.cpu().numpy(), dref.cpu().numpy(), granted.cpu().numpy(), [p.cpu().numpy() for p in dp],
            int(st.item()))


@pytest.mark.parametrize("seed", range(6))
def test_reserve(seed):
    """Shared partial pages are copied, missing ones taken from the lowest free pages, until the
    pool runs out."""
    rng = np.random.default_rng(seed)
    R = [1, 5, 64, 64, 300, 1500][seed]
    lens = rng.integers(0, 500, R)
    n_pages = int(sum(-(-n // 64) for n in lens) + [3, 40, 300, 20, 700, 5000][seed])
    table, ref = state(rng, lens, n_pages, 12)
    parent = np.where(rng.random(R) < 0.5, np.arange(R), rng.integers(-1, R, R))
    table, ref = o.fork(table, parent, ref)
    n = np.where(parent >= 0, lens[parent], 0)
    n = np.maximum(n - rng.integers(0, 90, R) * (rng.random(R) < 0.3), 0)   # some were rolled back
    add = rng.integers(0, 3, R) * rng.integers(1, 100, R)
    pools = make_pools(rng, n_pages, SHAPES[:5] if seed else SHAPES)
    want = o.reserve(table, n, add, ref, pools_w := [p.copy() for p in pools])
    got = run_reserve(table, ref, n, add, pools)
    for x, y in zip(got[:3], want):
        assert np.array_equal(x, y)
    for x, y in zip(got[3], pools_w):
        assert np.array_equal(x, y)
    assert got[4] == (0 if want[2].all() else B["NO_PAGES"])


def test_reserve_edges():
    rng = np.random.default_rng(0)
    table, ref = state(rng, [64, 100, 0], 4, 3)
    pools = make_pools(rng, 4, [(16,)])
    # the last free page goes to the first request that needs one
    t, rf, g, _, st = run_reserve(table, ref, [64, 100, 0], [1, 0, 1], pools)
    want = o.reserve(table, [64, 100, 0], [1, 0, 1], ref, [p.copy() for p in pools])
    assert np.array_equal(t, want[0]) and np.array_equal(rf, want[1]) and list(g) == [1, 1, 0]
    assert st == B["NO_PAGES"]
    # negative and oversized counts are refused, the others served
    t, rf, g, _, st = run_reserve(table, ref, [-1, 100, 0], [1, 200, 1], pools)
    want = o.reserve(table, [0, 0, 0], [0, 0, 1], ref, [p.copy() for p in pools])
    assert np.array_equal(t, want[0]) and np.array_equal(rf, want[1]) and list(g) == [0, 0, 1]
    assert st == B["BAD_N"]
    # a whole row from nothing, exactly to the table's end
    t, rf, g, _, st = run_reserve(np.full((1, 3), -1, np.int32), np.zeros(4, np.int32), [0], [192], pools)
    assert t.tolist() == [[0, 1, 2]] and rf.tolist() == [1, 1, 1, 0] and st == 0


@pytest.mark.parametrize("R,spare", [(1, 5), (40, 9000), (40, 100000), (1100, 20000)])
def test_reserve_long_prompts(R, spare):
    """Prompts of 3 to 700 blocks beside single tokens, some over blocks that are there already,
    alone or shared."""
    rng = np.random.default_rng(R + spare)
    lens = rng.integers(0, 20000, R) * (rng.random(R) < 0.3)
    n_pages = int(sum(-(-n // 64) for n in lens)) + spare
    table, ref = state(rng, lens, n_pages, 1100)
    parent = np.where(rng.random(R) < 0.6, np.arange(R), rng.integers(-1, R, R))
    table, ref = o.fork(table, parent, ref)
    n = np.where(parent >= 0, lens[parent], 0)
    n = n - rng.integers(0, n + 1) * (rng.random(R) < 0.5)                  # rolled back, far or not at all
    add = np.where(rng.random(R) < 0.5, rng.integers(0, 3, R), rng.choice([130, 257, 64 * 33, 64 * 128 + 1, 44800], R))
    if R == 1:
        n, add = np.array([100]), np.array([64 * 300])
    pools = make_pools(rng, n_pages, [(8,)])
    want = o.reserve(table, n, add, ref, pools_w := [p.copy() for p in pools])
    got = run_reserve(table, ref, n, add, pools)
    for x, y in zip(got[:3], want):
        assert np.array_equal(x, y)
    assert np.array_equal(got[3][0], pools_w[0])
    assert got[4] == (0 if want[2].all() else B["NO_PAGES"])


@pytest.mark.parametrize("n_pages,live", [(1, 0), (1, 1), (5, 2), (64, 64), (1000, 300), (1025, 1024), (5000, 1),
                                          (9000, 6000), (40000, 20000)])
def test_compact(n_pages, live):
    rng = np.random.default_rng(n_pages)
    pages = rng.permutation(n_pages)[:live]
    width = max(1, -(-live // 5))
    table = np.full((7, width), -1, np.int32)
    table.reshape(-1)[rng.permutation(5 * width)[:live]] = pages
    table[5] = table[0]                                     # shared pages
    ref = np.bincount(table[table >= 0], minlength=n_pages).astype(np.int32)
    pools = make_pools(rng, n_pages, SHAPES[:5] if n_pages > 100 else SHAPES)
    dt, dref, st = _kv.dev(table), _kv.dev(ref), status()
    dp = [_kv.dev(p) for p in pools]
    n_live = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = spin.pages_workspace(7, n_pages)
    ws.fill_(255)
    spin.pages_compact(dt, dref, spin.PagePools(*dp), n_live, ws, st)
    want = o.compact(table, ref, pools)
    assert int(n_live.item()) == want[2] == live
    assert np.array_equal(dt.cpu().numpy(), want[0]) and np.array_equal(dref.cpu().numpy(), want[1])
    for x, y in zip(dp, pools):
        assert np.array_equal(x.cpu().numpy(), y)
    assert int(st.item()) == 0


def test_compact_reports_bad_entries():
    rng = np.random.default_rng(2)
    pools = make_pools(rng, 8, [(16,)])
    table = np.array([[7, 9, -3], [5, 6, -1]], np.int32)    # 9, -3: no pages; 6: not counted
    ref = np.zeros(8, np.int32)
    ref[[7, 5]] = 1
    dt, dref, st = _kv.dev(table), _kv.dev(ref), status()
    n_live = torch.zeros(1, dtype=torch.int32, device="cuda")
    spin.pages_compact(dt, dref, spin.PagePools(*[_kv.dev(p) for p in pools]), n_live, spin.pages_workspace(2, 8), st)
    assert dt.cpu().numpy().tolist() == [[1, 9, -3], [0, 6, -1]]
    assert dref.cpu().numpy().tolist() == [1, 1, 0, 0, 0, 0, 0, 0] and int(n_live.item()) == 2
    assert int(st.item()) == B["BAD_PAGE"] | B["BAD_REF"]


def test_pools_beyond_32_bit_offsets():
    big = torch.zeros((70000, 65536), dtype=torch.uint8, device="cuda")
    big[69999] = 5
    ref = torch.zeros(70000, dtype=torch.int32, device="cuda")
    ref[69999] = 1
    table = torch.tensor([[69999]], dtype=torch.int32, device="cuda")
    n_live = torch.zeros(1, dtype=torch.int32, device="cuda")
    spin.pages_compact(table, ref, spin.PagePools(big), n_live, spin.pages_workspace(1, 70000), None)
    assert int(table.item()) == 0 and bool((big[0] == 5).all()) and int(big[1].sum()) == 0


def test_graph_replay():
    """fork, reserve, free and compact captured once and replayed on new contents."""
    rng = np.random.default_rng(7)
    R, n_pages = 6, 60
    new = torch.ones(R, dtype=torch.int32, device="cuda")
    dn = torch.zeros(R, dtype=torch.int32, device="cuda")
    t0, t1 = (torch.full((R, 8), -1, dtype=torch.int32, device="cuda") for _ in range(2))
    dref, granted, live, st = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (n_pages, R, 1, 1))
    parent, keep = (torch.zeros(R, dtype=torch.int32, device="cuda") for _ in range(2))
    pool = torch.zeros((n_pages, 64), dtype=torch.uint8, device="cuda")
    pools, ws = spin.PagePools(pool), spin.pages_workspace(R, n_pages)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        spin.pages_fork(t0, parent, t1, dref, st)
        spin.pages_reserve(t1, dn, new, dref, pools, granted, ws, st)
        spin.pages_free(t1, keep, dref, st)
        spin.pages_compact(t1, dref, pools, live, ws, st)
    for _ in range(4):
        lens = rng.integers(0, 400, R)
        table, ref = state(rng, lens, n_pages, 8)
        data = make_pools(rng, n_pages, [(64,)])
        par = rng.integers(0, R, R).astype(np.int32)
        n, kp = lens[par].astype(np.int32), rng.integers(-1, 300, R).astype(np.int32)
        for x, y in ((t0, table), (dref, ref), (pool, data[0]), (parent, par), (dn, n), (keep, kp)):
            x.copy_(torch.from_numpy(y))
        g.replay()
        torch.cuda.synchronize()
        t, rf = o.fork(table, par, ref)
        t, rf, gr = o.reserve(t, n, np.ones(R, int), rf, data)
        t, rf = o.free(t, kp, rf)
        t, rf, nl = o.compact(t, rf, data)
        assert np.array_equal(t1.cpu().numpy(), t) and np.array_equal(dref.cpu().numpy(), rf)
        assert np.array_equal(granted.cpu().numpy(), gr) and int(live.item()) == nl
        assert np.array_equal(pool.cpu().numpy(), data[0])
    assert int(st.item()) == 0


@pytest.mark.parametrize("count", [16, 17, 33, 244])
def test_layer_stacks_of_many_arrays(count):
    """More arrays than one C call takes move together all the same: reserve, then compact, of a stack of
    layers' arrays of several sizes."""
    rng = np.random.default_rng(count)
    R, n_pages = 9, 60
    lens = rng.integers(0, 400, R)
    table, ref = state(rng, lens, n_pages, 8)
    parent = rng.integers(-1, R, R)
    table, ref = o.fork(table, parent, ref)
    n = np.where(parent >= 0, lens[parent], 0)
    add = rng.integers(0, 3, R) * rng.integers(1, 60, R)
    pools = [p for i in range(count) for p in make_pools(rng, n_pages, [SHAPES[i % 5]])]
    want, first = o.reserve(table, n, add, ref, pools_w := [p.copy() for p in pools]), sum(p.size for p in pools)
    dt, dref, st = _kv.dev(table), _kv.dev(ref), status()
    dp = [_kv.dev(p) for p in pools]
    granted, live = torch.zeros(R, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    stack, ws = spin.PagePools(*dp), spin.pages_workspace(R, n_pages)
    assert sum(p.page_bytes for g in stack.groups for p in g) * n_pages == first
    spin.pages_reserve(dt, _kv.dev(n.astype(np.int32)), _kv.dev(add.astype(np.int32)), dref, stack, granted, ws, st)
    assert np.array_equal(dt.cpu().numpy(), want[0]) and np.array_equal(dref.cpu().numpy(), want[1])
    assert (want[0] != table).any()
    for x, y in zip(dp, pools_w):
        assert np.array_equal(x.cpu().numpy(), y)
    # some leave, and the pool is made dense
    t, rf = o.free(want[0], np.where(rng.random(R) < 0.5, 0, -1), want[1])
    dt, dref = _kv.dev(t), _kv.dev(rf)
    spin.pages_compact(dt, dref, stack, live, ws, st)
    t, rf, n_live = o.compact(t, rf, pools_w)
    assert np.array_equal(dt.cpu().numpy(), t) and np.array_equal(dref.cpu().numpy(), rf) and int(live.item()) == n_live
    for x, y in zip(dp, pools_w):
        assert np.array_equal(x.cpu().numpy(), y)
    assert bool(st.item()) == (not want[2].all())


def test_copies_outside_the_pool_are_left_out():
    """A workspace that holds no plan: every copy it seems to ask for is checked."""
    n_pages = 8
    pool = torch.arange(n_pages, dtype=torch.int32, device="cuda")[:, None].repeat(1, 4)
    old, group = pool.clone(), spin.PagePools(pool).groups[0]
    ws = spin.pages_workspace(2, n_pages).view(torch.int32)
    bad, ok = [-2, 8, -2 ** 31, 2 ** 31 - 1], [1, 1, 1, 1]
    for dst, src, want in ((bad, ok, old), (ok, bad, old), (bad, bad, old), ([5, 6], [1, 2], None)):
        for count in (len(dst), -1, 2 ** 31 - 1):
            pool.copy_(old)
            ws.fill_(-1)
            ws[0] = count
            ws[128:128 + len(dst)] = torch.tensor(dst, device="cuda")     # behind the header and the prefix
            ws[192:192 + len(src)] = torch.tensor(src, device="cuda")
            st = status()
            rc = spin.lib().spin_pages_copy(2, n_pages, group, 1, ws.data_ptr(), ws.numel() * 4, st.data_ptr(), None)
            torch.cuda.synchronize()
            assert rc == 0
            moved = old.clone()
            if want is None and count > 0:
                moved[5], moved[6] = old[1], old[2]
            assert torch.equal(pool, moved)
            assert int(st.item()) == (B["BAD_PAGE"] if want is not None and count > 0 else 0)


def test_pools_whose_pages_cannot_be_copied_are_refused_together():
    """Before the first call, wherever in the list they stand."""
    good = [torch.zeros((4, 8), dtype=torch.uint8, device="cuda") for _ in range(20)]
    for bad in (torch.zeros((4, 6), dtype=torch.uint8, device="cuda"), torch.zeros((4, 0), device="cuda"),
                torch.zeros(33, dtype=torch.uint8, device="cuda")[1:].view(4, 8)):
        with pytest.raises(spin.SpinError, match="pool 20"):
            spin.PagePools(*good, bad)
