"""The attention weight that cached slots gather, against its definition in 64 bits.

Tolerance.  A score is off by es = (d/16 + 4) 2^-22 S + 2^-22 (|s| + 8) (test_gpu_kv_attend.py), its
difference to the row's lse by 2^-22 |lse| more; a weight p by twice that, relatively.  The N weights of a slot are
added in fp32, a quarter of a key head's rows in one sequence and the rest in a few steps: (N/16 + 16) 2^-22 of
the sum.  The old weight, where it is read, its product and the final sum are rounded together: 2^-23 of both.
"""
import numpy as np
import pytest
import torch

import _kv
from oracle import kv as o
from sparse_attention_indexer_spin_gb300 import spin

pytestmark = pytest.mark.gpu


def check(dtype, heads, kvh, d, news, before, seed=0, decay=0.75, mutate=None, status_bits=0, max_slots=None,
          max_new=None, scale=None, tail=0, start=None):
    rng = np.random.default_rng(seed)
    R = len(news)
    lens = [a + max(0, b) for a, b in zip(news, before)]
    n_pages = sum(-(-n // 64) for n in lens) + 3
    k, v, ks, vs = _kv.make_pools(rng, n_pages, kvh, d)
    table = _kv.make_table(rng, lens, n_pages)
    start = np.concatenate([[0], np.cumsum(news)]).astype(np.int32) if start is None else np.asarray(start, np.int32)
    T = int(sum(news)) + tail
    before = np.asarray(before, np.int32)
    q = torch.from_numpy(rng.normal(size=(T, heads, d))).to(_kv.TYPES[dtype])
    max_slots, max_new = max_slots or max(max(lens), 1), max(news) if max_new is None else max_new
    table = np.pad(table, ((0, 0), (0, max(0, -(-max_slots // 64) - table.shape[1]))), constant_values=-1)
    cfg = spin.make_kv_config(R, max_slots, 1, heads, kvh, d, dtype, scale)
    # any lse will do: the rows' own where the test is about them, else a spread around ln n
    lse = (np.log(np.maximum(rng.integers(1, 50, (T, heads)), 1)) + rng.normal(size=(T, heads))).astype(np.float32)
    weight = rng.uniform(size=(R, table.shape[1] * 64)).astype(np.float32)
    if mutate:
        mutate(rng, k, ks, table, q, lse, weight)
    dw, status = _kv.dev(weight), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = spin.kv_weigh_workspace(cfg, T, max_new)
    ws.fill_(255)
    args = (cfg, q.cuda(), _kv.dev(lse), _kv.dev(start), max_new, _kv.dev(before), _kv.dev(k), _kv.dev(ks), _kv.dev(table),
            decay)
    spin.kv_weigh(*args, dw, ws, status)
    torch.cuda.synchronize()
    assert int(status.item()) == status_bits
    ref, info = o.weigh(q.double().numpy(), lse.astype(np.float64), start, before, k, ks, table, cfg.softmax_scale,
                        float(np.float32(decay)), weight.astype(np.float64), max_slots, max_new)
    got = dw.double().cpu().numpy()
    N = max_new * heads
    old = np.zeros_like(weight)
    for r, t, n in o.chunk_rows(start, before, max_slots, max_new, T):
        if decay:
            old[r, :before[r]] = np.abs(weight[r, :before[r]])
    with np.errstate(invalid="ignore"):
        tol = 2 * ((d / 16 + 4) * 2.0 ** -22 * info["eS"] + 2.0 ** -22 * (info["es"] + 8 * info["add"])) + \
            (N / 16 + 16) * 2.0 ** -22 * info["add"] + 2.0 ** -23 * (np.abs(ref) + old) + N * 2.0 ** -126
        assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.array_equal(np.isinf(got), np.isinf(ref))
        ok = np.isfinite(ref)
        err = np.abs(got - ref)
    assert (err[ok] <= tol[ok]).all(), float((err[ok] / tol[ok]).max())
    same = np.ones_like(weight, bool)              # what is behind the contexts stays
    for r, t, n in o.chunk_rows(start, before, max_slots, max_new, T):
        same[r, :n] = False
    assert np.array_equal(got[same], weight[same].astype(np.float64))
    dw2 = _kv.dev(weight)                          # the same bits again, whatever the workspace held
    ws.fill_(0x3f)
    spin.kv_weigh(*args, dw2, ws, status)
    assert torch.equal(dw2.view(torch.int32), dw.view(torch.int32))
    return got


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("heads,kvh", [(8, 8), (32, 8), (5, 5), (28, 4), (64, 1), (128, 1), (1, 1), (128, 2)])
def test_head_layouts(dtype, heads, kvh):
    check(dtype, heads, kvh, 128, [1, 5, 0, 33, 2], [0, 200, 64, 0, 319], seed=heads)


@pytest.mark.parametrize("d", [16, 32, 48, 64, 80, 96, 112, 128, 144, 192, 240, 256])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_head_dims(dtype, d):
    check(dtype, 6, 2, d, [30, 65, 7], [100, 0, 130], seed=d)


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300])
def test_lengths(n):
    check("bf16", 4, 2, 128, [n], [0], seed=n)
    check("f32", 2, 2, 64, [n, 1], [n, 64], seed=n)


@pytest.mark.parametrize("before", [0, 1, 15, 16, 63, 64, 65, 127, 128, 1000, 20000])
def test_decoded_tokens(before):
    check("bf16", 16, 2, 128, [1, 1, 1], [before, 7, before // 2], seed=before)


def test_many_requests():
    rng = np.random.default_rng(5)
    news = np.exp(rng.uniform(0, np.log(60), 70)).astype(int)
    news[::9] = 0
    check("bf16", 4, 2, 64, list(news), list(rng.integers(0, 300, 70)), seed=6, max_slots=1000)


@pytest.mark.parametrize("kvh,n", [(2, 50), (2, 100), (3, 33), (3, 70), (5, 17), (8, 40), (8, 64)])
def test_small_parts(kvh, n):
    # parts of the cut that hold nothing but what a key head's codes cost
    for before in (0, 300, 333):
        check("bf16", 8 * kvh, kvh, 64, [n, 1, n // 2], [before, 70, 5], seed=n + before)


def test_rows_of_very_different_sizes():
    # (rows that do not share a power of two, beside row tiles whose rows do, and rows of zeros)
    def mutate(rng, k, ks, table, q, lse, weight):
        q[:40] *= torch.exp2(-torch.randint(0, 60, (40, q.shape[1], 1)).double()).to(q.dtype)
        q[50:60] = 0
        q[70, 1] = 0
    for dtype in ("bf16", "f32", "f16"):
        check(dtype, 8, 2, 128, [200], [300], seed=3, mutate=mutate)


def test_zero_keys_of_a_huge_scale():
    def mutate(rng, k, ks, table, q, lse, weight):
        q *= 2.0 ** 100
        k[:], ks[:] = 0, 2.0 ** 60
    check("bf16", 8, 2, 64, [70, 1], [100, 5], seed=4, mutate=mutate)
    check("bf16", 8, 2, 64, [1, 1], [100, 5], seed=4, mutate=mutate)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("news,before", [([70, 1], [500, 5]), ([200, 40], [300, 64]), ([1, 1], [500, 5]), ([5, 2], [500, 64])])
def test_queries_as_small_as_the_scales_are_large(dtype, news, before):
    # moderate scores, although a score and its page's scale alone are too large for each other's product
    def large(rng, k, ks, table, q, lse, weight):
        q *= 2.0 ** -100
        ks *= np.float32(2.0 ** 101)
    check(dtype, 8, 2, 128, news, before, seed=5, mutate=large)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("news,before", [([200, 40], [300, 64]), ([1, 1], [500, 5]), ([5, 2], [500, 64])])
def test_zero_keys_of_a_huge_scale_beside_others(dtype, news, before):
    # (with rows that do not share a power of two, too)
    def mutate(rng, k, ks, table, q, lse, weight):
        q *= 2.0 ** 100
        q[:2] *= 2.0 ** -30
        ks *= np.float32(2.0 ** -100)
        for r in range(table.shape[0]):
            at = table[r, ::2]
            k[at[at >= 0]], ks[at[at >= 0]] = 0, 2.0 ** 60
    check(dtype, 8, 2, 128, news, before, seed=6, mutate=mutate)


@pytest.mark.parametrize("R", [257, 1100])
def test_very_many_requests(R):
    rng = np.random.default_rng(R)
    before = rng.integers(0, 150, R)
    check("bf16", 2, 1, 64, [1] * R, list(before), seed=R)
    news = np.where(rng.uniform(size=R) < 0.1, rng.integers(0, 60, R), 1)
    check("bf16", 2, 1, 64, list(news), list(before), seed=R, max_new=64)


def test_the_largest_heads():
    check("f32", 128, 2, 256, [3, 20], [65, 300], seed=9)
    check("f32", 128, 128, 256, [1, 2], [65, 30], seed=9)
    check("f32", 128, 128, 256, [40], [65], seed=9)


def test_a_long_chunk():
    check("bf16", 8, 2, 128, [700], [1000], seed=1)


@pytest.mark.parametrize("decay", [0.0, 1.0, -2.0, 0.5])
def test_decay(decay):
    check("bf16", 8, 2, 64, [10, 1], [100, 64], decay=decay)


def test_no_decay_reads_nothing():
    def spoil(rng, k, ks, table, q, lse, weight):
        weight[0, :110] = np.nan
    got = check("bf16", 8, 2, 64, [10], [100], decay=0.0, mutate=spoil)
    assert np.isfinite(got).all()


def test_new_slots_start_from_nothing():
    def spoil(rng, k, ks, table, q, lse, weight):
        weight[0, 100:110] = np.nan
    assert np.isfinite(check("bf16", 8, 2, 64, [10], [100], mutate=spoil)).all()


def test_rows_of_any_lse():
    """-inf: a row that saw nothing; +inf: one that outweighs everything; NaN reaches the slots that it sees."""
    def spoil(rng, k, ks, table, q, lse, weight):
        lse[3, 1], lse[5, 0] = -np.inf, np.inf
    check("bf16", 4, 2, 64, [10], [100], mutate=spoil)

    def nan(rng, k, ks, table, q, lse, weight):
        lse[3, 1] = np.nan
    got = check("bf16", 4, 2, 64, [10], [100], mutate=nan)
    assert np.isnan(got[0, :104]).all() and np.isfinite(got[0, 104:]).all()


def test_slots_that_a_token_does_not_see():
    """NaN keys behind the context, and one inside the chunk: only its own slot becomes NaN."""
    def spoil(rng, k, ks, table, q, lse, weight):
        k[table[0, 1], 46:] = 0x7f
        k[table[0, 1], 40, 1, 3] = 0xff
    got = check("bf16", 4, 2, 64, [10], [100], mutate=spoil)
    assert np.flatnonzero(np.isnan(got[0])).tolist() == [104]


def test_bad_pages_keep_their_weight():
    def spoil(rng, k, ks, table, q, lse, weight):
        table[0, 0], table[0, 2] = k.shape[0], -3
    check("bf16", 4, 2, 64, [100], [100], mutate=spoil, status_bits=spin.STATUS_BITS["BAD_PAGE"])


@pytest.mark.parametrize("kw", [
    dict(before=[0, -1, 5]), dict(before=[0, 1000, 5]), dict(before=[0, 5, 5], max_new=8),
    dict(before=[0, 3, 5], start=[0, 4, 2, 20]), dict(before=[0, 3, 5], start=[-1, 4, 13, 20]),
    dict(before=[0, 3, 5], start=[0, 4, 13, 21])])
def test_refused_requests_keep_their_weight(kw):
    kw = dict(kw)
    check("bf16", 4, 2, 64, [4, 9, 7], kw.pop("before"), status_bits=spin.STATUS_BITS["BAD_N"], max_slots=900, **kw)


def test_no_tokens():
    cfg = spin.make_kv_config(2, 64, 1, 4, 2, 64, "bf16")
    q = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones((2, 64), device="cuda")
    cache = spin.KvCache(2, 2, 64)
    z = torch.zeros(3, dtype=torch.int32, device="cuda")
    for max_new in (0, 5):
        spin.kv_weigh(cfg, q, torch.empty((0, 4), device="cuda"), z, max_new, z[:2].contiguous(), cache.k, cache.k_scale,
                      torch.zeros((2, 1), dtype=torch.int32, device="cuda"), 0.5, w,
                      spin.kv_weigh_workspace(cfg, 0, max_new), None)
        assert (w == 1).all()


def test_all_weight_of_a_chunk_is_shared_out():
    """With the lse of the attention itself, every row's weights sum to 1."""
    rng = np.random.default_rng(3)
    H, kvh, d, n, b = 16, 2, 128, 200, 500
    pools = [_kv.dev(x) for x in _kv.make_pools(rng, 12, kvh, d)]
    table = _kv.dev(rng.permutation(12)[:11].astype(np.int32)[None])
    q = torch.from_numpy(rng.normal(size=(n, H, d))).bfloat16().cuda()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cfg = spin.make_kv_config(1, 704, 1, H, kvh, d, "bf16")
    out, lse, w = torch.empty_like(q), torch.empty((n, H), device="cuda"), torch.zeros((1, 704), device="cuda")
    args = (i32([0, n]), n, i32([b]))
    spin.kv_prefill(cfg, q, *args, *pools, table, out, lse, spin.kv_prefill_workspace(cfg, n, n), None)
    spin.kv_weigh(cfg, q, lse, *args, pools[0], pools[2], table, 1.0, w, spin.kv_weigh_workspace(cfg, n, n), None)
    assert abs(float(w.double().sum()) - n * H) < n * H * 1e-5


def test_other_streams_and_graphs():
    rng = np.random.default_rng(4)
    H, kvh, d, n, b = 16, 2, 128, 3, 500
    k, _, ks, _ = [_kv.dev(x) for x in _kv.make_pools(rng, 12, kvh, d)]
    table = _kv.dev(rng.permutation(12)[:10].astype(np.int32)[None])
    q = torch.from_numpy(rng.normal(size=(n, H, d))).bfloat16().cuda()
    lse = torch.full((n, H), 6.0, device="cuda")
    start, before = _kv.dev(np.array([0, n], np.int32)), _kv.dev(np.array([b], np.int32))
    cfg = spin.make_kv_config(1, 640, 1, H, kvh, d, "bf16")
    ws = [spin.kv_weigh_workspace(cfg, n, n) for _ in range(2)]
    w = [torch.zeros((1, 640), device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    call = lambda y, x, **kw: spin.kv_weigh(cfg, q, lse, start, n, before, k, ks, table, 0.5, y, x, None, **kw)  # noqa: E731
    for _ in range(4):
        call(w[0], ws[0], stream=s)
        call(w[1], ws[1])
    torch.cuda.synchronize()
    assert torch.equal(w[0], w[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(w[2], ws[0])
    for _ in range(4):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(w[0], w[2])
