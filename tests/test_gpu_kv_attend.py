"""Attention over the paged 8-bit KV cache against its definition in 64 bits.

Tolerances.  With w the softmax weights, A = sum w |v| and S = max softmax_scale ks sum |q||k|:
  * a score is a fp32 dot product of d exact products, accumulated 16 at a time (each step off
    by at most 2^-22 of the magnitude bound), then scaled and turned into an exponent with a few
    fp32 roundings: |ds| <= es = (d/16 + 4) 2^-22 S + 2^-22 (|s| + 8), where the 8 also covers
    the exponential's relative error;
  * it moves a weight and the weights' sum by e^es each: 2 es A;
  * a weight enters its product rounded to f16 (bf16 and f16: 2^-11) or to two f16 terms (f32:
    2^-22, doubled here): ew A, with weights far below the largest (2^-14 after its scaling by at
    least 2^10) off by at most 2^-37 of the largest weight times value scale times 448;
  * the weights' sum and the product's sum are accumulated in fp32: el = (n/16 + 8) 2^-22 each;
  * the result is rounded once: half a step of the output's type.
lse = ln of the sum: es + el, and fp32 roundings of its own, relative 2^-22.
"""
import numpy as np
import pytest
import torch

import _kv
from oracle import kv as o
from sparse_attention_indexer_spin_gb300 import spin

pytestmark = pytest.mark.gpu


def check(dtype, heads, kvh, d, lens, rows=1, top_k=0, seed=0, spread=0.3, scale=None, n_slots=None, listed=None,
          mutate=None, status_bits=0, q_size=1.0, max_slots=None):
    """One call against the oracle; `lens` are the requests' cached slots."""
    rng = np.random.default_rng(seed)
    R = len(lens)
    n_pages = sum(-(-int(n) // 64) for n in lens) + 3
    pools = list(_kv.make_pools(rng, n_pages, kvh, d, spread))
    table = _kv.make_table(rng, lens, n_pages)
    if n_slots is None:                # row r of a verification sees one slot more than row r - 1
        n_slots = np.maximum(np.asarray(lens)[:, None] - np.arange(rows - 1, -1, -1), 0)
    n_slots = np.ascontiguousarray(n_slots, dtype=np.int32)
    q = torch.from_numpy(rng.normal(size=(R, rows, heads, d)) * q_size).to(_kv.TYPES[dtype])
    if top_k and listed is None:
        listed = np.full((R, rows, top_k), -1, np.int32)
        for b in range(R):
            for r in range(rows):
                m = min(top_k, int(n_slots[b, r]))
                listed[b, r, :m] = np.sort(rng.permutation(int(n_slots[b, r]))[:m])
    if mutate:
        mutate(rng, pools, table, n_slots, listed)
    if max_slots:
        table = np.pad(table, ((0, 0), (0, -(-max_slots // 64) - table.shape[1])), constant_values=-1)
    cfg = spin.make_kv_config(R, max_slots or max(max(lens), 1), rows, heads, kvh, d, dtype, scale)
    dv = [_kv.dev(x) for x in pools]
    before = [x.clone() for x in dv]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dl = None if listed is None else _kv.dev(listed)
    out, lse = _kv.run_attend(cfg, q.cuda(), dv, _kv.dev(table), _kv.dev(n_slots), rows, dl, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == status_bits
    for x, y in zip(dv, before):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))   # the cache is only read
    good = np.where((n_slots < 0) | (n_slots > cfg.max_slots), 0, n_slots)
    ref, rlse, info = o.attend(q.double().numpy(), *pools, table, good, cfg.softmax_scale, listed)
    tol, ltol = _kv.attend_tolerance(dtype, d, ref, info)
    got, glse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    nan = np.isnan(ref)
    assert np.array_equal(np.isnan(got), nan)
    err = np.abs(got - ref)
    assert (err[~nan] <= tol[~nan]).all(), float((err[~nan] / tol[~nan]).max())
    empty = np.isneginf(rlse)
    assert np.array_equal(np.isneginf(glse), empty)
    assert (got[empty] == 0).all()
    ok = ~empty & ~np.isnan(rlse)
    assert (np.abs(glse[ok] - rlse[ok]) <= ltol[ok] + 2.0 ** -22 * (np.abs(rlse[ok]) + 1)).all()
    # without lse the output is the same
    out2, _ = _kv.run_attend(cfg, q.cuda(), dv, _kv.dev(table), _kv.dev(n_slots), rows, dl, want_lse=False)
    assert torch.equal(out.view(torch.uint8), out2.view(torch.uint8))
    return out, lse


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("heads,kvh", [(8, 8), (32, 8), (5, 5), (28, 4), (64, 1), (128, 1), (1, 1)])
def test_head_layouts(dtype, heads, kvh):
    check(dtype, heads, kvh, 128, [1, 200, 0, 64, 321], seed=heads)


@pytest.mark.parametrize("d", [16, 32, 48, 64, 80, 96, 112, 128, 144, 192, 240, 256])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_head_dims(dtype, d):
    check(dtype, 6, 2, d, [130, 65, 7], seed=d)
    check(dtype, 6, 2, d, [130, 65, 7], seed=d, rows=2, top_k=33)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 511, 1000, 5000])
def test_lengths(n):
    check("bf16", 16, 2, 128, [n], seed=n)
    check("f32", 8, 8, 64, [n, 1], seed=n)


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 8])
@pytest.mark.parametrize("heads,kvh", [(8, 8), (16, 2), (64, 1), (128, 2)])
def test_rows(rows, heads, kvh):
    """Verifier rows that see one slot more each, across a page's end and from no slots on."""
    check("bf16", heads, kvh, 128, [rows + 63, 66, 2, 0, 700], rows=rows, seed=rows)
    check("f16", heads, kvh, 64, [rows + 63, 66, 2, 0, 700], rows=rows, seed=rows)


@pytest.mark.parametrize("top_k", [1, 7, 64, 100, 256, 512, 2048])
@pytest.mark.parametrize("heads,kvh,rows", [(64, 1, 1), (8, 8, 3), (32, 8, 1), (12, 1, 2)])
def test_lists(top_k, heads, kvh, rows):
    check("bf16", heads, kvh, 128, [3000, 50, 0, 1, 777], rows=rows, top_k=top_k, seed=top_k)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_many_requests_of_mixed_length(dtype):
    rng = np.random.default_rng(5)
    lens = np.exp(rng.uniform(0, np.log(3000), 70)).astype(int)
    lens[::9] = 0
    check(dtype, 8, 2, 64, list(lens), seed=6)


@pytest.mark.parametrize("lens", [[1], [70], [2000, 100, 0, 7], [0, 0, 0], [64] * 9, [130, 0, 0, 0, 4000]])
def test_short_requests_under_a_large_capacity(lens):
    """The launch is sized by max_slots: most of its CTAs find no work."""
    check("bf16", 16, 2, 128, lens, max_slots=100000, seed=len(lens))
    check("f32", 4, 4, 64, lens, max_slots=100000, top_k=900, seed=len(lens))
    check("bf16", 64, 1, 128, lens, max_slots=100000, rows=3, seed=len(lens))


def test_long_context():
    check("bf16", 16, 2, 128, [40000, 3], seed=1)
    check("f32", 2, 1, 64, [40000], seed=1)


@pytest.mark.parametrize("scale", [0.0, 1.0, -0.5, 3.0])
def test_softmax_scale(scale):
    """Flat, sharp and inverted weights."""
    check("bf16", 8, 2, 128, [300, 40], scale=scale, seed=3)
    check("f32", 8, 2, 64, [300, 40], scale=scale, seed=3)


@pytest.mark.parametrize("spread", [0.0, 3.0, 6.0])
def test_scales_of_very_different_pages(spread):
    """Value scales e^+-18 apart: the small pages' products must not be lost beside the large
    ones' scale."""
    check("bf16", 8, 2, 128, [700, 64], spread=spread, seed=4, scale=1e-3)
    check("f32", 8, 2, 128, [700, 64], spread=spread, seed=4, scale=1e-3)


@pytest.mark.parametrize("dtype,size", [("bf16", 1e-30), ("bf16", 1e25), ("f32", 1e-25), ("f32", 1e20), ("f16", 1e-4)])
def test_queries_of_extreme_size(dtype, size):
    check(dtype, 8, 2, 64, [100, 30], q_size=size, scale=0.1 / size if dtype != "f16" else 30.0, seed=8)


def _zero_pages(rng, pools, table, n_slots, listed):
    for x in pools[2:]:
        x[rng.permutation(len(x))[: len(x) // 2]] = 0.0


def test_pages_of_scale_zero():
    check("bf16", 8, 2, 128, [700, 64, 10], mutate=_zero_pages, seed=2)
    check("f32", 8, 2, 64, [700, 64, 10], top_k=50, mutate=_zero_pages, seed=2)


def test_all_values_zero():
    def zero(rng, pools, table, n_slots, listed):
        pools[3][:] = 0.0
    check("bf16", 8, 2, 128, [700, 64, 10], mutate=zero, seed=2)


def _nan_behind(rng, pools, table, n_slots, listed):
    """NaN codes, and NaN and infinite scales, everywhere no row looks."""
    k, v, ks, vs = pools
    seen = np.zeros((len(k), 64), bool)
    used = np.zeros(len(k), bool)
    for b in range(len(table)):
        for r in range(n_slots.shape[1]):
            i = np.arange(n_slots[b, r]) if listed is None else listed[b, r][listed[b, r] >= 0]
            seen[table[b, i // 64], i % 64] = True
            used[table[b, i // 64]] = True
    k[~seen] = 0x7f
    v[~seen] = 0xff
    ks[~used], vs[~used] = np.nan, np.inf


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,top_k", [(1, 0), (3, 0), (1, 40), (2, 40)])
def test_nan_outside_the_set(dtype, rows, top_k):
    check(dtype, 8, 2, 128, [700, 64, 10, 0, 65], rows=rows, top_k=top_k, mutate=_nan_behind, seed=9)


@pytest.mark.parametrize("heads,kvh,rows", [(8, 2, 4), (64, 1, 4), (16, 2, 2)])
def test_nan_that_only_later_rows_see(heads, kvh, rows):
    """A NaN key or value in a slot that the last rows see and the first do not: only the rows
    that see it turn NaN (a NaN value only its dimension)."""
    for which in (0, 1):
        def one(rng, pools, table, n_slots, listed):
            i = int(n_slots[0, -1]) - 1
            pools[which][table[0, i // 64], i % 64, 0, 5] = 0x7f
        check("bf16", heads, kvh, 128, [130, 64], rows=rows, mutate=one, seed=1)


def test_nan_inside_the_set():
    for which in (0, 1):
        def one(rng, pools, table, n_slots, listed):
            pools[which][table[0, 0], 3, 1, 7] = 0xff
        check("bf16", 8, 2, 128, [130, 64], mutate=one, seed=1)
        check("f32", 8, 2, 64, [130, 64], mutate=one, seed=1)


def test_unordered_and_repeated_list_entries():
    rng = np.random.default_rng(0)
    listed = rng.integers(-1, 500, (2, 2, 300)).astype(np.int32)
    listed[0, 1] = 17                  # one slot 300 times
    listed[1, 0] = -1                  # nothing
    check("bf16", 16, 2, 128, [500, 500], rows=2, n_slots=np.full((2, 2), 500), listed=listed, top_k=300)


def test_bad_lengths_pages_and_entries_are_reported_and_left_out():
    check("bf16", 8, 2, 64, [100, 70, 30], n_slots=[[101], [-1], [30]], status_bits=spin.STATUS_BITS["BAD_N"])

    def lost_pages(rng, pools, table, n_slots, listed):
        table[0, 0], table[1, 1] = -1, 1000
    for top_k in (0, 90):
        check("bf16", 8, 2, 64, [100, 70, 30], mutate=lost_pages, top_k=top_k,
              status_bits=spin.STATUS_BITS["BAD_PAGE"])
    listed = np.tile(np.array([0, 5, 100, -2, 2 ** 30, -2 ** 31], np.int32), (2, 1, 1))
    check("bf16", 8, 2, 64, [100, 70], listed=listed, top_k=6, status_bits=spin.STATUS_BITS["BAD_LIST"])


def test_pool_beyond_32_bit_offsets():
    """Pages whose byte offset passes 2^32."""
    n_pages, kvh, d = 70000, 8, 128
    k, v = (torch.zeros((n_pages, 64, kvh, d), dtype=torch.uint8, device="cuda") for _ in range(2))
    rng = np.random.default_rng(0)
    pages = np.array([[69999, 3, 66001, 68000, 69998]], np.int32)
    small = _kv.make_pools(rng, 5, kvh, d)
    for i, p in enumerate(pages[0]):
        k[int(p)], v[int(p)] = _kv.dev(small[0][i]), _kv.dev(small[1][i])
    ks, vs = (torch.zeros((n_pages, kvh), device="cuda") for _ in range(2))
    ks[pages[0].tolist()], vs[pages[0].tolist()] = _kv.dev(small[2]), _kv.dev(small[3])
    q = torch.from_numpy(rng.normal(size=(1, 1, 16, d))).to(torch.bfloat16)
    cfg = spin.make_kv_config(1, 320, 1, 16, kvh, d, "bf16")
    n = np.array([[300]], np.int32)
    out, _ = _kv.run_attend(cfg, q.cuda(), (k, v, ks, vs), _kv.dev(pages), _kv.dev(n), 1)
    ref, _, info = o.attend(q.double().numpy(), *small, np.arange(5)[None], n, cfg.softmax_scale)
    tol, _ = _kv.attend_tolerance("bf16", d, ref, info)
    assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()


def test_streams_graphs_and_guard_bands():
    """The same bits on a side stream, in a replayed graph and from run to run; nothing written
    around the outputs."""
    rng = np.random.default_rng(3)
    lens = [2000, 100, 0, 7]
    pools = _kv.make_pools(rng, 40, 2, 128)
    table = _kv.make_table(rng, lens, 40)
    cfg = spin.make_kv_config(4, 2000, 1, 16, 2, 128, "bf16")
    dv, dt, dn = [_kv.dev(x) for x in pools], _kv.dev(table), _kv.dev(np.array(lens, np.int32)[:, None])
    q = torch.from_numpy(rng.normal(size=(4, 1, 16, 128))).to(torch.bfloat16).cuda()
    want, wlse = _kv.run_attend(cfg, q, dv, dt, dn, 1)
    for _ in range(3):
        out, lse = _kv.run_attend(cfg, q, dv, dt, dn, 1)
        assert torch.equal(out, want) and torch.equal(lse, wlse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out, lse = _kv.run_attend(cfg, q, dv, dt, dn, 1)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wlse)
    band = torch.full((q.numel() + 256,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = band[128:-128].view(q.shape)
    ws = spin.kv_workspace(cfg)
    g = torch.cuda.CUDAGraph()
    lse = torch.zeros((4, 1, 16), device="cuda")
    with torch.cuda.graph(g):
        spin.kv_attend(cfg, q, *dv, dt, dn, 1, None, out, lse, ws, None)
    for fill in (0, 255):
        ws.fill_(fill)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wlse)
    assert (band[:128] == 7).all() and (band[-128:] == 7).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("heads,kvh,rows,d", [(64, 1, 1, 128), (40, 2, 1, 80), (128, 2, 8, 64), (16, 2, 4, 128)])
def test_many_query_rows_of_a_key_head_under_a_large_capacity(dtype, heads, kvh, rows, d):
    """More than 16 query rows a key head, in jobs that are divided and in ones that are whole."""
    check(dtype, heads, kvh, d, [rows + 63, 66, 2, 0, 700], rows=rows, max_slots=30000, seed=rows)
    check(dtype, heads, kvh, d, [rows + 63, 66, 2, 0, 700], rows=rows, seed=rows)
    check(dtype, heads, kvh, d, [1500, 66, 2, 0, 700], rows=rows, top_k=1100, seed=rows)
    if dtype != "f32":                 # more whole jobs than fit at once
        check(dtype, heads, kvh, d, [70, 3, 0, 129] * 130, rows=rows, seed=rows)

    def nan(rng, pools, table, n_slots, listed):
        i = int(n_slots[0, -1]) - 1
        pools[1][table[0, i // 64], i % 64, 0, 5] = 0x7f
        _nan_behind(rng, pools, table, n_slots, listed)
    check(dtype, heads, kvh, d, [700, 64, 10, 0, 65], rows=rows, max_slots=30000, mutate=nan, seed=1)


@pytest.mark.parametrize("heads,kvh,d,max_slots", [(8, 2, 128, None), (8, 2, 64, 60000), (64, 1, 128, 60000), (8, 8, 256, 60000)])
def test_rows_of_very_different_lengths_and_nan_values(heads, kvh, d, max_slots):
    """Empty rows of a padded batch, short and long rows of one request, NaN values among the slots
    that only some of them see."""
    lens = [3000, 130, 4000]
    n_slots = np.array([[3000, 0, 100, 1500], [0, 0, 129, 64], [0, 4000, 0, 1]])

    def nan(rng, pools, table, n_slots, listed):
        for b, i, dim in ((0, 90, 3), (0, 120, 4), (0, 1499, 5), (0, 2999, 6), (1, 100, 7), (2, 1, 8), (2, 2500, 9)):
            pools[1][table[b, i // 64], i % 64, 0, dim] = 0x7f
    for dtype in ("bf16", "f32"):
        check(dtype, heads, kvh, d, lens, rows=4, n_slots=n_slots, max_slots=max_slots, mutate=nan, seed=2)
        check(dtype, heads, kvh, d, lens, rows=4, n_slots=n_slots, max_slots=max_slots, seed=3)


def _whole_requests(kvh):
    """Requests of kvh key heads whose whole jobs fill the GPU once, at three CTAs an SM."""
    return 3 * torch.cuda.get_device_properties(0).multi_processor_count // kvh


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vs", [0.0, 2.0 ** -99, 2.0 ** 99])
@pytest.mark.parametrize("divided", [True, False])
def test_sums_of_long_rows_at_the_ends_of_the_value_scales(dtype, vs, divided):
    """131072 slots of equal scores, whose weights' sum stays finite: lse = ln n and out is the values'
    mean.  Every term and partial sum is a power of two times a whole number below 2^24, so that sums
    are exact: out is off by the weight's rounding, 1/l and two products; the logarithm's parts are at
    most 2^7 in magnitude, so each of its roundings is at most 2^-18."""
    n, kvh, d = 131072, 8, 64
    R = 1 if divided else _whole_requests(kvh)
    k, v = (torch.full((4, 64, kvh, d), 0x38, dtype=torch.uint8, device="cuda") for _ in range(2))   # 1.0
    ks, vsc = torch.ones((4, kvh), device="cuda"), torch.full((4, kvh), vs, device="cuda")
    table = (torch.arange(n // 64, dtype=torch.int32, device="cuda") % 4).expand(R, -1).contiguous()
    cfg = spin.make_kv_config(R, n, 1, kvh, kvh, d, dtype, 0.0)
    q = torch.randn((R, 1, kvh, d), device="cuda").to(_kv.TYPES[dtype])
    ns = torch.full((R, 1), n, dtype=torch.int32, device="cuda")
    out, lse = _kv.run_attend(cfg, q, (k, v, ks, vsc), table, ns, 1)
    assert float((lse.double() - np.log(n)).abs().max()) <= 2.0 ** -16
    rel = (2.0 ** -21 if dtype == "f32" else 2.0 ** -11) + 2.0 ** -21 + _kv.HALF_STEP[dtype]
    assert bool(((out.double() - vs).abs() <= rel * vs).all())


def test_sums_of_long_lists_of_zero_values():
    """A list of 16384 slots whose scores rise by 2.5 octaves behind the first 128: the reference
    does not follow, so that weights are at their largest, and value scales of 0 count for 2^-100."""
    K, kvh, d, n = 16384, 8, 64, 8192
    R = _whole_requests(kvh)
    k, v = (torch.full((2, 64, kvh, d), 0x38, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks = torch.tensor([[1.0], [1.5]], device="cuda").expand(2, kvh).contiguous()
    table = torch.ones((R, n // 64), dtype=torch.int32, device="cuda")
    table[:, 0] = 0
    listed = torch.full((R, 1, K), 64, dtype=torch.int32, device="cuda")
    listed[:, :, :128] = 5
    s = 5 * np.log(2)
    cfg = spin.make_kv_config(R, n, 1, kvh, kvh, d, "bf16", s / d)
    q = torch.ones((R, 1, kvh, d), dtype=torch.bfloat16, device="cuda")
    ns = torch.full((R, 1), n, dtype=torch.int32, device="cuda")
    out, lse = _kv.run_attend(cfg, q, (k, v, ks, torch.zeros_like(ks)), table, ns, 1, listed)
    want = np.log(128 * np.exp(s) + (K - 128) * np.exp(1.5 * s))
    # parts of at most 2^7 with roundings of 2^-18, and sums of 4096 rounded 2^-24 each
    assert float((lse.double() - want).abs().max()) <= 2.0 ** -16 + 4096 * 2.0 ** -24
    assert not bool(out.any())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("exponent", [10, 12, 14, 15, 16, 18, 20, 24, 30, 60, 90])
@pytest.mark.parametrize("form", ["dense", "list", "rows", "divided"])
def test_scores_far_from_zero(dtype, exponent, form):
    """Scores of 2^16 to 2^98 that differ by 2^14 and more: one slot takes all of the weight, so that
    out is its value but for the roundings of a weight, 1/l and two products, and lse its score, off by
    at most eight roundings of 2^-24."""
    rng = np.random.default_rng(exponent)
    heads, kvh, d, n = 8, 2, 64, 700
    rows = 3 if form == "rows" else 1
    for sign in (1, -1):
        pools = list(_kv.make_pools(rng, 14, kvh, d))
        pools[0][:] = 0
        pools[0][..., 3] = o.e4m3_encode(rng.choice(np.arange(64, 192, 16), (14, 64, kvh)))
        pools[2][:] = 1.0
        table = _kv.make_table(rng, [n], 14, 2000 if form == "divided" else None)
        for g, i in enumerate(rng.integers(0, n - 2, kvh)):      # the largest score of each head
            pools[0][table[0, i // 64], i % 64, g, 3] = o.e4m3_encode([192.0 if sign > 0 else 48.0])[0]
        q = np.zeros((1, rows, heads, d))
        q[..., 3] = sign * 2.0 ** exponent
        q = torch.from_numpy(q).to(_kv.TYPES[dtype])
        cfg = spin.make_kv_config(1, 64 * table.shape[1], rows, heads, kvh, d, dtype, 1.0)
        listed = rng.permutation(n).astype(np.int32).reshape(1, 1, n) if form == "list" else None
        ns = (n - np.arange(rows - 1, -1, -1, dtype=np.int32))[None]
        out, lse = _kv.run_attend(cfg, q.cuda(), [_kv.dev(x) for x in pools], _kv.dev(table), _kv.dev(ns), rows,
                                  None if listed is None else _kv.dev(listed))
        ref, rlse, _ = o.attend(q.double().numpy(), *pools, table, ns, 1.0, listed)
        rel = (2.0 ** -21 if dtype == "f32" else 2.0 ** -11) + 2.0 ** -21 + _kv.HALF_STEP[dtype]
        assert (np.abs(out.double().cpu().numpy() - ref) <= rel * np.abs(ref)).all()
        assert (np.abs(lse.double().cpu().numpy() - rlse) <= 2.0 ** -21 * np.abs(rlse)).all()


def test_nan_scores_far_from_zero_stay_nan():
    """A NaN key among scores of 2^30."""
    def nan(rng, pools, table, n_slots, listed):
        pools[0][table[0, 1], 3, 1, 7] = 0x7f
    check("bf16", 8, 2, 64, [130], mutate=nan, q_size=2.0 ** 30, scale=1.0, seed=1)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kvh,rows,d,max_slots", [(8, 2, 2, 64, 700), (64, 1, 4, 128, 700), (16, 2, 3, 256, 700),
                                                        (8, 2, 4, 128, 60000)])
def test_value_scales_that_are_not_finite_stay_with_the_rows_that_see_them(bad, dtype, heads, kvh, rows, d, max_slots):
    """A page that every verifier row but the first sees: the first row's bits, and another request's,
    do not depend on its value scale."""
    rng = np.random.default_rng(1)
    pools = list(_kv.make_pools(rng, 16, kvh, d))
    table = _kv.make_table(rng, [128 + rows - 1, 700], 16, -(-max_slots // 64))
    n = np.array([[128 + r for r in range(rows)], [700] * rows], np.int32)
    q = torch.from_numpy(rng.normal(size=(2, rows, heads, d))).to(_kv.TYPES[dtype]).cuda()
    cfg = spin.make_kv_config(2, max_slots, rows, heads, kvh, d, dtype)
    got = []
    for x in (0.01, bad):
        pools[3][table[0, 2]] = x
        got.append(_kv.run_attend(cfg, q, [_kv.dev(p) for p in pools], _kv.dev(table), _kv.dev(n), rows))
    for clean, other in zip(*got):
        assert torch.equal(clean[0, 0], other[0, 0]) and torch.equal(clean[1], other[1])
    assert not bool(got[1][0][0, 1:].isfinite().any())


def test_a_nan_value_does_not_slow_the_call_down():
    """Rows of 100 and 16384 slots with one NaN value that only the long ones see: found while its tile is
    at hand, without a second look at the cache."""
    rng = np.random.default_rng(1)
    kvh, heads, d, R, n = 2, 16, 128, 4, 16384
    ns = _kv.dev(np.tile(np.array([100, n, 0, n], np.int32), (R, 1)))
    pools = list(_kv.make_pools(rng, R * n // 64, kvh, d))
    table = _kv.make_table(rng, [n] * R, R * n // 64)
    cfg = spin.make_kv_config(R, n, 4, heads, kvh, d, "bf16")
    q = torch.from_numpy(rng.normal(size=(R, 4, heads, d))).to(torch.bfloat16).cuda()
    ws, out, dt, times = spin.kv_workspace(cfg, 4), torch.empty_like(q), _kv.dev(table), []
    for nan in (False, True):
        if nan:
            pools[1][table[0, 1], 50, 0, 5] = 0x7f
        dv, best = [_kv.dev(p) for p in pools], float("inf")
        for _ in range(8):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            spin.kv_attend(cfg, q, *dv, dt, ns, 4, None, out, None, ws, None)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        times.append(best)
    got = out.isnan().cpu().numpy()
    assert got.sum() == 2 * heads // kvh and got[0, 1, :heads // kvh, 5].all() and got[0, 3, :heads // kvh, 5].all()
    assert times[1] <= 2 * times[0] + 0.05, times


def test_long_rows_keep_the_second_term_of_fp32_weights():
    """40000 slots of which four take most of the weight, against bounds that do not grow with n.  Scores
    come from one dimension, so that their dot products are exact: |ds| <= es = 4 x 2^-22 S + 2^-22
    (|s| + 8).  The row is divided over the GPU (a CTA an SM at least takes part, or four units of 64 slots
    each): a warp adds up ceil(units / 2) tiles with at most 12 roundings each, and a join every fourth of
    at most 158 pieces, so that sums are off by el = (12 tiles + 40 + 16) 2^-22.  The same weights
    rounded to one f16 term lie outside these bounds."""
    rng = np.random.default_rng(5)
    n, heads, d = 40000, 16, 64
    n_pages = -(-n // 64)
    k = np.zeros((n_pages, 64, 1, d), np.uint8)
    k[..., 3] = o.e4m3_encode(rng.uniform(0, 8, (n_pages, 64, 1)))
    for i, c in zip(rng.choice(n, 4, replace=False), (24.0, 26.0, 28.0, 28.0)):
        k[i // 64, i % 64, 0, 3] = o.e4m3_encode([c])[0]
    v = o.e4m3_encode(np.clip(rng.normal(size=(n_pages, 64, 1, d)) * 100, -448, 448))
    pools = [k, v, np.ones((n_pages, 1), np.float32), np.full((n_pages, 1), 0.01, np.float32)]
    q = np.zeros((1, 1, heads, d))
    q[..., 3] = rng.uniform(0.5, 0.7, heads).astype(np.float32)
    table, ns = rng.permutation(n_pages)[None].astype(np.int32), np.array([[n]], np.int32)
    cfg = spin.make_kv_config(1, n, 1, heads, 1, d, "f32", 1.0)
    out, lse = _kv.run_attend(cfg, torch.from_numpy(q).float().cuda(), [_kv.dev(x) for x in pools], _kv.dev(table),
                              _kv.dev(ns), 1)
    ref, rlse, info = o.attend(q, *pools, table, ns, 1.0)
    cost = n_pages + 4
    ranks = min(torch.cuda.get_device_properties(0).multi_processor_count, -(-cost // 4))
    tiles = -(-(-(-cost // ranks)) // 2)
    es = (4 * info["S"] + info["smax"] + 8) * 2.0 ** -22
    el = (12 * tiles + 40 + 16) * 2.0 ** -22
    tol = (2 * es + 2.0 ** -21 + 2 * el)[..., None] * info["A"] + 2.0 ** -24 * np.abs(ref)
    tol += (n * 2.0 ** -37 * info["top"] * 448)[..., None]
    assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()
    assert (np.abs(lse.double().cpu().numpy() - rlse) <= es + el + 2.0 ** -22 * (np.abs(rlse) + 1)).all()
    # one term of 11 bits instead of two
    i = np.arange(n)
    kc, vv = o.E4M3[k[table[0, i // 64], i % 64, 0]], o.E4M3[v[table[0, i // 64], i % 64, 0]] * float(pools[3][0, 0])
    t = kc @ q[0, 0].T * np.log2(np.e)
    w = np.exp2(t - t.max(0) + 12)
    one = (w.astype(np.float16).astype(float).T @ vv) / w.sum(0)[:, None]
    assert (np.abs(one - ref[0, 0]) > tol[0, 0]).any()
