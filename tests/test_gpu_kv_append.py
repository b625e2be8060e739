"""Appending to the 8-bit KV cache: codes and scales equal the definition's bit for bit (the
scales are powers of two, so every quotient is exact and only the rounding to e4m3 is left)."""
import numpy as np
import pytest
import torch

import _kv
from oracle import kv as o
from sparse_attention_indexer_spin_gb300 import spin

pytestmark = pytest.mark.gpu


def same_codes(a, b):
    """Equal codes, NaN codes of either sign being alike."""
    return np.array_equal(np.where((a & 127) == 127, 127, a), np.where((b & 127) == 127, 127, b))


def check(dtype, kvh, d, before, counts, seed=0, size=1.0, mutate=None, max_new=None, scale_pow2=True):
    rng = np.random.default_rng(seed)
    R = len(before)
    lens = [b + c for b, c in zip(before, counts)]
    n_pages = sum(-(-n // 64) for n in lens) + 3
    pools = list(_kv.make_pools(rng, n_pages, kvh, d))
    if scale_pow2:
        pools[2:] = [np.exp2(np.round(np.log2(x))).astype(np.float32) for x in pools[2:]]
    table = _kv.make_table(rng, lens, n_pages)
    start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    T = int(start[-1])
    new = [torch.from_numpy(rng.normal(size=(T, kvh, d)) * np.exp(2 * rng.normal(size=(T, kvh, 1))) * size)
           .to(_kv.TYPES[dtype]) for _ in range(2)]
    if mutate:
        mutate(rng, new, pools)
    cfg = spin.make_kv_config(R, max(max(lens), 1), 1, kvh, kvh, d, dtype)
    dv = [_kv.dev(x) for x in pools]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (cfg, new[0].cuda(), new[1].cuda(), _kv.dev(start), max(counts) if max_new is None else max_new,
            _kv.dev(np.array(before, np.int32)), *dv, _kv.dev(table), status)
    spin.kv_append(*args)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for i in range(2):
        o.append(new[i].double().numpy(), start, before, pools[i], pools[2 + i], table)
    got = [x.cpu().numpy() for x in dv]
    for i in range(2):
        assert np.array_equal(got[2 + i], pools[2 + i])
        assert same_codes(got[i], pools[i])
    # the same call again changes nothing: the scales already cover the new values
    spin.kv_append(*args)
    torch.cuda.synchronize()
    for x, y in zip(dv, got):
        assert np.array_equal(x.cpu().numpy(), y, equal_nan=x.dtype == torch.float32)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kvh,d", [(1, 16), (8, 128), (2, 64), (3, 80), (1, 256), (4, 240)])
def test_tokens_and_prompts(dtype, kvh, d):
    check(dtype, kvh, d, [0, 5, 63, 64, 100, 130], [1, 1, 1, 1, 1, 1], seed=d)
    check(dtype, kvh, d, [0, 5, 63, 64, 100, 130, 7], [64, 200, 1, 2, 0, 65, 130], seed=d)


@pytest.mark.parametrize("before,count", [(b, c) for b in (0, 1, 62, 63, 64) for c in (1, 2, 63, 64, 65, 66, 129)])
def test_page_borders(before, count):
    check("bf16", 2, 32, [before, 3], [count, 1], seed=before)


@pytest.mark.parametrize("size", [1e-30, 1e-6, 1.0, 1e6, 1e30])
def test_sizes_that_grow_or_keep_the_scale(size):
    check("f32", 2, 64, [0, 30, 63, 90], [3, 5, 2, 40], size=size, seed=1)
    check("bf16", 2, 64, [0, 30, 63, 90], [3, 5, 2, 40], size=size, seed=1)


def test_scale_borders():
    """max|x| exactly 448 s, one step above it, the smallest normal and subnormal numbers, and the
    largest finite one."""
    top = np.float32(3.4028235e38)
    vals = [448.0, np.nextafter(np.float32(448), np.float32(1e9)), 1.75, 1.7500001, 2.0 ** -126, 2.0 ** -149,
            448 * 2.0 ** -126, float(top), 1e-38, 0.0]

    def put(rng, new, pools):
        for x in new:
            x[:] = 0.0
            for t, val in enumerate(vals):
                x[t, 0, t] = float(val)
    check("f32", 1, 16, [0] * len(vals), [1] * len(vals), mutate=put)
    check("f32", 1, 16, [7] * len(vals), [1] * len(vals), mutate=put)


def test_nan_and_infinite_values():
    """Infinities saturate and do not set the scale; NaN stays NaN."""
    def put(rng, new, pools):
        for x in new:
            x[0, 0, 3], x[1, 1, 4], x[2, 0, :] = float("inf"), float("nan"), float("-inf")
        pools[0][:, 2] = 0x7f          # NaN codes among the earlier slots
    check("bf16", 2, 64, [10, 0], [4, 2], mutate=put)
    check("f32", 2, 64, [10, 0], [4, 2], mutate=put)


def test_all_zero_pages_then_values():
    def zero(rng, new, pools):
        for x in new:
            x[:] = 0.0
    check("bf16", 2, 64, [0, 64, 5], [3, 1, 2], mutate=zero)

    def was_zero(rng, new, pools):
        for i in range(2):
            pools[i][:] = 0
            pools[2 + i][:] = 0.0
    check("bf16", 2, 64, [3, 70, 5], [3, 1, 2], mutate=was_zero)


def test_scales_that_are_no_powers_of_two():
    check("bf16", 2, 64, [10, 20, 63], [4, 70, 2], scale_pow2=False, seed=3)


def test_appending_token_by_token_leaves_other_pages_alone():
    """Many single-token calls; the oracle follows call by call."""
    rng = np.random.default_rng(4)
    kvh, d, R = 2, 48, 3
    pools = list(_kv.make_pools(rng, 12, kvh, d))
    table = _kv.make_table(rng, [150, 150, 150], 12)
    cfg = spin.make_kv_config(R, 150, 1, kvh, kvh, d, "f16")
    dv, dt = [_kv.dev(x) for x in pools], _kv.dev(table)
    n = np.array([0, 50, 60], np.int32)
    for step in range(80):
        start = np.arange(R + 1, dtype=np.int32)
        new = [torch.from_numpy(rng.normal(size=(R, kvh, d)) * 2.0 ** rng.integers(-6, 6)).to(torch.float16)
               for _ in range(2)]
        spin.kv_append(cfg, new[0].cuda(), new[1].cuda(), _kv.dev(start), 1, _kv.dev(n), *dv, dt, None)
        for i in range(2):
            o.append(new[i].double().numpy(), start, n, pools[i], pools[2 + i], table)
        n = n + 1
    for x, y in zip(dv, pools):
        assert np.array_equal(x.cpu().numpy(), y)


def test_bad_counts_and_pages_are_skipped():
    rng = np.random.default_rng(4)
    kvh, d = 2, 32
    cfg = spin.make_kv_config(4, 128, 1, kvh, kvh, d, "f32")
    new = torch.randn((8, kvh, d), device="cuda")
    B = spin.STATUS_BITS

    def run(start, before, table, max_new, want, touched):
        pools = [_kv.dev(x) for x in _kv.make_pools(rng, 8, kvh, d)]
        old = [x.clone() for x in pools]
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        spin.kv_append(cfg, new, new, _kv.dev(np.array(start, np.int32)), max_new, _kv.dev(np.array(before, np.int32)),
                       *pools, _kv.dev(np.array(table, np.int32)), status)
        torch.cuda.synchronize()
        assert int(status.item()) == want
        changed = {int(p) for x, y in zip(pools, old) for p in (x != y).flatten(1).any(1).nonzero().view(-1)}
        assert changed == set(touched)

    table = [[0, 1], [2, 3], [4, 5], [6, 7]]
    run([0, 2, 4, 6, 8], [0, 0, 0, 0], table, 2, 0, {0, 2, 4, 6})
    run([0, 2, 4, 6, 8], [0, -1, 127, 64], table, 2, B["BAD_N"], {0, 7})          # negative, past max_slots
    run([0, 2, 1, 6, 9], [0, 0, 0, 0], table, 5, B["BAD_N"], {0, 4})              # descending, past the end
    run([0, 2, 5, 6, 8], [0, 0, 0, 0], table, 2, B["BAD_N"], {0, 4, 6})           # more than max_new
    run([0, 2, 4, 6, 8], [0, 63, 0, 0], [[0, 1], [2, -1], [8, 5], [6, 7]], 2, B["BAD_PAGE"], {0, 2, 6})
    run([0, 0, 0, 0, 0], [0, 0, 0, 0], table, 0, 0, set())


def test_pool_beyond_32_bit_offsets():
    n_pages, kvh, d = 70000, 8, 128
    k, v = (torch.zeros((n_pages, 64, kvh, d), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((n_pages, kvh), device="cuda") for _ in range(2))
    cfg = spin.make_kv_config(1, 128, 1, kvh, kvh, d, "bf16")
    x = torch.randn((3, kvh, d), device="cuda").to(torch.bfloat16)
    table = np.array([[69999, 69000]], np.int32)
    spin.kv_append(cfg, x, -x, _kv.dev(np.array([0, 3], np.int32)), 3, _kv.dev(np.array([62], np.int32)), k, v, ks, vs,
                   _kv.dev(table), None)
    pk, sk = np.zeros((2, 64, kvh, d), np.uint8), np.zeros((2, kvh), np.float32)
    o.append(x.double().cpu().numpy(), [0, 3], [62], pk, sk, np.array([[0, 1]]))
    at = [69999, 69000]
    assert np.array_equal(k[at].cpu().numpy(), pk) and np.array_equal(ks[at].cpu().numpy(), sk)
    assert np.array_equal(v[at].cpu().numpy()[pk != 0], (pk ^ 128)[pk != 0]) and np.array_equal(vs[at].cpu().numpy(), sk)
    assert int((k != 0).flatten(1).any(1).sum()) == 2


def test_one_prompt_among_many_requests():
    """Ragged counts of more requests than a CTA looks at in one go, some refused."""
    rng = np.random.default_rng(9)
    kvh, d, R = 2, 32, 700
    count = rng.integers(0, 4, R)
    count[[3, 255, 256, 640]] = [500, 130, 65, 333]
    before = rng.integers(0, 200, R)
    bad = np.array([0, 77, 256, 511, 699])
    n_pages = int(sum(-(-(b + c) // 64) for b, c in zip(before, count))) + 3
    table = _kv.make_table(rng, before + count, n_pages)
    start = np.concatenate([[0], np.cumsum(count)]).astype(np.int32)
    new = [torch.from_numpy(rng.normal(size=(int(start[-1]), kvh, d))).to(torch.bfloat16) for _ in range(2)]
    cfg = spin.make_kv_config(R, 64 * table.shape[1], 1, kvh, kvh, d, "bf16")
    pools = list(_kv.make_pools(rng, n_pages, kvh, d))
    dv, status = [_kv.dev(x) for x in pools], torch.zeros(1, dtype=torch.int32, device="cuda")
    given = before.copy()
    given[bad] = [-1, cfg.max_slots + 1, -5, cfg.max_slots + 1, -2 ** 31]
    spin.kv_append(cfg, *[x.cuda() for x in new], _kv.dev(start), 500, _kv.dev(given.astype(np.int32)), *dv, _kv.dev(table),
                   status)
    assert int(status.item()) == spin.STATUS_BITS["BAD_N"]
    for r in range(R):
        if r in bad:
            continue
        for i in range(2):
            o.append(new[i].double().numpy()[start[r]:start[r + 1]], [0, count[r]], before[r:r + 1], pools[i], pools[2 + i],
                     table[r:r + 1])
    for x, y in zip(dv, pools):
        assert np.array_equal(x.cpu().numpy(), y)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("d", [32, 128, 256])
def test_infinities_beside_nothing_finite(dtype, d):
    """A head whose new values are infinities, NaN and zeros: codes of 448 and NaN under a scale of 0, which
    the page's next finite values turn into zeros (and NaN)."""
    kvh, inf = 2, float("inf")
    cfg = spin.make_kv_config(1, 64, 1, kvh, kvh, d, dtype)
    c, table = spin.KvCache(1, kvh, d), _kv.dev(np.zeros((1, 1), np.int32))

    def put(x, at):
        x = x.to(_kv.TYPES[dtype]).cuda()
        spin.kv_append(cfg, x, -x, _kv.dev(np.array([0, 1], np.int32)), 1, _kv.dev(np.array([at], np.int32)), *c.tensors,
                       table, None)

    x = torch.zeros((1, kvh, d))
    x[0, 0, 3], x[0, 0, 5], x[0, 1, :] = inf, float("nan"), -inf
    put(x, 0)
    want = torch.zeros((kvh, d), dtype=torch.uint8)
    want[0, 3], want[1, :] = 0x7e, 0xfe
    for pool, flip in ((c.k, 0), (c.v, 0x80)):
        got = pool[0, 0].cpu()
        assert int(got[0, 5]) & 0x7f == 0x7f
        got[0, 5] = want[0, 5] ^ flip
        assert torch.equal(got ^ flip, want)
    assert not bool(c.k_scale.any()) and not bool(c.v_scale.any())
    put(torch.ones((1, kvh, d)), 1)
    assert bool((c.k_scale == 2.0 ** -8).all())
    old = c.k[0, 0].cpu() & 0x7f
    assert int(old[0, 5]) == 0x7f and int((old != 0).sum()) == 1

    def mixed(rng, new, pools):
        for x in new:
            x[:] = 0.0
            x[0, 0, 3], x[0, 1, :], x[2, 0, 5], x[3, 1, 6] = inf, -inf, float("nan"), inf
        for i in (0, 1):
            pools[2 + i][:] = 0.0
    check(dtype, 2, d, [0, 64, 5], [1, 1, 2], mutate=mixed)


def test_counts_are_checked_where_max_new_is_zero():
    """Counts above a max_new of 0, and bad places, are reported and nothing is written."""
    kvh, d = 2, 32
    cfg = spin.make_kv_config(3, 128, 1, kvh, kvh, d, "f32")
    new = torch.randn((8, kvh, d), device="cuda")
    table = _kv.dev(np.arange(6, dtype=np.int32).reshape(3, 2))
    for start, before, want in (([0, 2, 2, 2], [0, 0, 0], "BAD_N"), ([0, 0, 0, 0], [0, -1, 0], "BAD_N"),
                                ([3, 3, 3, 1], [0, 0, 0], "BAD_N"), ([5, 5, 5, 5], [0, 128, 7], None)):
        pools = [_kv.dev(x) for x in _kv.make_pools(np.random.default_rng(0), 6, kvh, d)]
        old = [x.clone() for x in pools]
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        spin.kv_append(cfg, new, new, _kv.dev(np.array(start, np.int32)), 0, _kv.dev(np.array(before, np.int32)), *pools,
                       table, status)
        assert int(status.item()) == (spin.STATUS_BITS[want] if want else 0)
        assert all(torch.equal(x, y) for x, y in zip(pools, old))
    # no new tokens at all: the arrays behind new_k and new_v are not looked at
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    spin.kv_append(cfg, new[:0], new[:0], _kv.dev(np.zeros(4, np.int32)), 0, _kv.dev(np.zeros(3, np.int32)), *pools, table,
                   status)
    assert int(status.item()) == 0 and all(torch.equal(x, y) for x, y in zip(pools, old))
