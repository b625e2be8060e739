"""A prompt's life through the calls together: pages reserved, chunks rotated, appended, attended and weighed, the cache cut
down by that weight, and decoding on what is left; each step against its restatement in 64 bits on the cache as it is."""
import numpy as np
import pytest
import torch

import _kv
from oracle import kv as o
from sparse_attention_indexer_spin_gb300 import spin
from sparse_attention_indexer_spin_gb300 import synthetic as syn

pytestmark = pytest.mark.gpu
H, KVH, D, PAGES, W = 16, 2, 64, 40, 12


def i32(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


def cpu(x):
    return x.cpu().numpy()


class Loop:
    """Two requests and their cache."""

    def __init__(self, dtype="bf16", seed=0):
        self.dtype, self.rng = dtype, np.random.default_rng(seed)
        self.cfg = spin.make_kv_config(2, W * 64, 1, H, KVH, D, dtype)
        self.cache = spin.KvCache(PAGES, KVH, D)
        self.ref, self.status = i32([0] * PAGES), i32([0])
        self.pools, self.pws = spin.PagePools(*self.cache.tensors), spin.pages_workspace(2, PAGES)
        self.table, self.granted = i32(np.full((2, W), -1)), i32([0, 0])
        self.freq, self.magnitude = spin.rope_frequencies(32, 1e4, "parts", 4.0, original=256)
        self.rope = spin.make_rope_config(D, dtype, 32, 16, "interleaved", self.magnitude)
        self.core = spin.PromptAttention(self.cfg, self.cache, 400, 300, self.rope, spin.rope_turns(self.freq))
        self.weight = torch.zeros((2, W * 64), device="cuda")
        self.slots, self.tokens = [0, 0], [0, 0]     # cached slots; tokens so far (positions go on after an eviction)

    def chunk(self, counts, decay=1.0):
        """One chunk of new tokens of each request; returns what the oracle needs."""
        T = sum(counts)
        spin.pages_reserve(self.table, i32(self.slots), i32(counts), self.ref, self.pools, self.granted, self.pws, self.status)
        qkv = torch.from_numpy(self.rng.normal(size=(T, H + 2 * KVH, D))).to(_kv.TYPES[self.dtype]).cuda()
        start = np.concatenate([[0], np.cumsum(counts)])
        pos = np.concatenate([np.arange(t, t + c) for t, c in zip(self.tokens, counts)]).astype(np.int32)
        before, w0 = list(self.slots), cpu(self.weight).copy()
        out, lse = spin.run_prompt(self.core, qkv[:, :H], qkv[:, H:H + KVH], qkv[:, H + KVH:], i32(start), max(counts), i32(before),
                                   self.table, self.status, i32(pos), self.weight, decay)
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0 and cpu(self.granted).tolist() == [1, 1]
        # queries: the rotation's own bound is tested elsewhere; the attention is checked on what it read
        q = self.core.q[:T].double().cpu().numpy()
        half = _kv.HALF_STEP[self.dtype]
        x = qkv[:, :H].double().cpu().numpy()
        ref = o.rope(x, pos, self.freq.tolist(), 16, False, float(np.float32(self.magnitude)))
        assert (np.abs(q - ref) <= half * np.abs(ref) + 1e-5).all()
        pools, table = [cpu(t) for t in self.cache.tensors], cpu(self.table)
        want, wlse, info, live = o.prefill(q, start, before, *pools, table, self.cfg.softmax_scale, W * 64, max(counts))
        assert live.all()
        tol, ltol = _kv.attend_tolerance(self.dtype, D, want, info)
        tol = tol + (info["n"] * 2.0 ** -34 * info["top"] * 448)[..., None]
        assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()
        assert (np.abs(lse.double().cpu().numpy() - wlse) <= ltol + 2.0 ** -22 * (np.abs(wlse) + 1)).all()
        ww, more = o.weigh(q, lse.double().cpu().numpy(), start, before, pools[0], pools[2], table, self.cfg.softmax_scale, decay,
                           w0.astype(np.float64), W * 64, max(counts))
        N = max(counts) * H                # (the bound of test_gpu_kv_weigh.py)
        tol = 2 * ((D / 16 + 4) * 2.0 ** -22 * more["eS"] + 2.0 ** -22 * (more["es"] + 8 * more["add"])) + \
            (N / 16 + 16) * 2.0 ** -22 * more["add"] + 2.0 ** -23 * (np.abs(ww) + np.abs(w0)) + N * 2.0 ** -126
        err = np.abs(cpu(self.weight) - ww)
        assert (err <= tol).all(), [(tuple(i), cpu(self.weight)[tuple(i)], ww[tuple(i)], tol[tuple(i)])
                                    for i in np.argwhere(~(err <= tol))[:8]]
        for r in range(2):
            self.slots[r] += counts[r]
            self.tokens[r] += counts[r]
        return out

    def evict(self, keep):
        table, ref, weight = cpu(self.table), cpu(self.ref), cpu(self.weight)
        n, out, kept = i32(self.slots), torch.empty_like(self.weight), torch.empty_like(self.table)
        spin.pages_evict(self.table, n, self.weight, out, i32(keep), 1, 1, self.ref, kept, spin.pages_evict_workspace(2, W), self.status)
        want = o.evict(table, np.array(self.slots), weight, keep, 1, 1, ref, PAGES)
        for x, y in zip((self.table, n, out, self.ref, kept), want):
            assert np.array_equal(cpu(x), y)
        self.slots, self.weight = [int(x) for x in n.tolist()], out
        assert int(self.status.item()) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_prompt_evict_and_decode(dtype):
    loop = Loop(dtype)
    loop.chunk([300, 70])                     # a first chunk, many query rows
    loop.chunk([100, 1], decay=0.5)           # the next one behind it, and a single token
    assert loop.slots == [400, 71]
    loop.evict([4, -1])
    assert loop.slots == [400 - 3 * 64, 71]
    for _ in range(3):                        # decoded tokens, over what is left
        loop.chunk([1, 1])
    # the attention of single tokens agrees on the cut context
    q = torch.from_numpy(loop.rng.normal(size=(2, 1, H, D))).to(_kv.TYPES[dtype])
    out, lse = _kv.run_attend(loop.cfg, q.cuda(), loop.cache.tensors, loop.table, i32([[n] for n in loop.slots]), 1)
    pools, table = [cpu(t) for t in loop.cache.tensors], cpu(loop.table)
    ref, _, info = o.attend(q.double().numpy(), *pools, table, np.array([[n] for n in loop.slots]), loop.cfg.softmax_scale)
    tol, _ = _kv.attend_tolerance(dtype, D, ref, info)
    assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()
    # nothing of the evicted pages is still counted
    used = table[table >= 0]
    assert np.array_equal(np.bincount(used, minlength=PAGES), cpu(loop.ref))


def test_without_rotation_and_on_another_stream():
    rng = np.random.default_rng(1)
    cfg = spin.make_kv_config(1, 256, 1, H, KVH, D, "bf16")
    cache, table = [spin.KvCache(4, KVH, D) for _ in range(2)], i32([[2, 0, 3, 1]])
    qkv = torch.from_numpy(rng.normal(size=(200, H + 2 * KVH, D))).bfloat16().cuda()
    args = (qkv[:, :H], qkv[:, H:H + KVH], qkv[:, H + KVH:], i32([0, 200]), 200, i32([10]), table, None)
    core = [spin.PromptAttention(cfg, c, 200, 200) for c in cache]
    want = spin.run_prompt(core[0], *args)[0].clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = spin.run_prompt(core[1], *args, stream=s)[0]
    s.synchronize()
    assert torch.equal(want, got) and all(torch.equal(x, y) for x, y in zip(cache[0].tensors, cache[1].tensors))


def test_captured_prompt():
    loop, eager = Loop(seed=3), Loop(seed=3)
    for x in (loop, eager):
        x.chunk([200, 64])
    T, counts = 90, [60, 30]
    for x in (loop, eager):
        spin.pages_reserve(x.table, i32(x.slots), i32([70, 70]), x.ref, x.pools, x.granted, x.pws, x.status)
    qkv = torch.from_numpy(loop.rng.normal(size=(T, H + 2 * KVH, D))).bfloat16().cuda()
    start, before, pos = i32([0, 60, 90]), i32(loop.slots), i32(np.arange(T))
    call = lambda x: spin.run_prompt(x.core, qkv[:, :H], qkv[:, H:H + KVH], qkv[:, H + KVH:], start, 64, before, x.table,  # noqa: E731
                                     x.status, pos, x.weight)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out, lse = call(loop)
    qkv.mul_(1.5)                              # other values, positions and counts than the captured ones
    pos.add_(1000)
    start.copy_(i32([0, 64, 84]))
    graph.replay()
    want, wlse = call(eager)
    torch.cuda.synchronize()
    assert counts and torch.equal(out[:84], want[:84]) and torch.equal(lse[:84], wlse[:84])
    assert torch.equal(loop.weight, eager.weight)
    assert all(torch.equal(x, y) for x, y in zip(loop.cache.tensors, eager.cache.tensors))


def test_two_streams_at_once():
    want, streams, got = [], [torch.cuda.Stream(), torch.cuda.Stream()], []
    loops = [Loop(seed=s) for s in (5, 6)]
    qkv = [torch.from_numpy(x.rng.normal(size=(360, H + 2 * KVH, D))).bfloat16().cuda() for x in loops]

    def call(x, y, stream=None):
        spin.pages_reserve(x.table, i32([0, 0]), i32([290, 70]), x.ref, x.pools, x.granted, x.pws, x.status)
        start, before, pos = i32([0, 290, 360]), i32([0, 0]), i32(np.arange(360))
        torch.cuda.synchronize()
        for _ in range(10):
            spin.run_prompt(x.core, y[:, :H], y[:, H:H + KVH], y[:, H + KVH:], start, 290, before, x.table, x.status, pos, x.weight,
                            0.5, stream=stream)
        return start, before, pos
    for x, y in zip(loops, qkv):
        call(x, y)
        torch.cuda.synchronize()
        want.append([t.clone() for t in (x.core.out[:360], x.core.lse[:360], x.weight)])
        x.weight.zero_()
        x.core.out.zero_()
    keep = [[i32([0, 290, 360]), i32([0, 0]), i32(np.arange(360))] for _ in loops]
    torch.cuda.synchronize()
    for _ in range(10):
        for x, y, s, (start, before, pos) in zip(loops, qkv, streams, keep):
            spin.run_prompt(x.core, y[:, :H], y[:, H:H + KVH], y[:, H + KVH:], start, 290, before, x.table, x.status, pos, x.weight,
                            0.5, stream=s)
    torch.cuda.synchronize()
    for x, w in zip(loops, want):
        for a, b in zip((x.core.out[:360], x.core.lse[:360], x.weight), w):
            assert torch.equal(a, b)
        assert int(x.status.item()) == 0


def test_nothing_behind_the_workspaces_is_written():
    rng = np.random.default_rng(2)
    for dtype, d, counts, before in (("bf16", 128, [200, 3], [0, 500]), ("f32", 256, [130, 1], [70, 64]), ("f16", 64, [1, 1], [900, 7])):
        cfg = spin.make_kv_config(2, 1024, 1, H, KVH, d, dtype)
        T = sum(counts)
        cache, table = spin.KvCache(40, KVH, d), i32(np.arange(32).reshape(2, 16))
        q = torch.from_numpy(rng.normal(size=(T, H, d))).to(_kv.TYPES[dtype]).cuda()
        out, lse, weight = torch.empty_like(q), torch.empty((T, H), device="cuda"), torch.zeros((2, 1024), device="cuda")
        start, before, status = i32([0, counts[0], T]), i32(before), i32([0])
        for size in (spin.kv_prefill_workspace, spin.kv_weigh_workspace):
            n = size(cfg, T, max(counts)).numel()
            room = torch.full((n + 65536,), 0x5a, dtype=torch.uint8, device="cuda")
            if size is spin.kv_prefill_workspace:
                spin.kv_prefill(cfg, q, start, max(counts), before, *cache.tensors, table, out, lse, room[:n], status)
            else:
                spin.kv_weigh(cfg, q, lse, start, max(counts), before, cache.k, cache.k_scale, table, 1.0, weight, room[:n], status)
            assert (room[n:] == 0x5a).all()
        assert int(status.item()) == 0


def test_pages_beyond_four_gigabytes():
    # the same pages at the end of a pool of 5 GB (each for keys and values) and in a small one: the same bits
    rng = np.random.default_rng(8)
    kvh, d, n = 8, 256, 40000
    small, big = spin.KvCache(8, kvh, d), spin.KvCache(n, kvh, d)
    for s, b in zip(small.tensors, big.tensors):
        if s.dtype == torch.uint8:
            s.copy_(torch.from_numpy(rng.integers(0, 0x70, tuple(s.shape), dtype=np.uint8)))
        else:
            s.fill_(0.01)
        b[-8:] = s
    table = rng.permutation(8).reshape(1, 8)
    for dtype, new, before in (("bf16", 150, 300), ("f32", 40, 460), ("bf16", 1, 500)):
        cfg = spin.make_kv_config(1, 512, 1, 16, kvh, d, dtype)
        q = torch.from_numpy(rng.normal(size=(new, 16, d))).to(_kv.TYPES[dtype]).cuda()
        got = []
        for cache, at in ((small, 0), (big, n - 8)):
            out, lse = torch.empty_like(q), torch.empty((new, 16), device="cuda")
            weight, status, t = torch.zeros((1, 512), device="cuda"), i32([0]), i32(table + at)
            args = (i32([0, new]), new, i32([before]))
            spin.kv_prefill(cfg, q, *args, *cache.tensors, t, out, lse, spin.kv_prefill_workspace(cfg, new, new), status)
            spin.kv_weigh(cfg, q, lse, *args, cache.k, cache.k_scale, t, 1.0, weight, spin.kv_weigh_workspace(cfg, new, new), status)
            assert int(status.item()) == 0 and abs(float(weight.double().sum()) - 16 * new) < 0.01 * new
            got.append((out, lse, weight))
        for x, y in zip(*got):
            assert torch.equal(x, y)


def test_no_tokens():
    loop = Loop()
    loop.chunk([70, 3])
    before = [t.clone() for t in loop.cache.tensors] + [loop.weight.clone()]
    q, kv = (torch.empty((0, h, D), dtype=torch.bfloat16, device="cuda") for h in (H, KVH))
    out, lse = spin.run_prompt(loop.core, q, kv, kv, i32([0, 0, 0]), 0, i32(loop.slots), loop.table, loop.status, i32([]), loop.weight)
    torch.cuda.synchronize()
    assert out.shape == (0, H, D) and lse.shape == (0, H) and int(loop.status.item()) == 0
    for x, y in zip(loop.cache.tensors + (loop.weight,), before):
        assert torch.equal(x, y)


def test_refused_chunks_launch_nothing():
    loop = Loop()
    loop.chunk([10, 10])
    before = [t.clone() for t in loop.cache.tensors] + [loop.weight.clone()]
    q = torch.randn((4, H, D), device="cuda").bfloat16()
    kv = torch.randn((4, KVH, D), device="cuda").bfloat16()
    good = dict(q=q, k=kv, v=kv, new_start=i32([0, 2, 4]), max_new=2, n_before=i32([10, 10]), block_table=loop.table, status=loop.status,
                positions=i32(range(4)), weight=loop.weight)
    for name, bad in (("q", q.float()), ("k", kv[:2]), ("v", kv[:, :1]), ("new_start", i32([0, 4])), ("max_new", 301), ("max_new", -1),
                      ("n_before", i32([1])), ("block_table", loop.table[:, :3]), ("positions", i32([1])), ("positions", None),
                      ("weight", loop.weight[:, :64]), ("status", i32([0, 0])), ("q", q.transpose(0, 1).contiguous().transpose(0, 1))):
        with pytest.raises(spin.SpinError):
            spin.run_prompt(loop.core, **{**good, name: bad})
    for x, y in zip(loop.cache.tensors + (loop.weight,), before):
        assert torch.equal(x, y)
    with pytest.raises(spin.SpinError):
        spin.PromptAttention(loop.cfg, loop.cache, 4, 4, spin.make_rope_config(128, "bf16"), loop.core.turns)


@pytest.mark.parametrize("hinted", [False, True])
def test_the_indexer_after_an_eviction(hinted):
    """Requests that lost blocks have their state reset: the next step selects all that stayed and scores it as a state does
    that never saw what left; the request that kept its blocks goes on as it was."""
    wl = syn.CONFIGS["pr1"].replace(steps=6, n_layers=1, n_req=3, n0=900, top_k=64)
    inp = syn.SyntheticInputs(wl, "cuda")
    cfg = spin.make_config(**wl.config_fields())
    R, width = wl.n_req, inp.block_table.shape[1]
    states = [spin.LayerState(cfg) for _ in range(2)]
    bufs = [spin.StepBuffers(cfg) for _ in range(2)]
    hints = [spin.TopkHint(cfg) if hinted else None for _ in range(2)]

    def step(i, n):
        spin.run_step(cfg, states[i], bufs[i], q, w, inp.k_pool[0], inp.k_scale[0], inp.n_pages, table, n, qp, n_step, 0, hint=hints[i])

    table = inp.block_table.clone()
    for n_step in range(3):
        q, w, qp = inp.step_inputs()
        step(0, inp.n_slots)
        inp.advance(n_step)
    q, w, qp = inp.step_inputs()
    n = inp.n_slots.clone()
    blocks = (n + 63) // 64
    ref = torch.bincount(table[table >= 0].long(), minlength=inp.n_pages).to(torch.int32)
    weight = torch.rand((R, 64 * width), device="cuda")
    left, kept, status = torch.empty_like(weight), torch.empty_like(table), i32([0])
    spin.pages_evict(table, n, weight, left, i32([int(blocks[0]) - 5, -1, 3]), 1, 1, ref, kept, spin.pages_evict_workspace(R, width), status)
    assert int(n[0]) == int(inp.n_slots[0]) - 5 * 64 and int(status.item()) == 0
    for r in (0, 2):
        spin.init_state(cfg, *(getattr(states[0], x) for x in ("V", "D", "Vmax", "warm")), r)
        if hinted:
            hints[0].reset(r)
    qp, n_step = n - 1, 3                          # (a query stands in its slot)
    step(0, n)
    step(1, n)                                     # a state that is new for every request
    torch.cuda.synchronize()
    assert int(bufs[0].status.item()) == 0 and int(bufs[1].status.item()) == 0
    for r in (0, 2):
        m = (int(n[r]) + 63) // 64
        assert int(bufs[0].n_blocks[r, 0]) == m and bufs[0].blocks[r, 0, :m].tolist() == list(range(m))
        for x, y in ((bufs[0].topk, bufs[1].topk), *((getattr(states[0], x), getattr(states[1], x)) for x in ("V", "D", "Vmax", "warm"))):
            assert torch.equal(x[r], y[r])
    assert int(bufs[0].n_blocks[1, 0]) < int(bufs[1].n_blocks[1, 0])      # (warm: it selects)
