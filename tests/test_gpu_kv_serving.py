"""The cache's calls together, as a serving loop makes them: decode steps of the indexer with the
core attention behind it, and beams that fork, write, leave and are compacted."""
import numpy as np
import pytest
import torch

import _kv
from oracle import kv as o
from sparse_attention_indexer_spin_gb300 import spin
from sparse_attention_indexer_spin_gb300 import synthetic as syn

pytestmark = pytest.mark.gpu


def dev32(x):
    return _kv.dev(np.asarray(x, np.int32))


@pytest.mark.parametrize("name,over,heads,kvh,d", [
    ("pr1", dict(n_req=3, n0=500, top_k=64), 16, 2, 64),
    ("v4flash", dict(n_req=2, n0=900, top_k=256), 64, 1, 128),
    ("mtp", dict(n_req=2, n0=700, top_k=128, mean_accept=2.4), 32, 8, 128),
])
def test_decode_steps_with_core_attention(name, over, heads, kvh, d):
    """run_step with a CoreAttention: each step appends the newest slots' keys and values, and the
    core attention reads the step's top-K of them (eagerly, and from a captured graph for one row)."""
    wl = syn.CONFIGS[name].replace(steps=4, n_layers=1, **over)
    inp = syn.SyntheticInputs(wl, "cuda")
    cfg = spin.make_config(**wl.config_fields())
    rows, R = wl.rows, wl.n_req
    st, buf = spin.LayerState(cfg), spin.StepBuffers(cfg, rows)
    spin.init_state(cfg, st.V, st.D, st.Vmax, st.warm)
    cache = spin.KvCache(inp.n_pages, kvh, d)
    kcfg = spin.make_kv_config(R, wl.max_slots, rows, heads, kvh, d, "bf16")
    core = spin.CoreAttention(kcfg, cache, rows, wl.top_k)
    rng = np.random.default_rng(1)
    table = inp.block_table.cpu().numpy()
    pools = [x.cpu().numpy().copy() for x in cache.tensors]
    n = np.zeros(R, np.int64)
    for step in range(wl.steps):
        q, w, qp = inp.step_inputs()
        # the slots the cache does not hold yet
        now = inp.n_slots.cpu().numpy().astype(np.int64)
        counts = now - n
        start = np.concatenate([[0], np.cumsum(counts)])
        new = [torch.from_numpy(rng.normal(size=(int(start[-1]), kvh, d))).to(torch.bfloat16) for _ in range(2)]
        spin.kv_append(kcfg, new[0].cuda(), new[1].cuda(), dev32(start), int(counts.max()), dev32(n), *cache.tensors,
                       inp.block_table, buf.status)
        for i in range(2):
            o.append(new[i].double().numpy(), start, n, pools[i], pools[2 + i], table)
        n = now
        cq = torch.from_numpy(rng.normal(size=(R, rows, heads, d))).to(torch.bfloat16)
        accepted = inp.draw_accepted() if rows > 1 else None
        spin.run_step(cfg, st, buf, q, w, inp.k_pool[0], inp.k_scale[0], inp.n_pages, inp.block_table, inp.n_slots, qp,
                      step, 0, accepted=None if accepted is None else accepted.cuda(), core=core, core_q=cq.cuda())
        torch.cuda.synchronize()
        assert int(buf.status.item()) == 0
        for x, y in zip(cache.tensors, pools):
            assert np.array_equal(x.cpu().numpy(), y)
        topk = buf.topk.cpu().numpy()
        assert (topk[:, :, 0] >= 0).all()
        ns = np.repeat(now[:, None], rows, 1)
        ref, rlse, info = o.attend(cq.double().numpy(), *pools, table, ns, kcfg.softmax_scale, topk)
        tol, ltol = _kv.attend_tolerance("bf16", d, ref, info)
        assert (np.abs(core.out.double().cpu().numpy() - ref) <= tol).all()
        assert (np.abs(core.lse.double().cpu().numpy() - rlse) <= ltol + 2.0 ** -22 * (np.abs(rlse) + 1)).all()
        inp.advance(step, accepted)
    if rows > 1:
        return
    # the attention alone, captured and replayed on the last step's buffers
    want = core.out.clone()
    cq, seen = cq.cuda(), dev32(now)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        core.attend(cq, inp.block_table, seen, buf.topk, buf.status)
    core.out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(core.out, want)


def test_beams_fork_write_leave_and_compact():
    """A beam search over a page pool: every beam's attention always equals that of a private, never
    shared copy of its history; compaction changes no output bit."""
    rng = np.random.default_rng(3)
    R, kvh, heads, d, max_slots, n_pages = 6, 2, 8, 64, 640, 64
    MB = max_slots // 64
    cfg = spin.make_kv_config(R, max_slots, 1, heads, kvh, d, "f16")
    cache, ws = spin.KvCache(n_pages, kvh, d), spin.pages_workspace(R, n_pages)
    extra = torch.zeros((n_pages, 64), dtype=torch.float32, device="cuda")   # e.g. an indexer's key scales
    pools = spin.PagePools(*cache.tensors, extra)
    tables = [torch.full((R, MB), -1, dtype=torch.int32, device="cuda") for _ in range(2)]
    ref = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    status, granted, n_live = (torch.zeros(k, dtype=torch.int32, device="cuda") for k in (1, R, 1))
    # each beam's private history: a cache of its own in numpy
    own = [[np.zeros((MB, 64, kvh, d), np.uint8) for _ in range(2)] + [np.zeros((MB, kvh), np.float32) for _ in range(2)]
           for _ in range(R)]
    n = np.zeros(R, np.int64)
    line = np.arange(MB)[None]

    def write(counts):
        counts = np.asarray(counts)
        spin.pages_reserve(tables[0], dev32(n), dev32(counts), ref, pools, granted, ws, status)
        assert bool(granted.all())
        start = np.concatenate([[0], np.cumsum(counts)])
        new = [torch.from_numpy(rng.normal(size=(int(start[-1]), kvh, d)) * 2.0 ** rng.integers(-3, 3)).to(torch.float16)
               for _ in range(2)]
        spin.kv_append(cfg, new[0].cuda(), new[1].cuda(), dev32(start), int(counts.max()), dev32(n), *cache.tensors,
                       tables[0], status)
        for b in range(R):
            for i in range(2):
                o.append(new[i][start[b]:start[b + 1]].double().numpy(), [0, counts[b]], [n[b]], own[b][i],
                         own[b][2 + i], line)
            n[b] += counts[b]

    def attend():
        q = torch.from_numpy(rng.normal(size=(R, 1, heads, d))).to(torch.float16)
        out, _ = _kv.run_attend(cfg, q.cuda(), cache.tensors, tables[0], dev32(n[:, None]), 1, status=status)
        again = lambda: _kv.run_attend(cfg, q.cuda(), cache.tensors, tables[0], dev32(n[:, None]), 1, status=status)[0]
        for b in range(R):
            want, _, info = o.attend(q[b:b + 1].double().numpy(), *own[b], line, n[b:b + 1, None], cfg.softmax_scale)
            tol, _ = _kv.attend_tolerance("f16", d, want, info)
            assert (np.abs(out[b:b + 1].double().cpu().numpy() - want) <= tol).all(), b
        return out, again

    def check_counts():
        t = tables[0].cpu().numpy()
        assert np.array_equal(np.bincount(t[t >= 0], minlength=n_pages), ref.cpu().numpy())

    write([100, 64, 30, 1, 0, 200])
    attend()
    for step in range(12):
        parent = rng.integers(0, R, R)
        spin.pages_fork(tables[0], dev32(parent), tables[1], ref, status)
        tables.reverse()
        own = [[x.copy() for x in own[p]] for p in parent]
        n = n[parent].copy()
        write(rng.integers(0, 40, R) * (rng.random(R) < 0.8))
        out, again = attend()
        check_counts()
        if step % 3 == 2:
            # some beams are cut back (a rejected draft), others leave
            keep = np.where(rng.random(R) < 0.3, np.maximum(n - 50, 0), -1)
            keep[rng.integers(0, R)] = 0
            spin.pages_free(tables[0], dev32(keep), ref, status)
            n = np.where(keep >= 0, keep, n)
            out, again = attend()
            before = tables[0].cpu().numpy()
            spin.pages_compact(tables[0], ref, pools, n_live, ws, status)
            live = int(n_live.item())
            assert live == len(set(before[before >= 0])) and bool((ref[:live] > 0).all()) and int(ref[live:].sum()) == 0
            check_counts()
            assert torch.equal(again().view(torch.uint8), out.view(torch.uint8))
    assert int(status.item()) == 0


def test_two_streams_at_once():
    """Two attentions on two streams at the same time, each with a workspace of its own, and an
    append on a third: the results are those of the calls one after the other."""
    rng = np.random.default_rng(2)
    lens, kvh, d = [3000, 700, 64, 2], 2, 128
    cfg = spin.make_kv_config(4, 3100, 1, 16, kvh, d, "bf16")
    n_pages = 80
    pools = [_kv.dev(x) for x in _kv.make_pools(rng, n_pages, kvh, d)]
    table = _kv.dev(_kv.make_table(rng, lens, n_pages, 49))
    n = dev32(np.array(lens)[:, None])
    q = [torch.from_numpy(rng.normal(size=(4, 1, 16, d))).to(torch.bfloat16).cuda() for _ in range(2)]
    want = [_kv.run_attend(cfg, x, pools, table, n, 1)[0] for x in q]
    other = spin.KvCache(8, kvh, d)
    acfg = spin.make_kv_config(1, 512, 1, kvh, kvh, d, "bf16")
    x = torch.randn((500, kvh, d), device="cuda").to(torch.bfloat16)
    args = (acfg, x, x, dev32([0, 500]), 500, dev32([3]))
    tail = (*other.tensors, dev32(np.arange(8)[None]), None)
    spin.kv_append(*args, *tail)
    codes = other.k.clone()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs, ws = [torch.zeros_like(x_) for x_ in q], [spin.kv_workspace(cfg) for _ in q]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            spin.kv_attend(cfg, q[i], *pools, table, n, 1, None, outs[i], None, ws[i], None, stream=streams[i])
        spin.kv_append(*args, *tail, stream=streams[2])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1]) and torch.equal(other.k, codes)


def test_a_step_with_a_wrong_core_attention_launches_nothing():
    wl = syn.CONFIGS["pr1"].replace(steps=2, n_layers=1, n_req=3, n0=500, top_k=64)
    inp, cfg = syn.SyntheticInputs(wl, "cuda"), spin.make_config(**wl.config_fields())
    st, buf = spin.LayerState(cfg), spin.StepBuffers(cfg, 1)
    spin.init_state(cfg, st.V, st.D, st.Vmax, st.warm)
    q, w, qp = inp.step_inputs()
    torch.cuda.synchronize()
    want = [x.clone() for x in (st.V, st.D, st.Vmax, st.warm, buf.blocks, buf.n_blocks, buf.topk, buf.scores)]

    def core(max_slots=wl.max_slots, rows=1, pages=inp.n_pages):
        return spin.CoreAttention(spin.make_kv_config(3, max_slots, rows, 16, 2, 64, "bf16"), spin.KvCache(pages, 2, 64),
                                  rows, wl.top_k)

    def step(c, cq, table=inp.block_table):
        spin.run_step(cfg, st, buf, q, w, inp.k_pool[0], inp.k_scale[0], inp.n_pages, table, inp.n_slots, qp, 0, 0,
                      core=c, core_q=cq)

    good = torch.zeros((3, 1, 16, 64), dtype=torch.bfloat16, device="cuda")
    odd = torch.zeros(good.numel() + 1, dtype=torch.bfloat16, device="cuda")[1:].view(good.shape)
    for c, cq in ((core(), None), (core(), good.float()), (core(), good[:2]), (core(), good.cpu()), (core(), odd),
                  (core(rows=2), good.repeat(1, 2, 1, 1)), (core(max_slots=1 << 24), good)):
        with pytest.raises(spin.SpinError):
            step(c, cq)
    torch.cuda.synchronize()
    for x, y in zip((st.V, st.D, st.Vmax, st.warm, buf.blocks, buf.n_blocks, buf.topk, buf.scores), want):
        assert torch.equal(x, y)
    step(core(), good)
    torch.cuda.synchronize()
    assert int(buf.status.item()) == 0 and not torch.equal(buf.topk, want[6])
