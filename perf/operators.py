"""The operators around the paged 8-bit KV cache, as cases to measure.

A cache page holds 64 slots.  Keys and values are e4m3 codes [n_pages][64][kv_heads][dim] with
one fp32 scale per page and head; a block table maps a request's logical blocks to pages, and
`ref` counts the table entries that use a page (0: free).

  attend  attention of a request's query rows over its cached slots, all of them or a listed
          top-K of them (the core attention behind the indexer's top-K)
  append  new keys and values quantised into the cache
  branch  beams re-parented (fork) and given their next page, copying pages still shared
  drain   finished requests' pages freed and the pool compacted

`run` computes them in plain torch, or, where `own` is set, by the library's calls.
"""
import math

import torch

own = False

BLOCK = 64
E4M3 = torch.float8_e4m3fn
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # a first token: one short request in fp32, where latency is all there is
        dict(name="attend_start", op="attend", n_req=1, rows=1, heads=8, kv_heads=8, dim=64, dtype="f32",
             lo=37, hi=37, top_k=0),
        # a decode batch of mixed contexts with grouped heads
        dict(name="attend_batch", op="attend", n_req=64, rows=1, heads=32, kv_heads=8, dim=128, dtype="bf16",
             lo=100, hi=8192, top_k=0),
        # one long context (131072 slots): all of the GPU on a single request
        dict(name="attend_long", op="attend", n_req=1, rows=1, heads=64, kv_heads=8, dim=128, dtype="bf16",
             lo=131072, hi=131072, top_k=0),
        # dense attention with one key/value head shared by 64 query heads, the largest case
        dict(name="attend_shared", op="attend", n_req=32, rows=1, heads=64, kv_heads=1, dim=128, dtype="bf16",
             lo=100000, hi=131072, top_k=0),
        # sparse decode at serving size: 96 requests attend to the 512 slots their indexer picked
        dict(name="attend_topk", op="attend", n_req=96, rows=1, heads=64, kv_heads=1, dim=128, dtype="bf16",
             lo=131072, hi=131072, top_k=512),
        # speculative verification: four rows per request, each seeing one slot more than the last
        dict(name="attend_verify", op="attend", n_req=16, rows=4, heads=64, kv_heads=8, dim=128, dtype="f16",
             lo=4096, hi=32768, top_k=0),
        # one decoded token per request written to the cache
        dict(name="append_token", op="append", n_req=96, kv_heads=8, dim=128, dtype="bf16", lo=1, hi=1, before=5000),
        # ragged prompts written to the cache, some behind a cached prefix that ends inside a page
        dict(name="append_prompt", op="append", n_req=8, kv_heads=8, dim=128, dtype="bf16", lo=1000, hi=16384,
             before=100),
        # a small beam search step
        dict(name="branch_small", op="branch", n_req=8, group=4, kv_heads=1, dim=128, lo=300, hi=2000),
        # a large beam search step: 256 beams, a pool of 2.3 GB
        dict(name="branch_beams", op="branch", n_req=256, group=4, kv_heads=8, dim=128, lo=2000, hi=8192),
        # a few finished requests leave a small pool
        dict(name="drain_small", op="drain", n_req=12, kv_heads=1, dim=64, lo=200, hi=3000),
        # half of a serving batch finishes and a pool of 1.6 GB is made dense again
        dict(name="drain_pool", op="drain", n_req=96, kv_heads=8, dim=128, lo=2000, hi=24000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "branch", "drain"])
    if op == "attend":
        heads, kv_heads = rng.choice([(8, 8), (32, 8), (64, 8), (40, 8), (16, 2), (28, 4), (64, 1), (16, 1), (5, 5)])
        dim = rng.choice([64, 80, 96, 112, 128, 128, 192, 256])
        n_req, rows = _log(rng, 1, 128), rng.choice([1, 1, 1, 2, 3, 4, 8])
        # in slots, so that cache bytes, the head count and the rows stay below the largest case
        most = min(131072, 32 * 116000 * 64 // (n_req * max(heads * rows, 4 * kv_heads) * max(1, dim // 64)))
        hi = _log(rng, 1, most)
        lo = _log(rng, max(1, hi // 50), hi)
        top_k = rng.choice([0, 0, min(_log(rng, 64, 2048), 1 + (1 << 29) // (n_req * rows * kv_heads * dim))])
        return dict(op=op, n_req=n_req, rows=rows, heads=heads, kv_heads=kv_heads, dim=dim,
                    dtype=rng.choice(["f32", "bf16", "bf16", "f16"]), lo=lo, hi=hi, top_k=top_k)
    if op == "append":
        n_req = _log(rng, 1, 128)
        hi = _log(rng, 1, max(1, 40000 // n_req))
        return dict(op=op, n_req=n_req, kv_heads=rng.choice([1, 2, 4, 8]), dim=rng.choice([64, 80, 128, 256]),
                    dtype=rng.choice(["f32", "bf16", "f16"]), lo=_log(rng, max(1, hi // 20), hi), hi=hi,
                    before=_log(rng, 1, 10000))
    hi = _log(rng, 64, 10000)
    case = dict(op=op, n_req=_log(rng, 2, 96), kv_heads=rng.choice([1, 2, 8]), dim=rng.choice([64, 80, 128]),
                lo=_log(rng, max(1, hi // 10), hi), hi=hi)
    if op == "branch":
        case["group"] = rng.choice([1, 2, 3, 4, 8])
    return case


def _lens(case):
    """The requests' lengths: spread over [lo, hi] by their logarithm, in a mixed order."""
    n, lo, hi = case["n_req"], case["lo"], case["hi"]
    step = next(s for s in (7, 11, 13, 17, 19) if n % s)
    return [int(lo * (hi / lo) ** ((i * step % n) / max(1, n - 1))) for i in range(n)]


def _before(case):
    """Slots already cached by the requests that append: up to `before`, one of them none."""
    return [case["before"] * i // max(1, case["n_req"] - 1) if case["n_req"] > 1 else case["before"]
            for i in range(case["n_req"])]


def _pages(n):
    return -(-n // BLOCK)


def _size(dtype):
    return 4 if dtype == "f32" else 2


def work(case):
    lens = _lens(case)
    op = case["op"]
    if op == "attend":
        rows, K, kvh, d, h = case["rows"], case["top_k"], case["kv_heads"], case["dim"], case["heads"]
        per_row = sum(min(n, K) if K else n for n in lens)
        # a dense request's rows share its slots; a list is read per row, at most the whole context
        slots = sum(min(n, K * rows) for n in lens) if K else per_row
        qo = 2 * case["n_req"] * rows * h * d * _size(case["dtype"])
        scales = 8 * kvh * (slots if K else sum(map(_pages, lens)))
        lists = 4 * case["n_req"] * rows * K
        return {"bytes": 2 * slots * kvh * d + qo + scales + lists, "flops": 4 * per_row * rows * h * d}
    if op == "append":
        n = sum(lens) * case["kv_heads"] * case["dim"]
        return {"bytes": 2 * n * (_size(case["dtype"]) + 1), "flops": 4 * n}
    page = 2 * BLOCK * case["kv_heads"] * case["dim"] + 8 * case["kv_heads"]
    if op == "branch":
        parents = lens[:: case["group"]]
        width = _pages(max(lens) + 1)
        n_pages = _branch_pages(case)
        children = [min(case["group"], case["n_req"] - i * case["group"]) for i in range(len(parents))]
        copies = sum(c for p, c in zip(parents, children) if p % BLOCK and c > 1)
        reads = sum(1 for p, c in zip(parents, children) if p % BLOCK and c > 1)
        return {"bytes": 8 * case["n_req"] * width + 8 * n_pages + page * (copies + reads), "flops": 0}
    gone = [i % 2 == 0 for i in range(case["n_req"])]
    counts = [_pages(n) for n in lens]
    live, total = sum(c for c, g in zip(counts, gone) if not g), sum(counts)
    moved = live * (total - live) // total   # expected number of live pages above the live count
    return {"bytes": 8 * case["n_req"] * max(counts) + 8 * total + 2 * page * moved, "flops": 0}


def _branch_pages(case):
    # the old beams' pages and a fresh one for each beam
    return sum(map(_pages, _lens(case))) + case["n_req"]


# ----------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _codes(g, n_pages, kv_heads, dim):
    """e4m3 codes of normal values that use most of a page's range."""
    x = torch.randn((n_pages, BLOCK, kv_heads, dim), generator=g, device="cuda", dtype=torch.bfloat16)
    return x.mul_(100.0).clamp_(-448.0, 448.0).to(E4M3).view(torch.uint8)


def _scales(g, n_pages, kv_heads, spread):
    """Scales that give unit values up to a factor of about exp(spread) a page."""
    x = torch.randn((n_pages, kv_heads), generator=g, device="cuda")
    return torch.exp(spread * x) * 0.01


def _pow2(e):
    """2^e in fp32 for whole numbers e >= -126, by its exponent bits."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _table(g, counts, width, n_pages):
    """A block table over a shuffled pool: request r owns counts[r] pages; the rest is -1."""
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    c = torch.tensor(counts, device="cuda")
    j = torch.arange(width, device="cuda")[None, :]
    at = (torch.cumsum(c, 0) - c)[:, None] + j
    return torch.where(j < c[:, None], order[at.clamp(max=n_pages - 1)], torch.full_like(at, -1, dtype=torch.int32))


def prepare(case, seed):
    g = _gen(seed)
    lens = _lens(case)
    R, kvh, d = case["n_req"], case["kv_heads"], case["dim"]
    s = {"case": dict(case)}
    if case["op"] == "attend":
        rows, K = case["rows"], case["top_k"]
        counts = [_pages(n) for n in lens]
        n_pages = sum(counts)
        s["table"] = _table(g, counts, max(counts), n_pages)
        # row r of a verification sees r slots more than row 0; the last row sees all of them
        n = torch.tensor(lens, device="cuda", dtype=torch.int32)[:, None]
        s["n_slots"] = (n - torch.arange(rows - 1, -1, -1, device="cuda", dtype=torch.int32)).clamp(min=0)
        s["q"] = torch.randn((R, rows, case["heads"], d), generator=g, device="cuda").to(TYPES[case["dtype"]])
        if K:
            # K slots of each row's context, ascending, as the indexer's top-K leaves them
            m = s["n_slots"].long()[..., None]
            u = torch.rand((R, rows, K), generator=g, device="cuda", dtype=torch.float64)
            lo = torch.arange(K, device="cuda") * m // K
            hi = (torch.arange(K, device="cuda") + 1) * m // K
            pick = lo + (u * (hi - lo)).long()
            short = torch.arange(K, device="cuda").expand(R, rows, K)
            pick = torch.where(m >= K, pick, torch.where(short < m, short, torch.full_like(short, -1)))
            s["list"] = pick.to(torch.int32).contiguous()
    elif case["op"] == "append":
        before = _before(case)
        counts = [_pages(b + n) for b, n in zip(before, lens)]
        n_pages = sum(counts)
        s["table"] = _table(g, counts, max(counts), n_pages)
        s["before"] = torch.tensor(before, device="cuda", dtype=torch.int32)
        start = [0]
        for n in lens:
            start.append(start[-1] + n)
        s["start"] = torch.tensor(start, device="cuda", dtype=torch.int32)
        s["max_new"] = max(lens)
        shape = (start[-1], kvh, d)
        # activations: a few large channels and tokens of different size
        size = torch.exp(torch.randn((start[-1], kvh, 1), generator=g, device="cuda"))
        for name in ("new_k", "new_v"):
            s[name] = (torch.randn(shape, generator=g, device="cuda") * size).to(TYPES[case["dtype"]])
    elif case["op"] == "branch":
        # beams in groups that descend from one parent each: beam r continues its group's first
        group = case["group"]
        parent = torch.arange(R, device="cuda") // group * group
        n_pages = _branch_pages(case)
        width = _pages(max(lens) + 1)
        s["table"] = _table(g, [_pages(n) for n in lens], width, n_pages)
        s["parent"] = parent.to(torch.int32)
        s["n_slots"] = torch.tensor(lens, device="cuda", dtype=torch.int32)[parent].contiguous()
        s["n_new"] = torch.ones((R,), device="cuda", dtype=torch.int32)
    else:
        counts = [_pages(n) for n in lens]
        n_pages = sum(counts)
        s["table"] = _table(g, counts, max(counts), n_pages)
        # every other request has finished: it keeps no slots; the others keep what they have
        s["keep"] = torch.tensor([0 if i % 2 == 0 else -1 for i in range(R)], device="cuda", dtype=torch.int32)
    if case["op"] in ("branch", "drain"):
        used = s["table"][s["table"] >= 0].long()
        ref = torch.bincount(used, minlength=n_pages).to(torch.int32)
        # the state that a pass starts from, in one buffer; a pass works on a copy of it
        n = s["table"].numel()
        at = -(-n // 64) * 64
        s["meta0"] = torch.zeros((at + n_pages,), dtype=torch.int32, device="cuda")
        s["meta0"][:n], s["meta0"][at:] = s["table"].view(-1), ref
        s["meta"] = s["meta0"].clone()
        for x in ("", "0"):
            s["table" + x], s["ref" + x] = s["meta" + x][:n].view(s["table"].shape), s["meta" + x][at:]
    s["k"], s["v"] = _codes(g, n_pages, kvh, d), _codes(g, n_pages, kvh, d)
    s["k_scale"], s["v_scale"] = _scales(g, n_pages, kvh, 0.3), _scales(g, n_pages, kvh, 0.3)
    if case["op"] == "append":  # an appending program's scales are powers of two, as it left them
        s["k_scale"], s["v_scale"] = (_pow2(torch.round(torch.log2(x))) for x in (s["k_scale"], s["v_scale"]))
    s["n_pages"] = n_pages
    return s


# -------------------------------------------------------------------------------- plain forms

def _attend(s):
    c = s["case"]
    R, rows, H, kvh, d = c["n_req"], c["rows"], c["heads"], c["kv_heads"], c["dim"]
    n = s["n_slots"].long()                                       # [R][rows]
    q = s["q"].float().view(R, rows, kvh, H // kvh, d) * (1.0 / math.sqrt(d))
    if c["top_k"]:
        i = s["list"].long()                                      # [R][rows][K]
        live = (i >= 0) & (i < n[..., None])
        i = torch.where(live, i, torch.zeros_like(i))
        page = torch.gather(s["table"].long(), 1, (i // BLOCK).view(R, -1)).view(i.shape)
        at = page * BLOCK + i % BLOCK
    else:
        i = torch.arange(max(_lens(c)), device="cuda")
        live = i < n[..., None]                                   # [R][rows][N]
        page = s["table"].long()[:, i // BLOCK].clamp(min=0)[:, None]
        at = page * BLOCK + i % BLOCK                             # [R][1][N]: shared by the rows

    def values(codes, scale):
        x = codes.view(E4M3).view(-1, kvh, d)
        x = x.view(torch.uint8)[at.reshape(-1)].view(E4M3).float().view(*at.shape, kvh, d)
        return x.mul_(scale[page][..., None])

    k = values(s["k"], s["k_scale"])
    if c["top_k"]:
        z = torch.einsum("brhgd,brnhd->brhgn", q, k)
    else:
        z = torch.einsum("brhgd,bnhd->brhgn", q, k[:, 0])
    del k
    z = z.masked_fill_(~live[:, :, None, None, :], -math.inf)
    m = z.amax(-1, keepdim=True)
    m0 = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(z.sub_(m0))
    total = p.sum(-1, keepdim=True)
    v = values(s["v"], s["v_scale"])
    if c["top_k"]:
        o = torch.einsum("brhgn,brnhd->brhgd", p, v)
    else:
        o = torch.einsum("brhgn,bnhd->brhgd", p, v[:, 0])
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (m0 + torch.log(total)).squeeze(-1)
    return {"out": o.view(R, rows, H, d).to(s["q"].dtype), "lse": lse.view(R, rows, H)}


def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s (448 = 0.875 * 2^9); 0 for amax = 0."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)
    return torch.where(amax > 0, _pow2(e), torch.zeros_like(amax))


def _append_pool(s, x, pool, scale):
    T, R = x.shape[0], s["case"]["n_req"]
    before, start, table = s["before"].long(), s["start"].long(), s["table"].long()
    t = torch.arange(T, device="cuda")
    r = torch.searchsorted(start, t, right=True) - 1
    slot = before[r] + t - start[r]
    page = table[r, slot // BLOCK]
    x = x.float()
    amax = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(-1)
    top = torch.zeros_like(scale).index_reduce_(0, page, amax, "amax")
    # the page a request's first new slot falls in keeps its scale, and its earlier slots, if it has any
    first = table[torch.arange(R, device="cuda"), before // BLOCK]
    n_old = before % BLOCK
    is_new = start[1:] > start[:-1]
    kept = torch.zeros_like(scale)
    kept[first] = torch.where(((n_old > 0) & is_new)[:, None], scale[first], torch.zeros_like(scale[first]))
    new = torch.maximum(kept, _pow2_scale(top))
    # the earlier slots of those pages move to the new scale
    old = pool[first].view(E4M3).float()
    ratio = torch.where(new[first] > 0, kept[first] / new[first], torch.zeros_like(new[first]))
    moved = (old * ratio[:, None, :, None]).to(E4M3).view(torch.uint8)
    keep = (torch.arange(BLOCK, device="cuda") < n_old[:, None])[:, :, None, None] & is_new[:, None, None, None]
    pool[first] = torch.where(keep, moved, pool[first])
    touched = torch.zeros_like(scale[:, 0], dtype=torch.bool)
    touched[page] = True
    scale.copy_(torch.where(touched[:, None], new, scale))
    inv = torch.where(new > 0, 1.0 / new, torch.zeros_like(new))[page][..., None]
    pool.view(-1, *pool.shape[2:])[page * BLOCK + slot % BLOCK] = \
        (x * inv).clamp(-448.0, 448.0).to(E4M3).view(torch.uint8)


def _append(s):
    _append_pool(s, s["new_k"], s["k"], s["k_scale"])
    _append_pool(s, s["new_v"], s["v"], s["v_scale"])
    return _append_out(s)


def _append_out(s):
    return {"k": s["k"].view(E4M3), "v": s["v"].view(E4M3), "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _uses(table, n_pages):
    return torch.bincount(table[table >= 0].long(), minlength=n_pages).to(torch.int32)


def _pools(s):
    return s["k"], s["v"], s["k_scale"], s["v_scale"]


def _pools_out(s):
    """The pools as what a page move sees of them: bytes, and the scales' bits."""
    return {"k": s["k"], "v": s["v"], "k_scale": s["k_scale"].view(torch.int32),
            "v_scale": s["v_scale"].view(torch.int32)}


def _branch(s):
    n_pages, old, parent = s["n_pages"], s["table0"], s["parent"].long()
    # fork
    table = torch.where(parent[:, None] >= 0, old[parent.clamp(min=0)], torch.full_like(old, -1))
    ref = s["ref0"] + _uses(table, n_pages) - _uses(old, n_pages)
    # reserve
    n, new = s["n_slots"].long(), s["n_new"].long()
    j = torch.arange(table.shape[1], device="cuda")[None, :]
    first = n // BLOCK
    inside = (j >= first[:, None]) & (j < ((n + new + BLOCK - 1) // BLOCK)[:, None]) & (new > 0)[:, None]
    shared = (table >= 0) & (ref[table.clamp(min=0).long()] > 1)
    need = inside & ((table < 0) | shared)
    count = need.sum(1)
    free = ref == 0
    granted = (count == 0) | (torch.cumsum(count, 0) <= free.sum())
    need &= granted[:, None]
    rank = torch.cumsum(need.view(-1), 0).view_as(need) - 1
    lowest = torch.argsort((~free).to(torch.uint8), stable=True)
    fresh = lowest[rank.clamp(min=0, max=n_pages - 1)]
    copied = need & shared & (j == first[:, None]) & (n % BLOCK > 0)[:, None]
    src, dst = table[copied].long(), fresh[copied]
    [p.index_copy_(0, dst, p[src]) for p in _pools(s)]
    ref = ref - _uses(torch.where(need, table, torch.full_like(table, -1)), n_pages)
    ref[fresh[need]] = 1
    table = torch.where(need, fresh.to(torch.int32), table)
    return {"table": table, "ref": ref, "granted": granted.to(torch.int32), **_pools_out(s)}


def _drain(s):
    n_pages, table = s["n_pages"], s["table0"]
    # free
    kept = (s["keep"].long() + BLOCK - 1) // BLOCK
    j = torch.arange(table.shape[1], device="cuda")[None, :]
    drop = (s["keep"] >= 0)[:, None] & (j >= kept[:, None])
    ref = s["ref0"] - _uses(torch.where(drop, table, torch.full_like(table, -1)), n_pages)
    table = torch.where(drop, torch.full_like(table, -1), table)
    # compact
    live = ref > 0
    n_live = live.sum()
    page = torch.arange(n_pages, device="cuda")
    src = page[live & (page >= n_live)]
    dst = page[~live & (page < n_live)]
    [p.index_copy_(0, dst, p[src]) for p in _pools(s)]
    ref[dst] = ref[src]
    ref[src] = 0
    to = page.to(torch.int32)
    to[src] = dst.to(torch.int32)
    table = torch.where(table >= 0, to[table.clamp(min=0).long()], table)
    return {"table": table, "ref": ref, "n_live": n_live.to(torch.int32).view(1), **_pools_out(s)}


# -------------------------------------------------------------------------- the library's calls

def _handles(s):
    """What a program keeps between calls: the configuration, outputs, workspace and status word."""
    from sparse_attention_indexer_spin_gb300 import spin
    c, h = s["case"], {"spin": spin}
    R, kvh, d = c["n_req"], c["kv_heads"], c["dim"]
    h["status"] = torch.zeros((1,), dtype=torch.int32, device="cuda")
    if c["op"] == "attend":
        h["cfg"] = spin.make_kv_config(n_req=R, max_slots=max(_lens(c)), max_rows=c["rows"], n_heads=c["heads"],
                                       kv_heads=kvh, head_dim=d, dtype=c["dtype"])
        h["out"] = torch.empty_like(s["q"])
        h["lse"] = torch.empty((R, c["rows"], c["heads"]), dtype=torch.float32, device="cuda")
        h["workspace"] = spin.kv_workspace(h["cfg"], c["rows"], c["top_k"])
    elif c["op"] == "append":
        h["cfg"] = spin.make_kv_config(n_req=R, max_slots=s["table"].shape[1] * BLOCK, max_rows=1, n_heads=kvh,
                                       kv_heads=kvh, head_dim=d, dtype=c["dtype"])
    else:
        h["pools"] = spin.PagePools(*_pools(s))
        h["table"] = torch.empty_like(s["table"])
        h["workspace"] = spin.pages_workspace(R, s["n_pages"])
        h["count"] = torch.zeros((R if c["op"] == "branch" else 1,), dtype=torch.int32, device="cuda")
    return h


def _run_own(s):
    if "own" not in s:
        s["own"] = _handles(s)
    h, c = s["own"], s["case"]
    spin = h["spin"]
    if c["op"] == "attend":
        spin.kv_attend(h["cfg"], s["q"], s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"], s["n_slots"],
                       c["rows"], s.get("list"), h["out"], h["lse"], h["workspace"], h["status"])
        return {"out": h["out"], "lse": h["lse"]}
    if c["op"] == "append":
        spin.kv_append(h["cfg"], s["new_k"], s["new_v"], s["start"], s["max_new"], s["before"], s["k"], s["v"],
                       s["k_scale"], s["v_scale"], s["table"], h["status"])
        return _append_out(s)
    if c["op"] == "branch":
        s["ref"].copy_(s["ref0"])
        spin.pages_fork(s["table0"], s["parent"], h["table"], s["ref"], h["status"])
        spin.pages_reserve(h["table"], s["n_slots"], s["n_new"], s["ref"], h["pools"], h["count"], h["workspace"],
                           h["status"])
        return {"table": h["table"], "ref": s["ref"], "granted": h["count"], **_pools_out(s)}
    s["meta"].copy_(s["meta0"])
    spin.pages_free(s["table"], s["keep"], s["ref"], h["status"])
    spin.pages_compact(s["table"], s["ref"], h["pools"], h["count"], h["workspace"], h["status"])
    return {"table": s["table"], "ref": s["ref"], "n_live": h["count"], **_pools_out(s)}


def run(state):
    if own:
        return _run_own(state)
    return {"attend": _attend, "append": _append, "branch": _branch, "drain": _drain}[state["case"]["op"]](state)


# ------------------------------------------------------------------------- 64-bit definitions

def exact(case, seed):
    if case["op"] in ("branch", "drain"):
        return None
    s = prepare(case, seed)
    return _exact_attend(case, s) if case["op"] == "attend" else _exact_append(case, s)


def _exact_attend(case, s):
    """Request by request: its slots in order, softmax by its definition in 64 bits."""
    H, kvh, d = case["heads"], case["kv_heads"], case["dim"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(out.shape[:-1], -math.inf, dtype=torch.float64, device="cuda")
    for b in range(case["n_req"]):
        pages = s["table"][b].long()
        for r in range(case["rows"]):
            n = int(s["n_slots"][b, r])
            if case["top_k"]:
                i = s["list"][b, r].long()
                i = i[(i >= 0) & (i < n)]
            else:
                i = torch.arange(n, device="cuda")
            if i.numel() == 0:
                continue
            p, at = pages[i // BLOCK], i % BLOCK
            for h in range(kvh):
                k, v = (s[x][:, :, h][p, at].view(E4M3).double() * s[x + "_scale"][p, h].double()[:, None]
                        for x in ("k", "v"))
                of = slice(h * (H // kvh), (h + 1) * (H // kvh))
                z = s["q"][b, r, of].double() @ k.T / math.sqrt(d)
                lse[b, r, of] = torch.logsumexp(z, -1)
                out[b, r, of] = torch.softmax(z, -1) @ v
    return {"out": out, "lse": lse}


def _exact_append(case, s):
    """Request by request and page by page; the codes' places hold the quotients, not rounded."""
    out = {}
    for name in ("k", "v"):
        x, pool, scale = s["new_" + name], s[name].view(E4M3).double(), s[name + "_scale"].double()
        start, before = s["start"].tolist(), s["before"].tolist()
        table = s["table"].tolist()
        for r in range(case["n_req"]):
            t = start[r]
            while t < start[r + 1]:
                slot = before[r] + t - start[r]
                at, page = slot % BLOCK, table[r][slot // BLOCK]
                m = min(BLOCK - at, start[r + 1] - t)
                new = x[t:t + m].double()
                top = new.abs().amax((0, 2))
                # a power of two at or below the wanted one, doubled while it is too small
                want = ((torch.log2(top / 448.0).round().long().clamp(min=-125) + 1022) << 52).view(torch.float64)
                for _ in range(2):
                    want = torch.where(448.0 * want < top, 2.0 * want, want)
                want = torch.where(top > 0, want, torch.zeros_like(top))
                had = scale[page] if at else torch.zeros_like(top)
                got = torch.maximum(had, want)
                div = torch.where(got > 0, got, torch.ones_like(got))
                pool[page, :at] *= (had / div)[:, None]
                pool[page, at:at + m] = new / div[:, None]
                scale[page] = got
                t += m
        out[name], out[name + "_scale"] = pool, scale
    return out
