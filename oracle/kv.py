"""Plain 64-bit restatement of the KV cache's operators (test infrastructure only).

numpy, request by request, from the definitions in include/spin.h; shares nothing with the
library.  Codes are uint8 e4m3, decoded from their bits here.
"""
import numpy as np

BLOCK = 64


def _e4m3_table():
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


E4M3 = _e4m3_table()
_POS = E4M3[:127]                      # 0 .. 448, ascending by code


def e4m3_encode(x):
    """Round to nearest, ties to the even code, saturating; NaN -> 0x7f."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    a = np.where(np.isnan(a), 0.0, a)
    hi = np.clip(np.searchsorted(_POS, a), 1, 126)
    lo = hi - 1
    dl, dh = a - _POS[lo], _POS[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    code = code | np.where(np.signbit(x), 128, 0)
    return np.where(np.isnan(x), 127, code).astype(np.uint8)


def attend(q, k, v, k_scale, v_scale, table, n_slots, scale, listed=None):
    """q [R][rows][H][d] float64.  Returns out, lse and the bounds' ingredients per (b, row, h):
    A = sum w |v| per dim, S = max |scale ks| sum |q||k|, top = max w |vs|, n = set size."""
    R, rows, H, d = q.shape
    kvh = k.shape[2]
    out, A = np.zeros(q.shape), np.zeros(q.shape)
    lse = np.full(q.shape[:3], -np.inf)
    S, top, smax = np.zeros(q.shape[:3]), np.zeros(q.shape[:3]), np.zeros(q.shape[:3])
    cnt = np.zeros(q.shape[:3])
    n_pages = k.shape[0]
    for b in range(R):
        for r in range(rows):
            n = int(n_slots[b, r])
            i = np.arange(max(n, 0)) if listed is None else listed[b, r]
            i = i[(i >= 0) & (i < n)].astype(np.int64)
            p = table[b, i // BLOCK] if i.size else np.zeros(0, np.int64)
            ok = (p >= 0) & (p < n_pages)
            i, p = i[ok], p[ok]
            if i.size == 0:
                continue
            for g in range(kvh):
                kc = E4M3[k[p, i % BLOCK, g]]
                vv = E4M3[v[p, i % BLOCK, g]] * v_scale[p, g].astype(np.float64)[:, None]
                ks = k_scale[p, g].astype(np.float64)
                for h in range(g * (H // kvh), (g + 1) * (H // kvh)):
                    s = scale * ks * (kc @ q[b, r, h])
                    m = s.max()
                    e = np.exp(s - m)
                    w = e / e.sum()
                    out[b, r, h], lse[b, r, h] = w @ vv, m + np.log(e.sum())
                    A[b, r, h] = w @ np.abs(vv)
                    S[b, r, h] = (np.abs(scale * ks) * (np.abs(kc) @ np.abs(q[b, r, h]))).max()
                    smax[b, r, h] = np.abs(s).max()
                    top[b, r, h] = (w * np.abs(v_scale[p, g])).max()
                    cnt[b, r, h] = i.size
    return out, lse, dict(A=A, S=S, smax=smax, top=top, n=cnt)


def pow2_scale(amax):
    """The smallest power of two s >= 2^-126 with amax <= 448 s; 0 for amax = 0."""
    if amax == 0:
        return 0.0
    s = 2.0 ** -126
    while 448.0 * s < amax:
        s *= 2.0
    return s


def append(x, start, before, pool, scale, table):
    """New values x [T][kvh][d] (float64 of the given values) into pool / scale, in place."""
    f32 = np.float32
    for r in range(len(before)):
        t = int(start[r])
        while t < start[r + 1]:
            slot = int(before[r]) + t - int(start[r])
            at, page = slot % BLOCK, int(table[r, slot // BLOCK])
            m = min(BLOCK - at, int(start[r + 1]) - t)
            for h in range(x.shape[1]):
                new = x[t:t + m, h]
                fin = np.abs(new[np.isfinite(new)])
                old = float(scale[page, h]) if at else 0.0
                s = max(old, pow2_scale(fin.max() if fin.size else 0.0))
                if s != old and at:
                    ratio = f32(old) / f32(s) if s >= 2.0 ** -126 else f32(0)
                    c = E4M3[pool[page, :at, h]].astype(f32) * ratio
                    pool[page, :at, h] = e4m3_encode(c)
                inv = f32(1) / f32(s) if s >= 2.0 ** -126 else f32(0)
                with np.errstate(invalid="ignore", over="ignore"):
                    quotient = new.astype(f32) * inv
                # an infinity stays one, whatever the scale, and saturates
                pool[page, at:at + m, h] = e4m3_encode(np.where(np.isinf(new), new, quotient))
                scale[page, h] = s
            t += m


def fork(table, parent, ref):
    out = np.full_like(table, -1)
    for r, p in enumerate(parent):
        if p >= 0:
            out[r] = table[p]
    ref = ref.copy()
    for page in out[out >= 0]:
        ref[page] += 1
    for page in table[table >= 0]:
        ref[page] -= 1
    return out, ref


def free(table, keep, ref):
    table, ref = table.copy(), ref.copy()
    for r, k in enumerate(keep):
        if k < 0:
            continue
        for j in range(-(-int(k) // BLOCK), table.shape[1]):
            if table[r, j] >= 0:
                ref[table[r, j]] -= 1
            table[r, j] = -1
    return table, ref


def reserve(table, n_slots, n_new, ref, pools):
    """Returns table, ref, granted; pools are changed in place."""
    table, start = table.copy(), ref.copy()
    ref = ref.copy()
    fresh = [p for p in range(len(ref)) if start[p] <= 0]
    granted = np.ones(len(n_slots), np.int32)
    used = 0
    full = False
    for r in range(len(n_slots)):
        n, add = int(n_slots[r]), int(n_new[r])
        if add == 0:
            continue
        want = [j for j in range(n // BLOCK, -(-(n + add) // BLOCK))
                if table[r, j] < 0 or start[table[r, j]] > 1]
        if not want:
            continue
        if full or used + len(want) > len(fresh):
            full = True
            granted[r] = 0
            continue
        for j in want:
            old, page = table[r, j], fresh[used]
            used += 1
            ref[page] = 1
            table[r, j] = page
            if old >= 0:
                ref[old] -= 1
                if j == n // BLOCK and n % BLOCK:
                    for p in pools:
                        p[page] = p[old]
    return table, ref, granted


def compact(table, ref, pools):
    """Returns table, ref, number of used pages; pools are changed in place."""
    table, ref = table.copy(), ref.copy()
    used = np.flatnonzero(ref > 0)
    n = len(used)
    src = [p for p in used if p >= n]
    dst = [p for p in range(n) if ref[p] <= 0]
    to = {}
    for a, b in zip(src, dst):
        to[a] = b
        ref[b], ref[a] = ref[a], 0
        for p in pools:
            p[b] = p[a]
    for i in np.ndindex(*table.shape):
        table[i] = to.get(table[i], table[i])
    return table, ref, n
