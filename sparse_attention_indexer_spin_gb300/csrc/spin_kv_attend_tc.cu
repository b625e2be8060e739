// spin_kv_attend_tc.cu -- attention over the paged 8-bit KV cache on tcgen05 tensor cores, for many
// query rows per key/value head (sm_103a).
//
// Same mathematics and numbers as spin_kv_attend.cu, in tiles of 128 query rows x 128 slots:
//   S = Q K^T     A = Q f16 in TMEM (rows in lanes), B = K f16 in shared memory (slots x dims)
//   O += P V      A = P f16 in TMEM,                 B = V f16 in shared memory (slots x dims, N contiguous)
// with fp32 accumulators in TMEM.  With fewer than 128 rows the products' other rows are wasted,
// but a tile's 16 MMAs (64 cycles each) still take less than fetching its 32 KB from HBM; what the
// kernel must keep low is the work per byte of the other pipes:
//   * a code is turned into f16 once for all the rows, and crosses shared memory twice (the store,
//     the MMA's read); the codes come straight from global memory to registers;
//   * the softmax has a row per thread: no shuffles, no shared-memory operands, packed weights
//     written back over the scores in TMEM.
//
// Warps of a CTA (one CTA an SM):
//   0-7    softmax: warp w reads TMEM lanes 32 (w mod 4) .. (a row a thread), columns 64 (w / 4) ..:
//          one page of the tile.  Lane quarters without query rows leave at once.
//   8      issues the MMAs: S of tile n + 1 goes in before P V of tile n
//   9-12   keys, 13-16 values: load a tile's codes two tiles ahead, convert, store in the 128-byte
//          swizzled layout the MMAs read
//   17     scout: walks the segments and looks up lists, pages and scales, a ring of tiles ahead
// A row's reference moves rarely (see kAtSlack); then its two threads agree on the new one through
// shared memory and rescale O in TMEM, after the products before it are done.
// Every wait is bounded; a wait that runs out unwinds all roles.
#include "spin_kv_attend.cuh"
#include "spin_tc.cuh"

namespace spin {

constexpr int kXTile = 128;                    // slots of a tile
constexpr int kXSoft = 8, kXConv = 4;          // warps: softmax; each of keys and values
constexpr int kXMma = kXSoft, kXKeys = kXMma + 1, kXValues = kXKeys + kXConv, kXScout = kXValues + kXConv;
constexpr int kXWarps = kXScout + 1, kXThreads = 32 * kXWarps;
constexpr int kXRing = 6;                      // tiles the scout is ahead
constexpr int kXUnit = kXTile;
constexpr int kXJobUnits = 6;                  // a job's start: 3 us beside 0.5 us a tile
constexpr int kXSplitGain = 12;

enum XFlag { kXFirst = 1, kXLast = 2, kXOdd = 4, kXStop = 8 };

struct XEntry {                // a tile as the scout publishes it
    int64_t row[kXTile];       // offset of a slot's codes of this head in either pool, -1: none
    float ks[kXTile], lv[kXTile], iv[kXTile], ratio[kXTile];
    int flags, slot0, v, g, mc, u0, u1, units, len, nmin;
    int pad[6];
};

struct XHdr {
    uint64_t scfull[kXRing], scempty[kXRing];
    uint64_t kfull[2], kempty[2], vfull[2], vempty[2];
    uint64_t sfull[2], pready[2], pvdone, qready, fin;
    uint32_t tmem_base;
    volatile int abort_flag;
    int nan_seen;              // a NaN value among slots that some rows see and others do not
    int64_t scan[kXWarps + 3];
    float top[2][128], l[2][128];
};

template <int D> struct XSmem {
    static constexpr int kStage = kXTile * D * 2;  // one of keys, values: D / 64 blocks of 128 rows x 128 bytes
    static constexpr int kK = 0, kV = 2 * kStage, kRingAt = 4 * kStage;
    static constexpr int kHdr = kRingAt + kXRing * (int)sizeof(XEntry);
    static constexpr int kBytes = kHdr + (int)sizeof(XHdr) + 1024;
};

// TMEM columns
template <int D> struct XTmem {
    static constexpr uint32_t kQ = 0, kS = D / 2, kO = kS + 2 * kXTile;
    static_assert(kO + D <= 512, "fits TMEM");
};

template <typename T> __device__ __forceinline__ void unpack8(const uint4 u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (std::is_same<T, __half>::value) {
            const float2 f = unpack_f16(w[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        } else {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}

template <typename T, int D, bool SPARSE>
__global__ void __launch_bounds__(kXThreads, 1)
kv_attend_tc_kernel(const __grid_constant__ spin_kv_config cfg, const __grid_constant__ KvAttendArgs a, AtPlan plan) {
    pdl_wait();
    using L = XSmem<D>;
    using TM = XTmem<D>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    XEntry* ring = reinterpret_cast<XEntry*>(smem + L::kRingAt);
    XHdr* hdr = reinterpret_cast<XHdr*>(smem + L::kHdr);
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int H = cfg.n_heads, kvh = cfg.kv_heads, d = cfg.head_dim, group = H / kvh;
    const int rows = SPARSE ? 1 : a.rows, M = group * rows;
    const int quarters = (min(plan.crows, M) + 31) / 32;  // TMEM lane quarters with query rows
    const float ninf = __uint_as_float(0xff800000u);

    if (tid == 0) {
        for (int i = 0; i < kXRing; ++i) {
            mbar_init(&hdr->scfull[i], 1);
            mbar_init(&hdr->scempty[i], 2 * kXConv + 2 * quarters + 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&hdr->kfull[i], kXConv);
            mbar_init(&hdr->vfull[i], kXConv);
            mbar_init(&hdr->kempty[i], 1);
            mbar_init(&hdr->vempty[i], 1);
            mbar_init(&hdr->sfull[i], 1);
            mbar_init(&hdr->pready[i], 2 * quarters);
        }
        mbar_init(&hdr->pvdone, 1);
        mbar_init(&hdr->qready, 2 * quarters);
        mbar_init(&hdr->fin, 1);
        hdr->abort_flag = 0;
        hdr->nan_seen = 0;
        fence_barrier_init();
    }
    if (wid == kXMma) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&hdr->tmem_base)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    AtWalk<SPARSE> walk;
    walk.template start<kXWarps>(cfg, a, plan, hdr->scan);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = hdr->tmem_base;

    auto fail_wait = [&]() {
        hdr->abort_flag = 1;
        set_status(a.status, SPIN_STATUS_TIMEOUT);
    };
    // one lane waits for the warp
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        int ok = 1;
        if (lane == 0) {
            ok = mbar_wait(bar, parity, &hdr->abort_flag);
            if (!ok) fail_wait();
        }
        return __shfl_sync(0xffffffffu, ok, 0);
    };

    if (wid == kXScout) {
        // ------------------------------------------------------------------------- scout
        // Four steps a tile, one per turn of the loop, so that the loads of four tiles are in flight:
        // its place in the ring and its list entries, its pages, its scales, the publication.
        int e1[4], e2[4], e3[4], p2[4], p3[4], n = 0, n1 = -1, n2 = -1, n3 = -1;  // nI: tile in step I, -1: none
        float ks3[4], vs3[4];
        AtSegment seg;
        int at = 0, to = 0, nmin = 0;          // units of the current segment
        bool more = true;
        for (;;) {
            n3 = n2;
            n2 = n1;
            n1 = -1;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                e3[i] = e2[i];
                p3[i] = p2[i];
                e2[i] = e1[i];
            }
            if (more && at == to) {
                more = walk.next(cfg, a, plan, seg);
                if (more) {
                    at = seg.u0;
                    to = seg.u1;
                    nmin = 0x7fffffff;
                    if constexpr (SPARSE) {
                        nmin = row_slots(a, seg.v, cfg.max_slots);  // the row's slots bound its entries
                    } else {
                        for (int r = 0; r < rows; ++r) nmin = min(nmin, row_slots(a, (int64_t)seg.v * rows + r, cfg.max_slots));
                    }
                    if (lane == 0) walk.own(plan, seg);
                }
            }
            if (!more && n2 < 0 && n3 < 0) break;
            if (more) {  // step 1
                XEntry* e = ring + n % kXRing;
                if (!warp_wait(&hdr->scempty[n % kXRing], (uint32_t)(n / kXRing & 1) ^ 1u)) break;
                const int slot0 = at * kXTile;
                if (lane == 0) {
                    e->flags = (at == seg.u0 ? kXFirst : 0) | (at + 1 == seg.u1 ? kXLast : 0);
                    e->slot0 = slot0;
                    e->v = seg.v;
                    e->g = seg.g;
                    e->mc = seg.mc;
                    e->u0 = seg.u0;
                    e->u1 = seg.u1;
                    e->units = seg.units;
                    e->len = seg.len;
                    e->nmin = nmin;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = slot0 + 32 * i + lane;
                    e1[i] = -1;
                    if (j < seg.len) {
                        if constexpr (SPARSE) e1[i] = a.list[(int64_t)seg.v * a.top_k + j];
                        else e1[i] = j;
                    }
                }
                n1 = n++;
                ++at;
            }
            __syncwarp();
            if (n2 >= 0) {  // step 2
                const XEntry* e = ring + n2 % kXRing;
                const int32_t* table = a.block_table + (SPARSE ? e->v / a.rows : e->v) * a.bt_stride;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (SPARSE) {
                        if (e2[i] < -1 || e2[i] >= e->nmin) {
                            set_status(a.status, SPIN_STATUS_BAD_LIST);
                            e2[i] = -1;
                        }
                    }
                    p2[i] = e2[i] >= 0 ? table[e2[i] >> 6] : -1;
                }
            }
            if (n3 >= 0) {  // step 3, and 4: the scales' latency is the only one not hidden by another tile's
                XEntry* e = ring + n3 % kXRing;
                const int g = e->g;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (e3[i] >= 0 && (p3[i] < 0 || p3[i] >= a.n_pages)) {
                        set_status(a.status, SPIN_STATUS_BAD_PAGE);
                        p3[i] = -1;
                    }
                    ks3[i] = p3[i] >= 0 ? a.k_scale[(int64_t)p3[i] * kvh + g] : 0.0f;
                    vs3[i] = p3[i] >= 0 ? a.v_scale[(int64_t)p3[i] * kvh + g] : 0.0f;
                }
                bool odd = false;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = 32 * i + lane;
                    const bool live = p3[i] >= 0, fine = in_log_range(vs3[i]);
                    const float lg = scale_log2(vs3[i]);
                    e->row[j] = live ? (((int64_t)p3[i] * kBlock + (e3[i] & 63)) * kvh + g) * d : -1;
                    e->ks[j] = ks3[i];
                    e->lv[j] = live ? lg : ninf;
                    e->iv[j] = !live ? 0.0f : fine ? __frcp_rn(vs3[i]) : ex2(-lg);
                    e->ratio[j] = fine || !live ? 1.0f : vs3[i] * ex2(-lg);
                    odd |= live && !fine;
                }
                odd = __any_sync(0xffffffffu, odd);
                if (lane == 0 && odd) e->flags |= kXOdd;
                __syncwarp();
                if (lane == 0) mbar_arrive(&hdr->scfull[n3 % kXRing]);
            }
        }
        pdl_trigger();
        if (!hdr->abort_flag && warp_wait(&hdr->scempty[n % kXRing], (uint32_t)(n / kXRing & 1) ^ 1u) && lane == 0) {
            ring[n % kXRing].flags = kXStop;
            mbar_arrive(&hdr->scfull[n % kXRing]);
        }
    } else if (wid >= kXKeys) {
        // --------------------------------------------------------------------- converters
        const bool values = wid >= kXValues;
        const int t = tid - 32 * (values ? kXValues : kXKeys);
        constexpr int CH = D / 16, RS = 128 / CH, NP = CH;  // chunks of a row, rows at a time, pieces a thread
        const int prow = t / CH, x = t % CH;
        const uint8_t* pool = (values ? a.v_pool : a.k_pool) + 16 * x;
        const bool in_row = 16 * x < d;
        uint64_t* full = values ? hdr->vfull : hdr->kfull;
        uint64_t* empty = values ? hdr->vempty : hdr->kempty;
        const uint32_t base = smem_u32(smem + (values ? L::kV : L::kK));
        // A piece's 16 codes fill chunks 2x and 2x + 1 of its row's 16-byte chunks of f16; in the second
        // block of 64 dims the two trade places, so that the eight stores of a row hit different banks.
        const int c0 = 2 * (x & 3) + (x >> 2), c1 = 2 * (x & 3) + 1 - (x >> 2), block = x >> 2;

        auto fetch = [&](int n, uint4 (&buf)[NP], int& lim) -> bool {
            XEntry* e = ring + n % kXRing;
            if (!warp_wait(&hdr->scfull[n % kXRing], (uint32_t)(n / kXRing & 1))) return false;
            if (e->flags & kXStop) return false;
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int64_t off = e->row[prow + RS * i];
                buf[i] = off >= 0 && in_row ? *reinterpret_cast<const uint4*>(pool + off) : make_uint4(0, 0, 0, 0);
            }
            lim = !SPARSE && values ? e->nmin - e->slot0 : kXTile;  // rows from here on: seen by some query rows only
            __syncwarp();
            if (lane == 0) mbar_arrive(&hdr->scempty[n % kXRing]);
            return true;
        };
        auto put = [&](int n, uint4 (&buf)[NP], int lim) -> bool {
            if (!warp_wait(&empty[n & 1], (uint32_t)(n >> 1 & 1) ^ 1u)) return false;
            const uint32_t st = base + (uint32_t)((n & 1) * L::kStage) + block * (kXTile * 128);
            if (!SPARSE && lim < kXTile) {
                // a NaN here must not reach the rows that do not see it (0 x NaN): it leaves the tile, and the
                // epilogue looks for the rows that do
                bool nan = false;
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    if (prow + RS * i < lim) continue;
                    uint32_t w[4] = {buf[i].x, buf[i].y, buf[i].z, buf[i].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t m = ((w[k] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;  // bytes that are NaN
                        nan |= m != 0;
                        w[k] &= ~((m >> 7) * 0xffu);
                    }
                    buf[i] = make_uint4(w[0], w[1], w[2], w[3]);
                }
                if (nan) hdr->nan_seen = 1;
            }
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int row = prow + RS * i;
                uint4 u, v;
                codes_to_f16(buf[i].x, u.x, u.y);
                codes_to_f16(buf[i].y, u.z, u.w);
                codes_to_f16(buf[i].z, v.x, v.y);
                codes_to_f16(buf[i].w, v.z, v.w);
                const uint32_t r = st + row * 128;
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(r + ((c0 ^ (row & 7)) << 4)), "r"(u.x), "r"(u.y),
                             "r"(u.z), "r"(u.w)
                             : "memory");
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(r + ((c1 ^ (row & 7)) << 4)), "r"(v.x), "r"(v.y),
                             "r"(v.z), "r"(v.w)
                             : "memory");
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[n & 1]);
            return true;
        };
        uint4 b0[NP], b1[NP];
        int lim0 = 0, lim1 = 0, n = 0;
        bool ok0 = fetch(0, b0, lim0), ok1 = ok0 && fetch(1, b1, lim1);
        while (ok0) {
            if (!put(n, b0, lim0)) break;
            ok0 = ok1 && fetch(n + 2, b0, lim0);
            if (!ok1 || !put(n + 1, b1, lim1)) break;
            ok1 = ok0 && fetch(n + 3, b1, lim1);
            n += 2;
        }
    } else if (wid == kXMma) {
        // ------------------------------------------------------------------------ MMA issue
        if (lane == 0) {
            const uint32_t id_s = idesc_mma(0u, kXTile, 128u), id_o = idesc_mma(0u, (uint32_t)D, 128u) | kIdescBn;
            const uint32_t kbase = smem_u32(smem + L::kK), vbase = smem_u32(smem + L::kV);
            auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
                if (mbar_wait(bar, parity, &hdr->abort_flag)) return true;
                fail_wait();
                return false;
            };
            auto product = [&](int n, bool first) -> bool {  // O (+)= P V of tile n
                if (!wait(&hdr->pready[n & 1], (uint32_t)(n >> 1 & 1)) || !wait(&hdr->vfull[n & 1], (uint32_t)(n >> 1 & 1)))
                    return false;
                tc_fence_after();
                const uint32_t st = vbase + (uint32_t)((n & 1) * L::kStage), p = tmem + TM::kS + (n & 1) * kXTile;
#pragma unroll
                for (int k = 0; k < kXTile / 16; ++k)
                    tc_mma_f16_ta(tmem + TM::kO, p + 8 * k, smem_desc_sw128_n(st + 2048 * k, kXTile * 128), id_o,
                                  !(first && k == 0));
                tc_commit(&hdr->vempty[n & 1]);
                tc_commit(&hdr->pvdone);
                return true;
            };
            int pend = -1, segs = 0;
            bool pend_first = false;
            for (int n = 0;; ++n) {
                if (!wait(&hdr->scfull[n % kXRing], (uint32_t)(n / kXRing & 1))) break;
                const int flags = ring[n % kXRing].flags;
                if (flags & kXStop) break;
                mbar_arrive(&hdr->scempty[n % kXRing]);
                if (flags & kXFirst) {
                    if (!wait(&hdr->qready, (uint32_t)(segs & 1))) break;
                    ++segs;
                }
                if (!wait(&hdr->kfull[n & 1], (uint32_t)(n >> 1 & 1))) break;
                tc_fence_after();
                // the scores' buffer held tile n - 2: its P V was issued, and reads it before this writes
                const uint32_t st = kbase + (uint32_t)((n & 1) * L::kStage);
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    tc_mma_f16_ta(tmem + TM::kS + (n & 1) * kXTile, tmem + TM::kQ + 8 * k,
                                  smem_desc_sw128(st + (k >> 2) * (kXTile * 128) + (k & 3) * 32), id_s, k != 0);
                tc_commit(&hdr->kempty[n & 1]);
                tc_commit(&hdr->sfull[n & 1]);
                if (pend >= 0 && !product(pend, pend_first)) break;
                pend = n;
                pend_first = flags & kXFirst;
                if (flags & kXLast) {
                    if (!product(n, pend_first)) break;
                    pend = -1;
                }
            }
            // never leave with MMAs in flight
            tc_commit(&hdr->fin);
            if (!mbar_wait(&hdr->fin, 0u, nullptr)) set_status(a.status, SPIN_STATUS_TIMEOUT);
        }
        __syncwarp();
    } else if ((wid & 3) < quarters) {
        // --------------------------------------------------------------------------- softmax
        const int qd = wid & 3, set = wid >> 2, m = 32 * qd + lane;  // this thread's row, its half of the columns
        const uint32_t trow = tmem + ((uint32_t)(32 * qd) << 16);
        const int bar_id = 1 + qd;                                   // the two warps of a quarter
        float mx = ninf, lsum = 0.0f, qs = 0.0f;
        int nlim = 0;
        int64_t out_row = 0;
        bool valid = false;
        for (int n = 0;; ++n) {
            const XEntry* e = ring + n % kXRing;
            bool ok = warp_wait(&hdr->scfull[n % kXRing], (uint32_t)(n / kXRing & 1));
            const int flags = ok ? e->flags : 0;
            if (flags & kXStop) break;
            if (ok && (flags & kXFirst)) {
                // ---- a new job: this row's query, scaled by a power of two and rounded to f16, into TMEM
                const int mm = e->mc * plan.crows + m;
                valid = m < plan.crows && mm < M;
                const int64_t br = (int64_t)e->v * rows + (valid ? mm / group : 0);
                out_row = br * H + (int64_t)e->g * group + (valid ? mm % group : 0);
                const uint4* qp = reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(a.q) + out_row * d);
                float amax = 0.0f;
                for (int i = 0; valid && i < d / 8; ++i) {
                    float x[8];
                    unpack8<T>(qp[i], x);
#pragma unroll
                    for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(x[k]));
                }
                const int k2 = max(-112, (int)(__float_as_uint(amax) >> 23) - 127);
                // a negative softmax scale goes into the query: scores then grow with t
                const float f = copysignf(__uint_as_float((uint32_t)(127 + 14 - k2) << 23), cfg.softmax_scale);
                qs = __uint_as_float((uint32_t)max(1, 127 - 14 + k2) << 23) * (fabsf(cfg.softmax_scale) * 1.4426950408889634f);
                nlim = valid && !SPARSE ? row_slots(a, br, cfg.max_slots) : 0x7fffffff;
                constexpr int CV = D / 16;  // vectors of 8 dims in this thread's half
#pragma unroll
                for (int h = 0; h < CV / 4; ++h) {
                    uint32_t w[16];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int chunk = 4 * h + c;
                        // D = 128: neighbouring chunks of the second block trade places, as the codes' do
                        const int i = set * CV + (D == 128 ? chunk ^ set : chunk);
                        float x[8];
                        unpack8<T>(valid && i < d / 8 ? qp[i] : make_uint4(0, 0, 0, 0), x);
#pragma unroll
                        for (int k = 0; k < 4; ++k) w[4 * c + k] = pack_f16(x[2 * k] * f, x[2 * k + 1] * f);
                    }
                    tc_st16(trow + TM::kQ + set * (D / 4) + 16 * h, w);
                }
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&hdr->qready);
                mx = ninf;
                lsum = 0.0f;
            }
            const uint32_t scol = trow + TM::kS + (n & 1) * kXTile;
            float s[64], top = ninf, c = 1.0f, lv = 0.0f;
            const int j0 = 64 * set;
            if (ok) ok = warp_wait(&hdr->sfull[n & 1], (uint32_t)(n >> 1 & 1));
            if (ok) {
                tc_fence_after();
                tc_ld64(scol + j0, s);
                if constexpr (SPARSE) {
                    // per slot: t + log2 vs, -inf where no slot is
#pragma unroll
                    for (int j = 0; j < 64; j += 4) {
                        const float4 k4 = *reinterpret_cast<const float4*>(e->ks + j0 + j);
                        const float4 v4 = *reinterpret_cast<const float4*>(e->lv + j0 + j);
                        s[j] = fmaf(s[j] * k4.x, qs, v4.x);
                        s[j + 1] = fmaf(s[j + 1] * k4.y, qs, v4.y);
                        s[j + 2] = fmaf(s[j + 2] * k4.z, qs, v4.z);
                        s[j + 3] = fmaf(s[j + 3] * k4.w, qs, v4.w);
                    }
                } else {
                    // one page: t + log2 vs = c s + lv
                    c = qs * e->ks[j0];
                    lv = e->lv[j0];
                    const int lim = nlim - (e->slot0 + j0);
                    if (lim < 64 || c < 0.0f) {  // the row ends here, or a negative key scale
#pragma unroll
                        for (int j = 0; j < 64; ++j) s[j] = j < lim ? s[j] * c : ninf;
                        c = 1.0f;
                    }
                }
#pragma unroll
                for (int j = 0; j < 64; ++j) top = fmaxf(top, s[j]);
                top = (SPARSE ? top : fmaf(top, c, lv)) - kAtTop;
                if (top != top) top = ninf;  // 0 x inf
            }
            hdr->top[set][m] = top;
            if (named_barrier_or(bar_id, 64, !ok || top > mx + kAtSlack)) {
                // some row's reference moves, or a wait gave up
                const float other = hdr->top[set ^ 1][m];
                if (ok && !(flags & kXFirst)) {
                    ok = warp_wait(&hdr->pvdone, (uint32_t)(n - 1) & 1u);
                    tc_fence_after();
                }
                if (named_barrier_or(bar_id, 64, !ok)) break;
                const float now = fmaxf(mx, fmaxf(top, other));
                const float f = now == ninf ? 1.0f : ex2(mx - now);
                mx = now;
                lsum *= f;
                if (!(flags & kXFirst)) {
#pragma unroll 1
                    for (int h = 0; h < D / 32; ++h) {
                        float o[16];
                        uint32_t w[16];
                        const uint32_t col = trow + TM::kO + set * (D / 2) + 16 * h;
                        tc_ld16(col, o);
#pragma unroll
                        for (int k = 0; k < 16; ++k) w[k] = __float_as_uint(o[k] * f);
                        tc_st16(col, w);
                    }
                    tc_wait_st();
                }
            }
            // ---- weights: 2^(t + log2 vs - m), written over the scores as f16
            const float bias = (SPARSE ? 0.0f : lv) - (mx == ninf ? 0.0f : mx);
            float add = 0.0f;
#pragma unroll
            for (int j = 0; j < 64; ++j) s[j] = ex2(SPARSE ? s[j] + bias : fmaf(s[j], c, bias));
            if constexpr (SPARSE) {
#pragma unroll
                for (int j = 0; j < 64; j += 4) {
                    const float4 i4 = *reinterpret_cast<const float4*>(e->iv + j0 + j);
                    add = fmaf(s[j], i4.x, add);
                    add = fmaf(s[j + 1], i4.y, add);
                    add = fmaf(s[j + 2], i4.z, add);
                    add = fmaf(s[j + 3], i4.w, add);
                }
                lsum += add;
            } else {
#pragma unroll
                for (int j = 0; j < 64; ++j) add += s[j];
                lsum = fmaf(add, e->iv[j0], lsum);
            }
            if (flags & kXOdd) {
#pragma unroll
                for (int j = 0; j < 64; ++j) s[j] *= e->ratio[j0 + j];
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t w[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) w[j] = pack_f16(s[32 * h + 2 * j], s[32 * h + 2 * j + 1]);
                tc_st16(scol + 32 * set + 16 * h, w);
            }
            tc_wait_st();
            tc_fence_before();
            // what the epilogue needs of the entry, before it is given back
            const int u0 = e->u0, u1 = e->u1, units = e->units, len = e->len, nmin = e->nmin, g = e->g, v = e->v;
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&hdr->pready[n & 1]);
                mbar_arrive(&hdr->scempty[n % kXRing]);
            }
            if (flags & kXLast) {
                // ---- the segment's result
                // (S of this tile came after P V of tile n - 2: one phase at a time from there)
                ok = warp_wait(&hdr->pvdone, (uint32_t)(n - 1) & 1u) && warp_wait(&hdr->pvdone, (uint32_t)n & 1u);
                hdr->l[set][m] = lsum;
                if (named_barrier_or(bar_id, 64, !ok)) break;
                tc_fence_after();
                const float l = lsum + hdr->l[set ^ 1][m];
                const bool whole = u0 == 0 && u1 == units;
                const float inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
                AtSegment sg;
                sg.u0 = u0;
                float* rec = AtWalk<SPARSE>::record(plan, sg, D);
                const bool nans = !SPARSE && rows > 1 && hdr->nan_seen;
#pragma unroll 1
                for (int h = 0; h < D / 32; ++h) {
                    float o[16];
                    tc_ld16(trow + TM::kO + set * (D / 2) + 16 * h, o);
#pragma unroll
                    for (int c8 = 0; c8 < 2; ++c8) {
                        const int chunk = 2 * h + c8;
                        const int dim = set * (D / 2) + 8 * (D == 128 ? chunk ^ set : chunk);
                        float* x = o + 8 * c8;
                        if (nans && valid) {
                            const int32_t* table = a.block_table + (int64_t)v * a.bt_stride;
                            for (int sl = max(nmin, u0 * kXTile); sl < min(min(nlim, len), u1 * kXTile); ++sl) {
                                const int p = table[sl >> 6];
                                if (p < 0 || p >= a.n_pages) continue;
#pragma unroll
                                for (int k = 0; k < 8; ++k)
                                    if (dim + k < d &&
                                        (a.v_pool[(((int64_t)p * kBlock + (sl & 63)) * kvh + g) * d + dim + k] & 0x7f) == 0x7f)
                                        x[k] = __uint_as_float(0x7fffffffu);
                            }
                        }
                        if (!valid) continue;
                        if (whole) {
                            if (l == 0.0f)
#pragma unroll
                                for (int k = 0; k < 8; ++k) x[k] = 0.0f;
                            T* out = reinterpret_cast<T*>(a.out) + out_row * d + dim;
                            if (dim < d) {
                                store4(out, make_float4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv));
                                store4(out + 4, make_float4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv));
                            }
                        } else {
                            float4* to = reinterpret_cast<float4*>(rec + (int64_t)m * D + dim);
                            to[0] = make_float4(x[0], x[1], x[2], x[3]);
                            to[1] = make_float4(x[4], x[5], x[6], x[7]);
                        }
                    }
                }
                if (valid && set == 0) {
                    if (!whole) {
                        rec[plan.crows * D + 2 * m] = mx;
                        rec[plan.crows * D + 2 * m + 1] = l;
                    } else if (a.lse) {
                        a.lse[out_row] = row_lse(mx, l);
                    }
                }
                tc_fence_before();
            }
        }
    }
    write_empty<T, SPARSE>(cfg, a, plan);

    // ------------------------------------------------------------------------- teardown
    tc_fence_before();
    __syncthreads();
    if (wid == kXMma) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

// ------------------------------------------------------------------------------ host side
static int tc_rows(int M) { return M >= 128 ? 128 : (M + 31) / 32 * 32; }

bool kv_attend_tc_takes(const spin_kv_config& cfg, int rows, bool listed) {
    const int M = cfg.n_heads / cfg.kv_heads * (listed ? 1 : rows);
    return cfg.dtype != SPIN_DTYPE_F32 && cfg.head_dim <= 128 && M > 16;
}

size_t kv_attend_tc_workspace_bytes(const spin_kv_config&) {
    const size_t G = device_sm_count();
    return (G * sizeof(int4) + 255) / 256 * 256 + G * 2 * 128 * (size_t)(128 + 2) * sizeof(float);
}

template <typename T, int D, bool SPARSE>
static cudaError_t launch_x(const spin_kv_config& cfg, const KvAttendArgs& a, cudaStream_t s) {
    using L = XSmem<D>;
    auto k = kv_attend_tc_kernel<T, D, SPARSE>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
    if (e != cudaSuccess) return e;
    const int M = cfg.n_heads / cfg.kv_heads * (SPARSE ? 1 : a.rows);
    AtPlan p;
    p.crows = tc_rows(M);
    p.mchunks = (M + p.crows - 1) / p.crows;
    p.n_virtual = SPARSE ? cfg.n_req * a.rows : cfg.n_req;
    p.per = cfg.kv_heads * p.mchunks;
    p.unit = kXUnit;
    p.job_units = kXJobUnits;
    const int64_t jobs = (int64_t)p.n_virtual * p.per;
    const int64_t most = ((SPARSE ? a.top_k : cfg.max_slots) + kXUnit - 1) / kXUnit;
    const int sms = device_sm_count() < kAtMostSms ? device_sm_count() : kAtMostSms;
    const int64_t ctas = sms, ranks = ctas / p.per;
    const int64_t most_ranks = (p.n_virtual * (most + kXJobUnits) + kAtMinCost - 1) / kAtMinCost;
    p.split = ranks > 0 && (jobs + ctas - 1) / ctas * most > jobs * most / (ranks * p.per) + kXSplitGain;
    const int G = (int)(p.split ? (most_ranks < ranks ? most_ranks : ranks) * p.per : jobs < ctas ? jobs : ctas);
    p.by_job = jobs <= G;
    p.owner = reinterpret_cast<int4*>(a.workspace);
    p.rec = a.workspace + ((size_t)device_sm_count() * sizeof(int4) + 255) / 256 * 64;
    e = launch_pdl(k, dim3(G), dim3(kXThreads), L::kBytes, s, nullptr, 0, cfg, a, p);
    if (e != cudaSuccess || !p.split) return e;
    return launch_pdl(kv_attend_join_kernel<T, D>, dim3(p.by_job ? (unsigned)jobs : G, M < p.crows ? M : p.crows),
                      dim3(32 * kJoinWarps), 0, s, nullptr, 0, cfg, a, p, SPARSE ? 1 : a.rows);
}

template <typename T>
static cudaError_t launch_x_typed(const spin_kv_config& cfg, const KvAttendArgs& a, cudaStream_t s) {
    if (cfg.head_dim <= 64) return a.list ? launch_x<T, 64, true>(cfg, a, s) : launch_x<T, 64, false>(cfg, a, s);
    return a.list ? launch_x<T, 128, true>(cfg, a, s) : launch_x<T, 128, false>(cfg, a, s);
}

cudaError_t launch_kv_attend_tc(const spin_kv_config& cfg, const KvAttendArgs& a, cudaStream_t s) {
    return cfg.dtype == SPIN_DTYPE_BF16 ? launch_x_typed<__nv_bfloat16>(cfg, a, s) : launch_x_typed<__half>(cfg, a, s);
}

}  // namespace spin
