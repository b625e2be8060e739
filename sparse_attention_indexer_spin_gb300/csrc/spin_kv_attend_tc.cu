// spin_kv_attend_tc.cu -- attention over the paged 8-bit KV cache on tcgen05 tensor cores, for many
// query rows per key/value head (sm_103a).
//
// Same mathematics and numbers as spin_kv_attend.cu, in tiles of 128 query rows x 128 slots:
//   S = Q K^T     A = Q f16 in TMEM (rows in lanes), B = K f16 in shared memory (slots x dims)
//   O += P V      A = P f16 in TMEM,                 B = V f16 in shared memory (slots x dims, N contiguous)
// with fp32 accumulators in TMEM.  With fewer than 128 rows the products' other rows would be wasted
// (a tile's 16 MMAs of 64 cycles still take less than fetching its 32 KB from HBM), and so would the
// SM's quarters that read their TMEM lanes.  So up to 64 (32) query rows are there twice (four
// times), each copy responsible for its half (quarter) of a tile's slots: its weights are zero for
// the others, it has a reference, a sum and an output of its own, and the copies are merged like
// the pieces of a divided job when the segment ends.  What the kernel must keep low is the work per
// byte of the other pipes:
//   * a code is turned into f16 once for all the rows;
//   * the softmax has a row per thread: no shuffles, no shared-memory operands, no exchange between
//     warps; the weights are written back over the scores in TMEM as f16.
//
// Warps of a CTA (one CTA an SM):
//   0-3    softmax: warp w reads TMEM lanes 32 w .., a row a thread
//   4      issues the MMAs: S of tile n + 1 goes in before P V of tile n
//   5, 6   scouts: walk the segments, look up lists, pages and scales, a ring of tiles ahead, and have
//          the codes copied to shared memory by TMA (pages as boxes, listed slots four rows an
//          instruction); every second tile each, for a tile takes a chain of memory latencies
//   7-10   keys, 11-14 values: turn a tile's codes into f16 in the 128-byte swizzled layout the MMAs
//          read.  (With copies of their own in flight their barrier arrivals, which release what
//          came before, took 1600 cycles each.)
// A row's reference moves rarely (see kAtSlack); then its thread rescales its row of O in TMEM, after
// the products before it are done.
// Every wait is bounded; a wait that runs out unwinds all roles.
#include "spin_kv_attend.cuh"
#include "spin_tc.cuh"

namespace spin {

constexpr int kXTile = 128;                    // slots of a tile
constexpr int kXSoft = 4, kXConv = 4;          // warps: softmax; each of keys and values
constexpr int kXScouts = 2;                    // one for each place that codes are copied to
constexpr int kXMma = kXSoft, kXScout = kXMma + 1, kXKeys = kXScout + kXScouts, kXValues = kXKeys + kXConv;
constexpr int kXWarps = kXValues + kXConv, kXThreads = 32 * kXWarps;
constexpr int kXCols = 32;                     // slots a softmax thread takes at a time
constexpr int kXRing = 6;                      // tiles the scouts are ahead: three of each
constexpr int kXUnit = kXTile;
constexpr int kXJobUnits = 6;                  // a job's start: 3 us beside 0.5 us a tile
constexpr int kXSplitGain = 12;

enum XFlag { kXFirst = 1, kXLast = 2, kXOdd = 4, kXStop = 8 };

struct XEntry {                // a tile as the scouts publish it
    float ks[kXTile], lv[kXTile], iv[kXTile], ratio[kXTile];
    uint32_t live[4];          // slots that are there
    int flags, slot0, v, g, mc, u0, u1, units, len, nmin;
    int pad[2];
};

struct XHdr {
    // A barrier's phases are told apart by their parity alone, so nobody may wait for one while the
    // phase two before or after it could be the current one: two barriers each for what alternates, and
    // one scout for each of the places that codes are copied to.
    uint64_t scfull[kXRing], scempty[kXRing];
    uint64_t rawfull[2], rawempty[2], kfull[2], kempty[2], vfull[2], vempty[2];
    uint64_t sfull[2], pready[2], pvdone[2], qready, merged, fin;
    uint32_t tmem_base;
    volatile int abort_flag;
    int nan_seen;              // a NaN value among slots that some rows see and others do not
    int64_t scan[kXWarps + 3];
    float m[128], l[128];      // references and sums of a segment's rows
};

template <int D> struct XSmem {
    static constexpr int kStage = kXTile * D * 2;  // one of keys, values: D / 64 blocks of 128 rows x 128 bytes
    static constexpr int kK = 0, kV = 2 * kStage;
    static constexpr int kRaw = 4 * kStage, kRawTile = kXTile * D;  // codes on their way: two tiles of keys, two of values
    static constexpr int kRingAt = kRaw + 4 * kRawTile;
    // 16 dims of the rows' copies while a segment is merged: at most 96 rows
    static constexpr int kPitch = 16 + 4;          // floats; a row a thread: the pitch spreads the banks
    static constexpr int kMerge = kRingAt + kXRing * (int)sizeof(XEntry);
    static constexpr int kHdr = kMerge + 96 * kPitch * 4;
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

// The roles' code is kept small -- loops over pieces, rare paths out of line: fifteen warps at work in
// different places of 100 KB of code spend most of their time fetching instructions (the first
// version took 4 times as long).

// A bounded wait; one that runs out is reported to the other roles.
static __device__ __noinline__ bool x_gave_up(XHdr* hdr, uint32_t* status) {
    hdr->abort_flag = 1;
    set_status(status, SPIN_STATUS_TIMEOUT);
    return false;
}
constexpr int kXSpins = 1 << 20;  // some 0.1 to 1 s of failed trials
__device__ __forceinline__ bool x_wait(uint64_t* bar, uint32_t parity, XHdr* hdr, uint32_t* status) {
    for (int i = 0; !mbar_try_wait(bar, parity); ++i)
        if (i == kXSpins || hdr->abort_flag) return x_gave_up(hdr, status);
    return true;
}

// A query row (d values of T at q, or none), scaled by a power of two and rounded to f16, into columns
// `col` .. of this thread's TMEM lane.  Returns what turns its products into exponents of two.
template <typename T, int D>
static __device__ __noinline__ float x_stage_q(const uint4* q, bool valid, int d, float softmax_scale, uint32_t col) {
    float amax = 0.0f;
#pragma unroll 1
    for (int i = 0; valid && i < d / 8; ++i) {
        float x[8];
        unpack8<T>(q[i], x);
#pragma unroll
        for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(x[k]));
    }
    const int k2 = max(-112, (int)(__float_as_uint(amax) >> 23) - 127);
    // a negative softmax scale goes into the query: scores then grow with t
    const float f = copysignf(__uint_as_float((uint32_t)(127 + 14 - k2) << 23), softmax_scale);
    __syncwarp();
#pragma unroll 1
    for (int h = 0; h < D / 32; ++h) {
        uint32_t w[16];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            // D = 128: neighbouring chunks of the second 64 dims trade places, as the codes' do
            const int chunk = 4 * h + c, i = D == 128 ? chunk ^ (chunk >> 3) : chunk;
            float x[8];
            unpack8<T>(valid && i < d / 8 ? q[i] : make_uint4(0, 0, 0, 0), x);
#pragma unroll
            for (int k = 0; k < 4; ++k) w[4 * c + k] = pack_f16(x[2 * k] * f, x[2 * k + 1] * f);
        }
        __syncwarp();
        tc_st16(col + 16 * h, w);
    }
    tc_wait_st();
    tc_fence_before();
    return __uint_as_float((uint32_t)max(1, 127 - 14 + k2) << 23) * (fabsf(softmax_scale) * 1.4426950408889634f);
}

// Scores of columns j0 .. j0 + cols that a row's end cuts, or whose key scale is negative: scaled (by
// qs and each page's key scale) and cut off in place.
static __device__ __noinline__ void x_cut(uint32_t scol, int j0, int cols, float qs, const float* ks, int lim0) {
#pragma unroll 1
    for (int j = j0; j < j0 + cols; j += 16) {
        float x[16];
        uint32_t w[16];
        tc_ld16(scol + j, x);
        const float c = qs * ks[j & ~63];
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(j + i < lim0 ? x[i] * c : __uint_as_float(0xff800000u));
        tc_st16(scol + j, w);
    }
    tc_wait_st();
}

// A row of O times f.
template <int D> static __device__ __noinline__ void x_rescale(uint32_t col, float f) {
#pragma unroll 1
    for (int h = 0; h < D / 16; ++h) {
        float o[16];
        uint32_t w[16];
        tc_ld16(col + 16 * h, o);
#pragma unroll
        for (int k = 0; k < 16; ++k) w[k] = __float_as_uint(o[k] * f);
        tc_st16(col + 16 * h, w);
    }
    tc_wait_st();
}

template <typename T, int D, bool SPARSE>
__global__ void __launch_bounds__(kXThreads, 1)
kv_attend_tc_kernel(const __grid_constant__ spin_kv_config cfg, const __grid_constant__ KvAttendArgs a, AtPlan plan,
                    const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
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
    const int fold = 128 / (plan.crows <= 64 ? plan.crows : 128);  // copies of a query row
    const float ninf = __uint_as_float(0xff800000u);

    if (tid == 0) {
        for (int i = 0; i < kXRing; ++i) {
            mbar_init(&hdr->scfull[i], 1);
            mbar_init(&hdr->scempty[i], 2 * kXConv + kXSoft + 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&hdr->rawfull[i], 1);
            mbar_init(&hdr->rawempty[i], 2 * kXConv);
            mbar_init(&hdr->kfull[i], kXConv);
            mbar_init(&hdr->vfull[i], kXConv);
            mbar_init(&hdr->kempty[i], 1);
            mbar_init(&hdr->vempty[i], 1);
            mbar_init(&hdr->sfull[i], 1);
            mbar_init(&hdr->pvdone[i], 1);
            mbar_init(&hdr->pready[i], kXSoft);
        }
        mbar_init(&hdr->qready, kXSoft);
        mbar_init(&hdr->merged, kXSoft);
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

    // one lane waits for the warp
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        int ok = 1;
        if (lane == 0) ok = x_wait(bar, parity, hdr, a.status);
        return __shfl_sync(0xffffffffu, ok, 0);
    };

    if (wid >= kXScout && wid < kXKeys) {
        // ------------------------------------------------------------------------ scouts
        // Two steps a tile, in successive turns of the loop: its place in the ring and its list entries;
        // its pages, scales and publication (before the next place is waited for).
        constexpr int NE = SPARSE ? 4 : 1;
        int e1[NE], e2[NE], n1 = -1, n2 = -1;   // nI: tile in step I, -1: none
        AtSegment seg;
        const uint32_t raw = smem_u32(smem + L::kRaw);
        int issued = -1;                          // last tile copied
        int at = 0, to = 0, nmin = 0, tile = -1;  // units of the current segment; tile: the last one met
        bool more = true;
        for (;;) {
            n2 = n1;
            n1 = -1;
#pragma unroll
            for (int i = 0; i < NE; ++i) e2[i] = e1[i];
            __syncwarp();
            if (n2 >= 0) {  // step 2
                XEntry* e = ring + n2 % kXRing;
                const int g = e->g;
                uint64_t* full = &hdr->rawfull[n2 & 1];
                const uint32_t kd = raw + (uint32_t)((n2 & 1) * L::kRawTile), vd = kd + 2 * L::kRawTile;
                bool odd = false;
                auto publish = [&](int j, bool live, float k, float v) {  // a slot's scales
                    const bool fine = in_log_range(v);
                    const float lg = scale_log2(v);
                    e->ks[j] = k;
                    e->lv[j] = live ? lg : ninf;
                    e->iv[j] = !live ? 0.0f : fine ? __frcp_rn(v) : ex2(-lg);
                    e->ratio[j] = fine || !live ? 1.0f : v * ex2(-lg);
                    odd |= live && !fine;
                };
                if constexpr (SPARSE) {
                    const int32_t* table = a.block_table + (int64_t)(e->v / a.rows) * a.bt_stride;
                    int page[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (e2[i] < -1 || e2[i] >= e->nmin) {
                            set_status(a.status, SPIN_STATUS_BAD_LIST);
                            e2[i] = -1;
                        }
                        page[i] = e2[i] >= 0 ? table[e2[i] >> 6] : -1;
                    }
                    float ks[4], vs[4];
                    uint32_t mask[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (e2[i] >= 0 && (page[i] < 0 || page[i] >= a.n_pages)) {
                            set_status(a.status, SPIN_STATUS_BAD_PAGE);
                            page[i] = -1;
                        }
                        ks[i] = page[i] >= 0 ? a.k_scale[(int64_t)page[i] * kvh + g] : 0.0f;
                        vs[i] = page[i] >= 0 ? a.v_scale[(int64_t)page[i] * kvh + g] : 0.0f;
                        mask[i] = __ballot_sync(0xffffffffu, page[i] >= 0);
                    }
                    // the codes' copies, once the converters have read tile n2 - 2
                    if (!warp_wait(&hdr->rawempty[n2 & 1], (uint32_t)(n2 >> 1 & 1) ^ 1u)) break;
                    // four rows a lane; a slot that is not there copies one that is (the converters drop it)
                    const int any = __ffs(mask[0] ? mask[0] : mask[1] ? mask[1] : mask[2] ? mask[2] : mask[3]) - 1;
                    if (any < 0) {
                        if (lane == 0) mbar_arrive(full);
                    } else {
                        if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)(2 * kXTile * d));
                        __syncwarp();
                        int y[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) y[i] = page[i] >= 0 ? page[i] * kBlock + (e2[i] & 63) : -1;
                        const int spare = __shfl_sync(0xffffffffu, mask[0] ? y[0] : mask[1] ? y[1] : mask[2] ? y[2] : y[3], any);
#pragma unroll
                        for (int i = 0; i < 4; ++i) y[i] = y[i] < 0 ? spare : y[i];
                        // lane l issues rows 4 l .. 4 l + 3, held by lanes 4 (l mod 8) .. of register l / 8
                        int r[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            r[k] = 0;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int x = __shfl_sync(0xffffffffu, y[i], 4 * (lane & 7) + k);
                                if (lane >> 3 == i) r[k] = x;
                            }
                        }
                        tma_gather4(kd + 4 * lane * d, &kmap, g * d, r[0], r[1], r[2], r[3], full);
                        tma_gather4(vd + 4 * lane * d, &vmap, g * d, r[0], r[1], r[2], r[3], full);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        publish(32 * i + lane, page[i] >= 0, ks[i], vs[i]);
                        if (lane == 0) e->live[i] = mask[i];
                    }
                } else {
                    // lanes 0 and 1 (and their like): the tile's pages
                    int p = e2[0];
                    if (p != -2 && (p < 0 || p >= a.n_pages)) {
                        set_status(a.status, SPIN_STATUS_BAD_PAGE);
                        p = -1;
                    }
                    const float k = p >= 0 ? a.k_scale[(int64_t)p * kvh + g] : 0.0f, v = p >= 0 ? a.v_scale[(int64_t)p * kvh + g] : 0.0f;
                    const uint32_t there = __ballot_sync(0xffffffffu, p >= 0);
                    if (!warp_wait(&hdr->rawempty[n2 & 1], (uint32_t)(n2 >> 1 & 1) ^ 1u)) break;
                    if (lane == 0) {
                        if (there & 3u) mbar_arrive_expect_tx(full, (uint32_t)(2 * kBlock * d) * __popc(there & 3u));
                        else mbar_arrive(full);
                    }
                    __syncwarp();
                    if (lane < 2 && p >= 0) {
                        tma_load_3d(kd + lane * kBlock * d, &kmap, g * d, 0, p, full);
                        tma_load_3d(vd + lane * kBlock * d, &vmap, g * d, 0, p, full);
                    }
                    if (lane < 2) publish(kBlock * lane, p >= 0, k, v);
                    if (lane < 4) {  // 32 slots each: those before the end, of a page that is there
                        const int left = e->len - e->slot0 - 32 * lane;
                        e->live[lane] = !(there >> (lane >> 1) & 1u) || left <= 0 ? 0u : left >= 32 ? 0xffffffffu : (1u << left) - 1;
                    }
                }
                issued = n2;
                odd = __any_sync(0xffffffffu, odd);
                if (lane == 0 && odd) e->flags |= kXOdd;
                __syncwarp();
                if (lane == 0) mbar_arrive(&hdr->scfull[n2 % kXRing]);
            }
            // this scout's next tile
            while (more) {
                if (at == to) {
                    more = walk.next(cfg, a, plan, seg);
                    if (!more) break;
                    at = seg.u0;
                    to = seg.u1;
                    nmin = 0x7fffffff;
                    if constexpr (SPARSE) {
                        nmin = row_slots(a, seg.v, cfg.max_slots);  // the row's slots bound its entries
                    } else {
                        for (int r = 0; r < rows; ++r) nmin = min(nmin, row_slots(a, (int64_t)seg.v * rows + r, cfg.max_slots));
                    }
                    if (lane == 0 && wid == kXScout) walk.own(plan, seg);
                }
                ++at;
                if (++tile % kXScouts == wid - kXScout) break;
            }
            if (!more) break;
            if (more) {  // step 1
                const int n = tile;
                XEntry* e = ring + n % kXRing;
                if (!warp_wait(&hdr->scempty[n % kXRing], (uint32_t)(n / kXRing & 1) ^ 1u)) break;
                const int slot0 = (at - 1) * kXTile;
                if (lane == 0) {
                    e->flags = (at - 1 == seg.u0 ? kXFirst : 0) | (at == seg.u1 ? kXLast : 0);
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
                if constexpr (SPARSE) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int j = slot0 + 32 * i + lane;
                        e1[i] = j < seg.len ? a.list[(int64_t)seg.v * a.top_k + j] : -1;
                    }
                } else {  // the page of this half of the tile already (-2: no slot there)
                    const int j = slot0 + kBlock * (lane & 1);
                    e1[0] = j < seg.len ? max(-1, a.block_table[(int64_t)seg.v * a.bt_stride + (j >> 6)]) : -2;
                }
                n1 = n;
            }
        }
        pdl_trigger();
        // the tile after the last one says stop
        ++tile;
        if (!hdr->abort_flag && tile % kXScouts == wid - kXScout &&
            warp_wait(&hdr->scempty[tile % kXRing], (uint32_t)(tile / kXRing & 1) ^ 1u) && lane == 0) {
            ring[tile % kXRing].flags = kXStop;
            mbar_arrive(&hdr->scfull[tile % kXRing]);
        }
        // Never leave with copies in flight: the converters have waited for every tile's, unless a wait gave up.
        if (hdr->abort_flag && issued >= 0 && lane == 0 && !mbar_wait(&hdr->rawfull[issued & 1], (uint32_t)(issued >> 1 & 1), nullptr, kWaitLimitNs))
            set_status(a.status, SPIN_STATUS_TIMEOUT);
    } else if (wid >= kXKeys) {
        // --------------------------------------------------------------------- converters
        const bool values = wid >= kXValues;
        const int t = tid - 32 * (values ? kXValues : kXKeys);
        constexpr int CH = D / 16, RS = 128 / CH, NP = CH;  // chunks of a row, rows at a time, pieces a thread
        const int prow = t / CH, x = t % CH;
        const bool in_row = 16 * x < d;
        uint64_t* full = values ? hdr->vfull : hdr->kfull;
        uint64_t* empty = values ? hdr->vempty : hdr->kempty;
        const uint32_t base = smem_u32(smem + (values ? L::kV : L::kK));
        // A piece's 16 codes fill chunks 2x and 2x + 1 of its row's 16-byte chunks of f16; in the second
        // block of 64 dims the two trade places, so that the eight stores of a row hit different banks.
        const int c0 = 2 * (x & 3) + (x >> 2), c1 = 2 * (x & 3) + 1 - (x >> 2), block = x >> 2;

        const uint32_t raw = smem_u32(smem + L::kRaw + (values ? 2 * L::kRawTile : 0)) + 16 * x;
        for (int n = 0;; ++n) {
            const XEntry* e = ring + n % kXRing;
            if (!warp_wait(&hdr->scfull[n % kXRing], (uint32_t)(n / kXRing & 1))) break;
            if (e->flags & kXStop) break;
            // the live bits of rows prow, prow + RS, ...
            uint32_t live = 0;
            if (in_row)
#pragma unroll
                for (int i = 0; i < NP; ++i) live |= (e->live[(RS * i) >> 5] >> (prow + ((RS * i) & 31)) & 1u) << i;
            const int lim = !SPARSE && values ? e->nmin - e->slot0 : kXTile;  // rows from here on: seen by some query rows only
            __syncwarp();
            if (lane == 0) mbar_arrive(&hdr->scempty[n % kXRing]);
            if (!warp_wait(&hdr->rawfull[n & 1], (uint32_t)(n >> 1 & 1)) ||
                !warp_wait(&empty[n & 1], (uint32_t)(n >> 1 & 1) ^ 1u))
                break;
            const uint32_t st = base + (uint32_t)((n & 1) * L::kStage) + block * (kXTile * 128);
            const uint32_t from = raw + (uint32_t)((n & 1) * L::kRawTile) + prow * d;
            if (!SPARSE && lim < kXTile) {
                // a NaN here must not reach the rows that do not see it (0 x NaN): it leaves the tile, and
                // the epilogue looks for the rows that do
#pragma unroll 1
                for (int i = 0; i < 4 * NP && in_row; ++i) {
                    if (prow + RS * (i >> 2) < lim) continue;
                    const uint32_t at = from + RS * d * (i >> 2) + 4 * (i & 3);
                    uint32_t w;
                    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(at) : "memory");
                    const uint32_t m = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;  // bytes that are NaN
                    if (m == 0) continue;
                    hdr->nan_seen = 1;
                    asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(w & ~((m >> 7) * 0xffu)) : "memory");
                }
            }
            // (rows RS apart share their swizzle)
            const uint32_t d0 = st + prow * 128 + ((c0 ^ (prow & 7)) << 4), d1 = st + prow * 128 + ((c1 ^ (prow & 7)) << 4);
#pragma unroll 2
            for (int i = 0; i < NP; ++i) {
                uint4 c = make_uint4(0, 0, 0, 0);
                if (live >> i & 1u) c = lds128(from + RS * d * i);
                uint4 u, v;
                codes_to_f16(c.x, u.x, u.y);
                codes_to_f16(c.y, u.z, u.w);
                codes_to_f16(c.z, v.x, v.y);
                codes_to_f16(c.w, v.z, v.w);
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(d0 + RS * 128 * i), "r"(u.x), "r"(u.y), "r"(u.z),
                             "r"(u.w)
                             : "memory");
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(d1 + RS * 128 * i), "r"(v.x), "r"(v.y), "r"(v.z),
                             "r"(v.w)
                             : "memory");
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&full[n & 1]);
                mbar_arrive(&hdr->rawempty[n & 1]);
            }
        }
    } else if (wid == kXMma) {
        // ------------------------------------------------------------------------ MMA issue
        if (lane == 0) {
            const uint32_t id_s = idesc_mma(0u, kXTile, 128u), id_o = idesc_mma(0u, (uint32_t)D, 128u) | kIdescBn;
            const uint64_t kdesc = smem_desc_sw128(smem_u32(smem + L::kK));
            const uint64_t vdesc = smem_desc_sw128_n(smem_u32(smem + L::kV), kXTile * 128);
            auto wait = [&](uint64_t* bar, uint32_t parity) -> bool { return x_wait(bar, parity, hdr, a.status); };
            auto product = [&](int n, bool first) -> bool {  // O (+)= P V of tile n
                if (!wait(&hdr->pready[n & 1], (uint32_t)(n >> 1 & 1)) || !wait(&hdr->vfull[n & 1], (uint32_t)(n >> 1 & 1)))
                    return false;
                tc_fence_after();
                uint64_t v = vdesc + (uint64_t)((n & 1) * (L::kStage >> 4));
                uint32_t p = tmem + TM::kS + (n & 1) * kXTile, add = !first;
#pragma unroll 2
                for (int k = 0; k < kXTile / 16; ++k, v += 2048 >> 4, p += 8, add = 1u) tc_mma_f16_ta(tmem + TM::kO, p, v, id_o, add);
                tc_commit(&hdr->vempty[n & 1]);
                tc_commit(&hdr->pvdone[n & 1]);
                return true;
            };
            int pend = -1, segs = 0, slot = 0;   // slot: n mod kXRing
            uint32_t turn = 0;                   // n / kXRing
            bool pend_first = false;
            for (int n = 0;; ++n) {
                if (!wait(&hdr->scfull[slot], turn & 1u)) break;
                const int flags = ring[slot].flags;
                if (flags & kXStop) break;
                mbar_arrive(&hdr->scempty[slot]);
                if (++slot == kXRing) slot = 0, ++turn;
                if ((flags & kXFirst) && !wait(&hdr->qready, (uint32_t)(segs++ & 1))) break;
                if (!wait(&hdr->kfull[n & 1], (uint32_t)(n >> 1 & 1))) break;
                tc_fence_after();
                // the scores' buffer held tile n - 2: its P V was issued, and reads it before this writes
                const uint64_t st = kdesc + (uint64_t)((n & 1) * (L::kStage >> 4));
                const uint32_t sc = tmem + TM::kS + (n & 1) * kXTile;
#pragma unroll 2
                for (int k = 0; k < D / 16; ++k)
                    tc_mma_f16_ta(sc, tmem + TM::kQ + 8 * k, st + ((uint32_t)((k >> 2) * (kXTile * 128) + (k & 3) * 32) >> 4), id_s, k);
                tc_commit(&hdr->kempty[n & 1]);
                tc_commit(&hdr->sfull[n & 1]);
                bool ok = true;
#pragma unroll 1
                for (int m = pend >= 0 ? n - 1 : n; ok && m < n + ((flags & kXLast) ? 1 : 0); ++m)
                    ok = product(m, m == n ? (flags & kXFirst) : pend_first);
                if (!ok) break;
                pend = (flags & kXLast) ? -1 : n;
                pend_first = flags & kXFirst;
            }
            // never leave with MMAs in flight
            tc_commit(&hdr->fin);
            if (!mbar_wait(&hdr->fin, 0u, nullptr)) set_status(a.status, SPIN_STATUS_TIMEOUT);
        }
        __syncwarp();
    } else {
        // --------------------------------------------------------------------------- softmax
        const int own_rows = 128 / fold, m = (32 * wid + lane) & (own_rows - 1);  // this thread's row of the chunk
        const int part = (32 * wid) / own_rows, cols = kXTile / fold;             // its copy, its share of the slots
        const int j0 = part * cols;
        const uint32_t trow = tmem + ((uint32_t)(32 * wid) << 16);
        float* merge = reinterpret_cast<float*>(smem + L::kMerge);
        float mx = ninf, lsum = 0.0f, qs = 0.0f;
        int nlim = 0;
        int64_t out_row = 0;
        bool valid = false;
        uint32_t meetings = 0;
        auto meet = [&]() -> bool {  // the softmax warps, by a barrier whose wait is bounded
            __syncwarp();
            if (lane == 0) mbar_arrive(&hdr->merged);
            return warp_wait(&hdr->merged, meetings++ & 1u);
        };
        for (int n = 0;; ++n) {
            const XEntry* e = ring + n % kXRing;
            if (!warp_wait(&hdr->scfull[n % kXRing], (uint32_t)(n / kXRing & 1))) break;
            const int flags = e->flags;
            if (flags & kXStop) break;
            if (flags & kXFirst) {
                // ---- a new job: this row's query, scaled by a power of two and rounded to f16, into TMEM
                const int mm = e->mc * plan.crows + m;
                valid = m < plan.crows && mm < M;
                const int64_t br = (int64_t)e->v * rows + (valid ? mm / group : 0);
                out_row = br * H + (int64_t)e->g * group + (valid ? mm % group : 0);
                nlim = valid && !SPARSE ? row_slots(a, br, cfg.max_slots) : 0x7fffffff;
                qs = x_stage_q<T, D>(reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(a.q) + out_row * d), valid, d,
                                     cfg.softmax_scale, trow + TM::kQ);
                __syncwarp();
                if (lane == 0) mbar_arrive(&hdr->qready);
                mx = ninf;
                lsum = 0.0f;
            }
            const uint32_t scol = trow + TM::kS + (n & 1) * kXTile;
            if (!warp_wait(&hdr->sfull[n & 1], (uint32_t)(n >> 1 & 1))) break;
            tc_fence_after();
            // Where a row ends within the tile, or a key scale is negative, the scores are scaled and cut off
            // in place first.
            bool cut = false;
            if constexpr (!SPARSE) {
                cut = nlim - (e->slot0 + j0) < cols || e->ks[j0] < 0.0f || e->ks[(j0 + cols - 1) & ~63] < 0.0f;
                cut = __any_sync(0xffffffffu, cut);
                if (cut) x_cut(scol, j0, cols, qs, e->ks, nlim - e->slot0);
            }
            // scores of W slots of one page: with a list x = t + log2 vs of every slot (-inf where there is
            // none); else what x = c s + lv is made of
            constexpr int W = kXCols;
            auto scores = [&](int j, float (&s)[W], float& c, float& lv) {
                tc_ld32(scol + j, s);
                c = 1.0f;
                lv = 0.0f;
                if constexpr (SPARSE) {
#pragma unroll
                    for (int i = 0; i < W; i += 4) {
                        const float4 k4 = *reinterpret_cast<const float4*>(e->ks + j + i);
                        const float4 v4 = *reinterpret_cast<const float4*>(e->lv + j + i);
                        s[i] = fmaf(s[i] * k4.x, qs, v4.x);
                        s[i + 1] = fmaf(s[i + 1] * k4.y, qs, v4.y);
                        s[i + 2] = fmaf(s[i + 2] * k4.z, qs, v4.z);
                        s[i + 3] = fmaf(s[i + 3] * k4.w, qs, v4.w);
                    }
                } else {
                    if (!cut) c = qs * e->ks[j & ~63];
                    lv = e->lv[j & ~63];
                }
            };
            float top = ninf;
#pragma unroll 1
            for (int j = j0; j < j0 + cols; j += W) {
                float s[W], c, lv, t[4] = {ninf, ninf, ninf, ninf};
                scores(j, s, c, lv);
#pragma unroll
                for (int i = 0; i < W; ++i) t[i & 3] = fmaxf(t[i & 3], s[i]);
                // (fmaxf drops the NaN of an infinite product)
                top = fmaxf(top, fmaf(fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])), c, lv));
            }
            top -= kAtTop;
            if (__any_sync(0xffffffffu, top > mx + kAtSlack)) {
                const float now = fmaxf(mx, top);
                const float f = now == ninf ? 1.0f : ex2(mx - now);
                mx = now;
                lsum *= f;
                if (!(flags & kXFirst)) {
                    if (!warp_wait(&hdr->pvdone[(n - 1) & 1], (uint32_t)((n - 1) >> 1 & 1))) break;
                    tc_fence_after();
                    x_rescale<D>(trow + TM::kO, f);
                }
            }
            // ---- weights: 2^(x - m), written over the scores as f16
            const float ref = mx == ninf ? 0.0f : mx;
#pragma unroll 1
            for (int j = j0; j < j0 + cols; j += W) {
                float s[W], c, lv, add[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                scores(j, s, c, lv);
                const float bias = lv - ref;
#pragma unroll
                for (int i = 0; i < W; ++i) s[i] = ex2(SPARSE ? s[i] + bias : fmaf(s[i], c, bias));
                if constexpr (SPARSE) {
#pragma unroll
                    for (int i = 0; i < W; i += 4) {
                        const float4 i4 = *reinterpret_cast<const float4*>(e->iv + j + i);
                        add[0] = fmaf(s[i], i4.x, add[0]);
                        add[1] = fmaf(s[i + 1], i4.y, add[1]);
                        add[2] = fmaf(s[i + 2], i4.z, add[2]);
                        add[3] = fmaf(s[i + 3], i4.w, add[3]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < W; ++i) add[i & 3] += s[i];
                }
                lsum = fmaf((add[0] + add[1]) + (add[2] + add[3]), SPARSE ? 1.0f : e->iv[j & ~63], lsum);
                if (flags & kXOdd) {
#pragma unroll
                    for (int i = 0; i < W; ++i) s[i] *= e->ratio[SPARSE ? j + i : j & ~63];
                }
#pragma unroll
                for (int h = 0; h < W / 32; ++h) {
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) w[i] = pack_f16(s[32 * h + 2 * i], s[32 * h + 2 * i + 1]);
                    tc_st16(scol + j / 2 + 16 * h, w);
                }
            }
            if (fold > 1) {  // the slots of the other copies
                uint32_t zero[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) zero[i] = 0u;
#pragma unroll 1
                for (int j = 0; j < kXTile; j += 32)
                    if (j < j0 || j >= j0 + cols) tc_st16(scol + j / 2, zero);
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
                if (!warp_wait(&hdr->pvdone[n & 1], (uint32_t)(n >> 1 & 1))) break;
                tc_fence_after();
                hdr->m[32 * wid + lane] = mx;
                hdr->l[32 * wid + lane] = lsum;
                if (fold > 1 && !meet()) break;
                float top_m = ninf, l = 0.0f;
                for (int i = 0; i < fold; ++i) top_m = fmaxf(top_m, hdr->m[i * own_rows + m]);
                for (int i = 0; i < fold; ++i) {
                    const float mi = hdr->m[i * own_rows + m];
                    l = fmaf(mi == ninf ? 0.0f : ex2(mi - top_m), hdr->l[i * own_rows + m], l);
                }
                const float f = mx == ninf ? 0.0f : ex2(mx - top_m);
                const bool whole = u0 == 0 && u1 == units;
                const float inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
                AtSegment sg;
                sg.u0 = u0;
                float* rec = AtWalk<SPARSE>::record(plan, sg, D);
                const bool nans = !SPARSE && rows > 1 && hdr->nan_seen;
                bool ok = true;
#pragma unroll 1
                for (int h = 0; h < D / 16 && ok; ++h) {
                    float o[16];
                    __syncwarp();
                    tc_ld16(trow + TM::kO + 16 * h, o);
#pragma unroll
                    for (int k = 0; k < 16; ++k) o[k] *= f;
                    if (fold > 1) {
                        float4* to = reinterpret_cast<float4*>(merge + ((part - 1) * own_rows + m) * L::kPitch);
                        if (part > 0) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) to[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                        }
                        if (!(ok = meet())) continue;
                        for (int i = 1; i < fold && part == 0; ++i) {
                            const float4* from = reinterpret_cast<const float4*>(merge + ((i - 1) * own_rows + m) * L::kPitch);
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float4 x = from[k];
                                o[4 * k] += x.x;
                                o[4 * k + 1] += x.y;
                                o[4 * k + 2] += x.z;
                                o[4 * k + 3] += x.w;
                            }
                        }
                        ok = meet();
                    }
                    if (!valid || part > 0) continue;
#pragma unroll
                    for (int c8 = 0; c8 < 2; ++c8) {
                        const int chunk = 2 * h + c8, dim = 8 * (D == 128 ? chunk ^ (chunk >> 3) : chunk);
                        float* x = o + 8 * c8;
                        uint32_t nan_bits = 0;
                        if (nans) {
                            const int last = min(min(nlim, len), u1 * kXTile);
#pragma unroll 1
                            for (int k = 0; k < 8 && dim + k < d; ++k)
                                if (nan_value(cfg, a, v, g, dim + k, max(nmin, u0 * kXTile), last)) nan_bits |= 1u << k;
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                if ((nan_bits >> k) & 1u) x[k] = __uint_as_float(0x7fffffffu);
                        }
                        if (!whole) {
                            float4* to = reinterpret_cast<float4*>(rec + (int64_t)m * D + dim);
                            to[0] = make_float4(x[0], x[1], x[2], x[3]);
                            to[1] = make_float4(x[4], x[5], x[6], x[7]);
                        } else if (dim < d) {
                            if (l == 0.0f)
#pragma unroll
                                for (int k = 0; k < 8; ++k) x[k] = 0.0f;
                            T* out = reinterpret_cast<T*>(a.out) + out_row * d + dim;
                            store4(out, make_float4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv));
                            store4(out + 4, make_float4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv));
                        }
                    }
                }
                if (!ok) break;
                if (part == 0) {
                    if (valid && !whole) {
                        rec[plan.crows * D + 2 * m] = top_m;
                        rec[plan.crows * D + 2 * m + 1] = l;
                    } else if (valid && a.lse) {
                        a.lse[out_row] = row_lse(top_m, l);
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
static int tc_rows(int M) { return M <= 32 ? 32 : M <= 64 ? 64 : 128; }

// Tensor-map coordinates are 32-bit (pages x 64 slots), and a copy of four rows starts on 128 bytes.
bool kv_attend_tc_takes(const spin_kv_config& cfg, int rows, bool listed, int64_t n_pages) {
    const int M = cfg.n_heads / cfg.kv_heads * (listed ? 1 : rows);
    return false && cfg.dtype != SPIN_DTYPE_F32 && cfg.head_dim <= 128 && M > 16 && n_pages >= 1 && n_pages < (1 << 25) &&
           (!listed || cfg.head_dim % 32 == 0);
}

// A pool as bytes: [page][slot][kv_heads * head_dim], one head of a page at a time; with a list
// [page * 64 + slot][kv_heads * head_dim], one head of a row.
static bool encode_pool(CUtensorMap* map, const spin_kv_config& cfg, const void* base, int64_t n_pages, bool rows) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t row = (cuuint64_t)cfg.kv_heads * cfg.head_dim;
    const cuuint64_t dim[3] = {row, rows ? (cuuint64_t)n_pages * kBlock : (cuuint64_t)kBlock, (cuuint64_t)n_pages};
    const cuuint64_t stride[2] = {row, row * kBlock};
    const cuuint32_t box[3] = {(cuuint32_t)cfg.head_dim, rows ? 1u : (cuuint32_t)kBlock, 1u}, estride[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, rows ? 2 : 3, const_cast<void*>(base), dim, stride, box, estride,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t kv_attend_tc_workspace_bytes(const spin_kv_config&) {
    const size_t G = device_sm_count();
    return (G * sizeof(int4) + 255) / 256 * 256 + G * 2 * 128 * (size_t)(128 + 2) * sizeof(float);
}

template <typename T, int D, bool SPARSE>
static cudaError_t launch_x(const spin_kv_config& cfg, const KvAttendArgs& a, cudaStream_t s) {
    using L = XSmem<D>;
    auto k = kv_attend_tc_kernel<T, D, SPARSE>;
    static std::atomic<uint64_t> allowed;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), L::kBytes, allowed);
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
    CUtensorMap kmap, vmap;
    if (!encode_pool(&kmap, cfg, a.k_pool, a.n_pages, SPARSE) || !encode_pool(&vmap, cfg, a.v_pool, a.n_pages, SPARSE))
        return cudaErrorInvalidValue;
    e = launch_pdl(k, dim3(G), dim3(kXThreads), L::kBytes, s, nullptr, 0, cfg, a, p, kmap, vmap);
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
