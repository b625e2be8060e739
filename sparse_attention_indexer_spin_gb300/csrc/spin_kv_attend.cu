// spin_kv_attend.cu -- attention over the paged 8-bit KV cache (sm_103a).
//
// Per query row and head, over the row's set of slots (its context, or the slots of a list):
//   s_i = softmax_scale ks (q . kc_i),  out = sum_i e^{s_i} vs vc_i / sum_i e^{s_i},
//   lse = ln sum_i e^{s_i}
// in one pass over the cache, with the running maximum and sum of the softmax.
//
// Numbers.  Everything is in base 2: t_i = log2(e) s_i.  A row keeps a reference m and
//   l = sum_i 2^(t_i - m),   o = sum_i 2^(t_i - m) vs_i vc_i,   out = o / l
// in fp32 (l times 2^-20: a value scale of 0 counts as 2^-100 below).  Codes become f16 exactly.  q is scaled by a power of two per row to just below 2^15
// and rounded to f16: bf16 and f16 values keep every bit unless they are below 2^-29 of the
// row's largest (f16's subnormals; off by at most 2^-39 of it).  The weights 2^(t_i - m) vs_i
// are rounded to f16 for their product with the codes (2^-11 each).  fp32 queries and
// weights go in as two f16 terms (22 bits).  The reference follows max(t_i + log2 vs_i) - 12, so
// that the largest weights, value scale included, sit between 2^12 and 2^15: a page's small
// value scale costs no precision, and weights lose bits only below 2^-26 of the largest.  The
// reference moves only when a maximum exceeds it by more than 2^3, which spares most of the
// rescaling of o.  From 2^20 on an exponent's roundings come near 2^0 (they are at most four of 2^-4 there),
// and weights would leave f16's range, or all of a row's vanish: such tiles round t_i as the maximum was
// rounded and keep it at 15 above the reference at most.
//
// Shape.  A warp takes every fourth tile of 32 slots of its CTA's segment through a ring of its own
// (two stages of cp.async, no barrier inside a segment), multiplies with mma.sync m16n8k16, and
// keeps queries, scores, weights and o in registers; the four warps are merged once per segment.
// The codes have to become f16 in registers anyway, on their way from shared memory to the
// products, and 16 or 32 query rows fill an m16 tile but an eighth or a quarter of a tcgen05 one:
// such a kernel (codes converted into shared memory, o in tensor memory) was built and took 511 us
// where this takes 398, its hand-offs between converting, multiplying and weighting warps alone
// 3100 cycles a tile of 128 slots.  Products of unconverted codes, with queries and weights as sums of e4m3
// terms, have not been tried.
//
// What bounds it (one GB300, D = 128): memory where few query rows share a key head, and then the
// ends of the launch (its start 2 us, CTAs that end up to a tenth apart, the join 6.5 us); above
// some 16 rows a key head the products: a scheduler has two warps to choose from, the tensor pipe
// is active 45 % of the time and conversions take a third of the issue slots.
//   1 request of 131072 slots, 64 heads on 8:          55 us, 4.9 TB/s (6.7 TB/s a slot more)
//   64 requests of 100 to 8192 slots, 32 heads on 8:   55 us, 4.5 TB/s
//   16 of 4096 to 32768, 4 rows of 64 heads on 8, f16: 120 us, 3.9 TB/s
//   32 of 100000 to 131072, 64 heads on one:           399 us, 2.4 TB/s, 0.3 PFLOP/s
//   96 requests, 512 listed slots, 64 heads on one:    22 us, list -> page -> code in turn;
//     2048 listed slots: 53 us, a tile's chain of dependent instructions
#include "spin_kv_attend.cuh"

namespace spin {

constexpr int kAtWarps = 4;      // warps of a CTA: each takes every fourth tile of a segment
constexpr int kAtThreads = 32 * kAtWarps;
constexpr int kAtTile = 32;      // slots a warp works on at a time
constexpr int kAtStages = 2;     // tiles in a warp's ring
constexpr int kAtUnit = 64;      // slots in a unit of work
// Starting a job costs about as much as this many units (its queries, its first pages and tiles,
// the merge of its warps: 4 us beside 1.1 us a unit with the GPU full).
constexpr int kAtJobUnits = 4;
// A job is split unless whole jobs cost at most this many units more on the busiest CTA: the
// joining launch costs about as much (6.5 us; a unit takes 1.1 us with the GPU full,
// less where it is not).  No value is best everywhere: with 5, lists of 64-wide heads took 46.7 us
// instead of 40, and 40 requests of mixed lengths 33.9 instead of 37.8.  The host knows max_slots and not
// the lengths, so that short contexts under a large max_slots are divided for nothing: 64 requests
// of 100 to 700 slots, 64 heads on one, 23 us under 700 and 29 under 131072 (a launch of its own, cold
// cache).
constexpr int kAtSplitGain = 12;

// ------------------------------------------------------------------------ small helpers
// D += A B, A 16 x 16 row-major, B 16 x 8 column-major, f16 in, fp32 sums.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint4 a, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}

// -------------------------------------------------------------------- shared-memory tiles
// A tile is 32 rows (slots) of D bytes in lines of 128 bytes, 16-byte chunk x of row `row` at
// the position below.  The swizzles make both fragment reads free of bank conflicts: keys are read
// by quads (four neighbouring chunks of one row, eight rows a warp), values by one chunk of every
// second row.
template <int D> __device__ __forceinline__ uint32_t key_at(int row, int x) {
    if constexpr (D == 64) return (uint32_t)(row * 64 + x * 16);
    else return (uint32_t)(row * D + (x >> 3) * 128 + (((x & 7) ^ ((row & 1) << 2)) << 4));
}
template <int D> __device__ __forceinline__ uint32_t value_at(int row, int x) {
    if constexpr (D == 64) return (uint32_t)((row >> 1) * 128 + (((((row & 1) << 2) | x) ^ (row & 6)) << 4));
    else return (uint32_t)(row * D + (x >> 3) * 128 + (((x & 7) ^ (row & 6)) << 4));
}

// Rows 32 / (D / 16) apart keep their place in a line of keys; the value swizzle flips these bits.
template <int D> __device__ __forceinline__ constexpr uint32_t value_flip(int i) {
    return D == 128 ? (uint32_t)(i & 1) << 6 : D == 256 ? (uint32_t)(i & 3) << 5 : 0u;
}

template <int D, bool SPARSE> struct AtStage {  // byte offsets in a stage
    // codes of keys and values, then words.  With a list: per slot the key scale, value scale, log2
    // of the value scale, its reciprocal (before those are known: the mask of live slots, at kMask).
    // Without: key scale, value scale and mask of the tile's page.
    static constexpr int kValues = kAtTile * D, kKs = 2 * kAtTile * D, kVs = kKs + (SPARSE ? 128 : 4),
                         kLv = kVs + 128, kIv = kLv + 128, kMask = SPARSE ? kIv : kVs + 4;
    static constexpr int kBytes = kKs + (SPARSE ? 512 : 128);
};

// CTAs on an SM: three where registers and shared memory allow
template <int D, int MT, bool SPLIT> constexpr int at_ctas() { return D == 256 ? 1 : MT == 2 || (SPLIT && D == 128) ? 2 : 3; }

template <int D, int MT, bool SPLIT, bool SPARSE> struct AtSmem {
    static constexpr int kRows = 16 * MT;
    static constexpr int kRing = kAtWarps * kAtStages * AtStage<D, SPARSE>::kBytes;
    static constexpr int kMerge = kAtWarps * kRows * D * 4;          // shares the ring's memory
    static constexpr int kMain = kRing > kMerge ? kRing : kMerge;
    static constexpr int kQ = MT * (SPLIT ? 2 : 1) * (D / 16) * 512;  // query fragments
    static constexpr int kNan = SPARSE ? 0 : D * 4;                   // first NaN taken out, of each dimension
    static constexpr int kBytes = kMain + kQ + kRows * 8 + 2 * kAtWarps * kRows * 4 + 128 + kNan;
};

// Merged rows in shared memory: float4 f of a row is kept at f ^ rot, so that the eight lanes of
// a store phase (two rows, four column groups) hit different banks.
template <int D> __device__ __forceinline__ int merge_at(int row, int f) {
    if constexpr (D == 64) return (f & ~3) | ((f & 3) ^ (((f >> 3) & 1) + 2 * (row & 1)));
    else return (f & ~7) | ((f & 7) ^ (((f >> 3) & 3) + 4 * (row & 1)));
}

// --------------------------------------------------------------------------- the kernel
template <typename T, int D, int MT, bool SPARSE>
__global__ void __launch_bounds__(kAtThreads, at_ctas<D, MT, std::is_same<T, float>::value>())
kv_attend_kernel(const __grid_constant__ spin_kv_config cfg, const __grid_constant__ KvAttendArgs a, AtPlan plan) {
    pdl_wait();
    constexpr bool SPLIT = std::is_same<T, float>::value;
    constexpr bool QREG = MT == 1 && !SPLIT && D <= 128;  // query fragments stay in registers
    using L = AtSmem<D, MT, SPLIT, SPARSE>;
    using St = AtStage<D, SPARSE>;
    constexpr int NT = D / 8;       // column tiles of o
    constexpr int KS = D / 16;      // contraction steps of q . k
    extern __shared__ __align__(128) unsigned char smem[];
    uint4* sQ = reinterpret_cast<uint4*>(smem + L::kMain);
    float* sQs = reinterpret_cast<float*>(smem + L::kMain + L::kQ);
    int* sN = reinterpret_cast<int*>(sQs + L::kRows);
    float* sM = reinterpret_cast<float*>(sN + L::kRows);
    float* sL = sM + kAtWarps * L::kRows;
    int64_t* sScan = reinterpret_cast<int64_t*>(sL + kAtWarps * L::kRows);
    int* sNan = reinterpret_cast<int*>(sScan + 16);  // per dimension, the first slot of a NaN that only some rows see
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, g8 = lane >> 2, t4 = lane & 3;
    const int H = cfg.n_heads, kvh = cfg.kv_heads, d = cfg.head_dim, group = H / kvh;
    const int rows = SPARSE ? 1 : a.rows, M = group * rows;
    const float ninf = __uint_as_float(0xff800000u);

    using Walk = AtWalk<SPARSE, kAtUnit, kAtJobUnits>;
    Walk walk;
    walk.template start<kAtWarps>(cfg, a, plan, sScan);
    AtSegment seg;
    while (walk.next(cfg, a, plan, seg)) {
        const int v = seg.v, g = seg.g, len = seg.len;
        const int64_t b = SPARSE ? v / a.rows : v;
        const int64_t br0 = SPARSE ? v : (int64_t)v * a.rows;  // first (request, row)
        const int m0 = seg.mc * L::kRows, mrows = min(L::kRows, M - m0);

        // ---- this warp's tiles: tile0 + wid, + kAtWarps, ... below tile1
        const int tile0 = seg.u0 * (kAtUnit / kAtTile);
        const int tile1 = min(seg.u1 * (kAtUnit / kAtTile), (len + kAtTile - 1) / kAtTile);
        const int nt = max(0, (tile1 - tile0 - wid + kAtWarps - 1) / kAtWarps);
        const uint32_t ring = smem_u32(smem) + (uint32_t)(wid * kAtStages * St::kBytes);
        const int32_t* table = a.block_table + b * a.bt_stride;
        const int row_n = SPARSE ? row_slots(a, br0, cfg.max_slots) : 0;
        const int64_t row_bytes = (int64_t)kvh * d;

        // Pages are read as many tiles ahead of the copies that need them as the ring holds, list
        // entries one more; they are looked at when they are needed, not when they are read, so that
        // nothing waits for them in between.
        auto entry = [&](int k) -> int {  // slot of this lane in the warp's k-th tile, -1: none; unchecked with a list
            const int i = (tile0 + wid + k * kAtWarps) * kAtTile + lane;
            if constexpr (SPARSE) return k < nt && i < a.top_k ? a.list[(int64_t)v * a.top_k + i] : -1;
            else return k < nt && i < len ? i : -1;
        };
        auto listed = [&](int i) -> int {
            if (i >= 0 && i < row_n) return i;
            if (i != -1) set_status(a.status, SPIN_STATUS_BAD_LIST);
            return -1;
        };
        auto page_at = [&](int i) -> int { return i >= 0 ? table[i >> 6] : -1; };  // unchecked
        int e[SPARSE ? kAtStages + 1 : 1], p[kAtStages];
        if constexpr (SPARSE) {
#pragma unroll
            for (int i = 0; i <= kAtStages; ++i) e[i] = entry(i);
#pragma unroll
            for (int i = 0; i < kAtStages; ++i) e[i] = listed(e[i]);
        }
#pragma unroll
        for (int i = 0; i < kAtStages; ++i) p[i] = page_at(SPARSE ? e[SPARSE ? i : 0] : entry(i));

        constexpr int CH = D / 16;             // 16-byte chunks of a row
        constexpr int RS = 32 / CH;            // rows a warp copies at a time
        const int crow = lane / CH, cx = lane % CH;
        const uint32_t kdst = ring + key_at<D>(crow, cx), vdst = ring + St::kValues + value_at<D>(crow, cx);
        const bool in_row = 16 * cx < d;
        const int64_t lane_src = (SPARSE ? 0 : crow * row_bytes) + (int64_t)g * d + 16 * cx;
        auto issue = [&](int k) {  // the k-th tile's copies into its stage
            if (k < nt) {
                const uint32_t so = (uint32_t)((k % kAtStages) * St::kBytes);
                const bool slot = (SPARSE ? e[0] : entry(k)) >= 0, live = slot && p[0] >= 0 && p[0] < a.n_pages;
                if (slot && !live) set_status(a.status, SPIN_STATUS_BAD_PAGE);
                const uint32_t mask = __ballot_sync(0xffffffffu, live);
                if constexpr (SPARSE) {
                    const int64_t row = live ? (int64_t)p[0] * kBlock + (e[0] & 63) : 0;
#pragma unroll
                    for (int i = 0; i < CH; ++i) {
                        const int from = crow + RS * i;
                        const int64_t src = __shfl_sync(0xffffffffu, row, from) * row_bytes + lane_src;
                        const bool ok = ((mask >> from) & 1u) && in_row;
                        cp16(kdst + so + 512 * i, a.k_pool + (ok ? src : 0), ok);
                        cp16((vdst ^ value_flip<D>(i)) + so + 512 * i, a.v_pool + (ok ? src : 0), ok);
                    }
                    const int64_t sc = live ? (int64_t)p[0] * kvh + g : 0;
                    cp4(ring + so + St::kKs + 4 * lane, a.k_scale + sc, live);
                    cp4(ring + so + St::kVs + 4 * lane, a.v_scale + sc, live);
                } else {
                    // one page: the live slots are the first ones
                    const int n_live = __popc(mask), page = __shfl_sync(0xffffffffu, p[0], 0);
                    const int first = (tile0 + wid + k * kAtWarps) * kAtTile & (kBlock - 1);
                    const int64_t src = n_live ? ((int64_t)page * kBlock + first) * row_bytes + lane_src : 0;
                    const int64_t step = RS * row_bytes;
#pragma unroll
                    for (int i = 0; i < CH; ++i) {
                        const bool ok = crow + RS * i < n_live && in_row;
                        cp16(kdst + so + 512 * i, a.k_pool + (ok ? src + i * step : 0), ok);
                        cp16((vdst ^ value_flip<D>(i)) + so + 512 * i, a.v_pool + (ok ? src + i * step : 0), ok);
                    }
                    if (lane < 2)
                        cp4(ring + so + (lane ? St::kVs : St::kKs), (lane ? a.v_scale : a.k_scale) + (n_live ? (int64_t)page * kvh + g : 0),
                            n_live > 0);
                }
                if (lane == 0)
                    asm volatile("st.shared.u32 [%0], %1;" ::"r"(ring + so + St::kMask), "r"(mask) : "memory");
#pragma unroll
                for (int i = 0; i + 1 < kAtStages; ++i) p[i] = p[i + 1];
                if constexpr (SPARSE) {
#pragma unroll
                    for (int i = 0; i < kAtStages; ++i) e[i] = e[i + 1];
                    e[kAtStages - 1] = listed(e[kAtStages - 1]);
                    p[kAtStages - 1] = page_at(e[kAtStages - 1]);
                    e[kAtStages] = entry(k + kAtStages + 1);
                } else {
                    p[kAtStages - 1] = page_at(entry(k + kAtStages));
                }
            }
            cp_commit();
        };
#pragma unroll 1
        for (int k = 0; k < kAtStages; ++k) issue(k);

        if (!SPARSE && rows > 1)
            for (int i = tid; i < D; i += kAtThreads) sNan[i] = 0x7fffffff;

        // ---- queries: row m is (row m / group, head g * group + m % group), scaled by a power
        // of two and rounded to f16, laid out as the fragments read them
        // (16 neighbouring values a thread, D / 16 threads a row)
#pragma unroll 1
        for (int it = tid; it < L::kRows * (D / 16); it += kAtThreads) {
            const int m = it / (D / 16), ch = it % (D / 16);
            const int mr = (m0 + m) / group;
            const int64_t br = br0 + mr;
            const uint4* qp = reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(a.q) +
                                                             (br * H + (int64_t)g * group + (m0 + m - mr * group)) * d + 16 * ch);
            constexpr int QN = 16 * (int)sizeof(T) / 16;
            uint4 qv[QN];
#pragma unroll
            for (int k = 0; k < QN; ++k) qv[k] = m < mrows && 16 * ch < d ? qp[k] : make_uint4(0, 0, 0, 0);
            float x[16], amax = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                x[i] = to_f(reinterpret_cast<const T*>(qv)[i]);
                amax = fmaxf(amax, fabsf(x[i]));
            }
#pragma unroll
            for (int o = D / 32; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            // amax in [2^k, 2^(k+1)) -> [2^14, 2^15); 2^(14 - k) within [2^-113, 2^126]
            const int k = max(-112, (int)(__float_as_uint(amax) >> 23) - 127);
            const float f = __uint_as_float((uint32_t)(127 + 14 - k) << 23);
            if (ch == 0) {
                sQs[m] = __uint_as_float((uint32_t)max(1, 127 - 14 + k) << 23) * (cfg.softmax_scale * 1.4426950408889634f);
                sN[m] = !SPARSE && m < mrows ? row_slots(a, br, cfg.max_slots) : 0x7fffffff;
            }
            // dims 64c + 16t + 4s + {0, 1} of row m are the pair k = 2t of contraction step 4c + s,
            // {2, 3} the pair k = 2t + 8; here ch = 4c + t
            uint32_t* to = reinterpret_cast<uint32_t*>(sQ) +
                           (((m >> 4) * KS + (ch >> 2) * 4) * 32 + (m & 7) * 4 + (ch & 3)) * 4 + ((m & 15) >> 3);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t hi = pack_f16(x[2 * i] * f, x[2 * i + 1] * f);
                to[(i >> 1) * 128 + 2 * (i & 1)] = hi;
                if constexpr (SPLIT) {
                    const float2 h = unpack_f16(hi);
                    to[MT * KS * 128 + (i >> 1) * 128 + 2 * (i & 1)] = pack_f16(x[2 * i] * f - h.x, x[2 * i + 1] * f - h.y);
                }
            }
        }
        __syncthreads();
        uint4 qr[QREG ? KS : 1];
        if constexpr (QREG) {
#pragma unroll
            for (int s = 0; s < KS; ++s) qr[s] = sQ[s * 32 + lane];
        }
        float qs[MT][2];
        int nlim[MT][2], nmin = 0x7fffffff, nseen = 0x7fffffff;  // shortest row; of those that see this segment
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                qs[i][x] = sQs[16 * i + 8 * x + g8];
                nlim[i][x] = sN[16 * i + 8 * x + g8];
                nmin = min(nmin, nlim[i][x]);
                if (nlim[i][x] > kAtUnit * seg.u0) nseen = min(nseen, nlim[i][x]);
            }
        nmin = __reduce_min_sync(0xffffffffu, nmin);
        nseen = __reduce_min_sync(0xffffffffu, nseen);

        float o[MT][NT][4], mx[MT][2], lsum[MT][2];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            mx[i][0] = mx[i][1] = ninf;
            lsum[i][0] = lsum[i][1] = 0.0f;
#pragma unroll
            for (int n = 0; n < NT; ++n) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.0f;
        }

        bool far = false;   // a reference of kAtFar or more
        for (int k = 0; k < nt; ++k) {
            cp_wait<kAtStages - 1>();
            __syncwarp();
            const uint32_t st = ring + (uint32_t)((k % kAtStages) * St::kBytes);
            const int slot0 = (tile0 + wid + k * kAtWarps) * kAtTile;
            uint32_t mask;
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(mask) : "r"(st + St::kMask) : "memory");

            // ---- scores of 32 slots: column tile j holds slots 8j ..
            float s[MT][4][4];
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i][j][0] = s[i][j][1] = s[i][j][2] = s[i][j][3] = 0.0f;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                uint4 qf[QREG ? 1 : MT * (SPLIT ? 2 : 1)][QREG ? 1 : 4];
                if constexpr (!QREG) {
#pragma unroll
                    for (int i = 0; i < MT * (SPLIT ? 2 : 1); ++i)
#pragma unroll
                        for (int w = 0; w < 4; ++w) qf[i][w] = sQ[(i * KS + 4 * c + w) * 32 + lane];
                }
                uint32_t kw[4][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint4 kc = lds128(st + key_at<D>(8 * j + g8, 4 * c + t4));
                    kw[j][0] = kc.x, kw[j][1] = kc.y, kw[j][2] = kc.z, kw[j][3] = kc.w;
                }
                // (the column tiles' chains of products take turns)
#pragma unroll
                for (int w = 0; w < 4; ++w)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t b0, b1;
                        codes_to_f16(kw[j][w], b0, b1);
                        if constexpr (QREG) {
                            mma_f16(s[0][j], qr[4 * c + w], b0, b1);
                        } else {
#pragma unroll
                            for (int i = 0; i < MT; ++i) {
                                mma_f16(s[i][j], qf[i][w], b0, b1);
                                if constexpr (SPLIT) mma_f16(s[i][j], qf[MT + i][w], b0, b1);
                            }
                        }
                    }
            }

            // ---- weights: 2^(t - m) vs, where t = qs ks s; with x = t + log2 vs they are 2^(x - m)
            // and l gains them divided by vs
            const bool border = mask != 0xffffffffu || slot0 + kAtTile > nmin;
            float top[MT][2], lv[SPARSE ? 8 : 1], iv[SPARSE ? 8 : 1], c[MT][2];
            bool odd = false;  // a value scale whose logarithm does not stand for it
            if constexpr (SPARSE) {
                uint32_t u;
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(u) : "r"(st + St::kVs + 4 * lane) : "memory");
                const float v_ = __uint_as_float(u);
                const bool fine = in_log_range(v_) || !((mask >> lane) & 1u);
                odd = __any_sync(0xffffffffu, !fine);
                const float lg = scale_log2(v_);
                __syncwarp();  // every lane has read the mask
                asm volatile("st.shared.f32 [%0], %1;" ::"r"(st + St::kLv + 4 * lane), "f"(lg) : "memory");
                asm volatile("st.shared.f32 [%0], %1;" ::"r"(st + St::kIv + 4 * lane), "f"(kAtSumUnit * (in_log_range(v_) ? __frcp_rn(v_) : ex2(-lg))) : "memory");
                __syncwarp();
                float ks[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t o4 = 4 * (8 * j + 2 * t4);
                    const uint2 x = lds64(st + St::kKs + o4), y = lds64(st + St::kLv + o4), z = lds64(st + St::kIv + o4);
                    ks[2 * j] = __uint_as_float(x.x), ks[2 * j + 1] = __uint_as_float(x.y);
                    lv[2 * j] = __uint_as_float(y.x), lv[2 * j + 1] = __uint_as_float(y.y);
                    iv[2 * j] = __uint_as_float(z.x), iv[2 * j + 1] = __uint_as_float(z.y);
                }
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    top[i][0] = top[i][1] = ninf;
                    c[i][0] = c[i][1] = 1.0f;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int col = 2 * j + (x & 1), r = x >> 1;
                            float y = fmaf(s[i][j][x] * ks[col], qs[i][r], lv[col]);
                            if (border && !((mask >> (8 * j + 2 * t4 + (x & 1))) & 1u)) y = ninf;
                            s[i][j][x] = y;
                            top[i][r] = fmaxf(top[i][r], y);
                        }
                }
            } else {
                uint32_t u, w;
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(u) : "r"(st + St::kKs) : "memory");
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(st + St::kVs) : "memory");
                const float ks = __uint_as_float(u), v_ = __uint_as_float(w);
                odd = !in_log_range(v_);
                lv[0] = scale_log2(v_);
                iv[0] = kAtSumUnit * (odd ? ex2(-lv[0]) : __frcp_rn(v_));
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int r = 0; r < 2; ++r) c[i][r] = qs[i][r] * ks;
                if (border) {
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
#pragma unroll
                                for (int x = 2 * r; x < 2 * r + 2; ++x) {
                                    const int at_slot = 8 * j + 2 * t4 + (x & 1);
                                    const bool ok = ((mask >> at_slot) & 1u) && slot0 + at_slot < nlim[i][r];
                                    s[i][j][x] = ok ? s[i][j][x] * c[i][r] : ninf;
                                }
                            c[i][r] = 1.0f;
                        }
                }
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    top[i][0] = top[i][1] = ninf;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int x = 0; x < 4; ++x) top[i][x >> 1] = fmaxf(top[i][x >> 1], s[i][j][x] * c[i][x >> 1]);
                    top[i][0] += lv[0];
                    top[i][1] += lv[0];
                }
            }
            bool move = false;
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    top[i][r] = fmaxf(top[i][r], __shfl_xor_sync(0xffffffffu, top[i][r], 1));
                    top[i][r] = fmaxf(top[i][r], __shfl_xor_sync(0xffffffffu, top[i][r], 2)) - kAtTop;
                    move |= top[i][r] > mx[i][r] + kAtSlack;
                }
            if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float now = fmaxf(mx[i][r], top[i][r]);
                        const float f = now == ninf ? 1.0f : ex2(mx[i][r] - now);
                        mx[i][r] = now;
                        far |= now != ninf && fabsf(now) >= kAtFar;
                        lsum[i][r] *= f;
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            o[i][n][2 * r] *= f;
                            o[i][n][2 * r + 1] *= f;
                        }
                    }
                far = __any_sync(0xffffffffu, far);
            }
            if (far) {  // the exponents, rounded as the maximum was and bounded
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float m = mx[i][r] == ninf ? 0.0f : mx[i][r];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int x = 2 * r; x < 2 * r + 2; ++x) {
                                const float y = SPARSE ? s[i][j][x] : __fadd_rn(__fmul_rn(s[i][j][x], c[i][r]), lv[0]);
                                const float e = __fsub_rn(y, m);
                                s[i][j][x] = e > kAtTop + kAtSlack ? kAtTop + kAtSlack : e;  // (NaN stays)
                            }
                        c[i][r] = 1.0f;
                    }
            }
            uint4 pw[MT][SPLIT ? 2 : 1][2];
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                float bias[2], add[2] = {0.0f, 0.0f};
#pragma unroll
                for (int r = 0; r < 2; ++r) bias[r] = far ? 0.0f : (SPARSE ? 0.0f : lv[0]) - (mx[i][r] == ninf ? 0.0f : mx[i][r]);
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int r = x >> 1;
                        const float p = ex2(SPARSE ? s[i][j][x] + bias[r] : fmaf(s[i][j][x], c[i][r], bias[r]));
                        s[i][j][x] = p;
                        add[r] = SPARSE ? fmaf(p, iv[SPARSE ? 2 * j + (x & 1) : 0], add[r]) : add[r] + p;
                    }
#pragma unroll
                for (int r = 0; r < 2; ++r) lsum[i][r] = SPARSE ? lsum[i][r] + add[r] : fmaf(add[r], iv[0], lsum[i][r]);
            }
            if (odd) {  // zero, negative, tiny, huge or NaN: the ratio of scale and power of two, for the
                        // slots that a row sees (0 x inf and 0 x NaN would reach the others)
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int at_slot = 8 * j + 2 * t4 + x;
                        uint32_t u;
                        asm volatile("ld.shared.u32 %0, [%1];"
                                     : "=r"(u)
                                     : "r"(st + St::kVs + (SPARSE ? 4 * at_slot : 0))
                                     : "memory");
                        const float v_ = __uint_as_float(u), f = in_log_range(v_) ? 1.0f : v_ * ex2(-scale_log2(v_));
#pragma unroll
                        for (int i = 0; i < MT; ++i)
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                const bool ok = !border || (((mask >> at_slot) & 1u) && (SPARSE || slot0 + at_slot < nlim[i][r]));
                                s[i][j][2 * r + x] *= ok ? f : 0.0f;
                            }
                    }
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                uint32_t ph[8], pl[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float p0 = s[i][j >> 1][2 * (j & 1)], p1 = s[i][j >> 1][2 * (j & 1) + 1];
                    ph[j] = pack_f16(p0, p1);
                    if constexpr (SPLIT) {
                        const float2 h = unpack_f16(ph[j]);
                        pl[j] = pack_f16(p0 - h.x, p1 - h.y);
                    }
                }
                pw[i][0][0] = make_uint4(ph[0], ph[1], ph[2], ph[3]);
                pw[i][0][1] = make_uint4(ph[4], ph[5], ph[6], ph[7]);
                if constexpr (SPLIT) {
                    pw[i][1][0] = make_uint4(pl[0], pl[1], pl[2], pl[3]);
                    pw[i][1][1] = make_uint4(pl[4], pl[5], pl[6], pl[7]);
                }
            }

            // A NaN code that some rows see and others do not would reach the others as 0 x NaN: such codes
            // leave the tile, and the first one's slot of each dimension is kept: a row sees a NaN of
            // that dimension if its slots reach so far.  (Rows that see nothing of the segment, the empty
            // ones of a padded batch, drop their sums instead.)
            if (!SPARSE && rows > 1 && slot0 + kAtTile > nseen) {
#pragma unroll 2
                for (int e = lane; e < kAtTile * CH; e += 32) {
                    const int row = e / CH, ch = e % CH;
                    const uint32_t at = st + St::kValues + value_at<D>(row, ch);
                    const uint4 x = lds128(at);
                    uint32_t w[4] = {x.x, x.y, x.z, x.w}, any = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) any |= (w[i] & 0x7f7f7f7fu) + 0x01010101u;
                    if (any & 0x80808080u) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t m = ((w[i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;  // bytes that are NaN
                            w[i] &= ~((m >> 7) * 0xffu);
#pragma unroll 1
                            for (uint32_t y = m; y; y &= y - 1) atomicMin(sNan + 16 * ch + 4 * i + ((__ffs(y) - 1) >> 3), slot0 + row);
                        }
                        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                                     : "memory");
                    }
                }
                __syncwarp();
            }

            // ---- o += weights x values: column n of tile i holds dim 16 n + i (of each 128; D = 64:
            // 8 n + i)
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                const int r0 = 16 * kk + 2 * t4;
                constexpr int HALVES = D == 64 ? 1 : D / 128, WORDS = D == 64 ? 2 : 4;
#pragma unroll
                for (int hh = 0; hh < HALVES; ++hh) {
                    uint32_t vw[4][4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int row = r0 + (q & 1) + 8 * (q >> 1);
                        if constexpr (D == 64) {
                            const uint2 x = lds64(st + St::kValues + value_at<D>(row, g8 >> 1) + 8 * (g8 & 1));
                            vw[q][0] = x.x;
                            vw[q][1] = x.y;
                        } else {
                            const uint4 x = lds128(st + St::kValues + value_at<D>(row, g8 + 8 * hh));
                            vw[q][0] = x.x;
                            vw[q][1] = x.y;
                            vw[q][2] = x.z;
                            vw[q][3] = x.w;
                        }
                    }
#pragma unroll
                    for (int w = 0; w < WORDS; ++w) {
                        uint32_t b0[4], b1[4];
                        codes_to_f16(__byte_perm(vw[0][w], vw[1][w], 0x5140), b0[0], b0[1]);
                        codes_to_f16(__byte_perm(vw[0][w], vw[1][w], 0x7362), b0[2], b0[3]);
                        codes_to_f16(__byte_perm(vw[2][w], vw[3][w], 0x5140), b1[0], b1[1]);
                        codes_to_f16(__byte_perm(vw[2][w], vw[3][w], 0x7362), b1[2], b1[3]);
#pragma unroll
                        for (int y = 0; y < 4; ++y)
#pragma unroll
                            for (int i = 0; i < MT; ++i) {
                                mma_f16(o[i][16 * hh + 4 * w + y], pw[i][0][kk], b0[y], b1[y]);
                                if constexpr (SPLIT) mma_f16(o[i][16 * hh + 4 * w + y], pw[i][SPLIT][kk], b0[y], b1[y]);
                            }
                    }
                }
            }
            __syncwarp();
            issue(k + kAtStages);
        }
        if (walk.done(plan)) pdl_trigger();
        cp_wait<0>();
        __syncthreads();   // the ring is free: the warps' results go there

        // ---- merge the warps
        float* sO = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = 16 * i + 8 * r + g8;
                lsum[i][r] += __shfl_xor_sync(0xffffffffu, lsum[i][r], 1);
                lsum[i][r] += __shfl_xor_sync(0xffffffffu, lsum[i][r], 2);
                if (t4 == 0) {
                    sM[wid * L::kRows + row] = mx[i][r];
                    sL[wid * L::kRows + row] = lsum[i][r];
                }
                float4* dst = reinterpret_cast<float4*>(sO + (wid * L::kRows + row) * D);
                constexpr int PER = D == 64 ? 8 : 16;  // tiles that one column spans
#pragma unroll
                for (int hh = 0; hh < NT / PER; ++hh)
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int q = 0; q < PER / 4; ++q) {
                            const int f = 32 * hh + (2 * t4 + x) * (PER / 4) + q, n = PER * hh + 4 * q;
                            dst[merge_at<D>(row, f)] = make_float4(o[i][n][2 * r + x], o[i][n + 1][2 * r + x],
                                                                   o[i][n + 2][2 * r + x], o[i][n + 3][2 * r + x]);
                        }
            }
        __syncthreads();
        const bool whole = seg.u0 == 0 && seg.u1 == seg.units;
        float* rec = Walk::record(plan, seg, D);
        if (tid == 0) walk.own(plan, seg);
#pragma unroll 1
        for (int e = tid; e < mrows * (D / 4); e += kAtThreads) {
            const int m = e / (D / 4), f = e % (D / 4);
            float top = ninf;
#pragma unroll
            for (int w = 0; w < kAtWarps; ++w) top = fmaxf(top, sM[w * L::kRows + m]);
            float l = 0.0f;
            float4 acc = make_float4(0, 0, 0, 0);
#pragma unroll
            for (int w = 0; w < kAtWarps; ++w) {
                const float mw = sM[w * L::kRows + m];
                const float c = mw == ninf ? 0.0f : ex2(mw - top);
                const float4 x = reinterpret_cast<const float4*>(sO + (w * L::kRows + m) * D)[merge_at<D>(m, f)];
                // a warp without a slot of this row has l = 0, and sums that may be 0 x NaN; one that
                // saw only NaN scores has l = NaN, which stays
                l = fmaf(c, sL[w * L::kRows + m], l);
                if (mw != ninf) {
                    acc.x = fmaf(c, x.x, acc.x);
                    acc.y = fmaf(c, x.y, acc.y);
                    acc.z = fmaf(c, x.z, acc.z);
                    acc.w = fmaf(c, x.w, acc.w);
                }
            }
            if (!SPARSE && rows > 1) {
                const int n = sN[m];
                const int4 first = reinterpret_cast<const int4*>(sNan)[f];
                if (first.x < n) acc.x = __uint_as_float(0x7fffffffu);
                if (first.y < n) acc.y = __uint_as_float(0x7fffffffu);
                if (first.z < n) acc.z = __uint_as_float(0x7fffffffu);
                if (first.w < n) acc.w = __uint_as_float(0x7fffffffu);
            }
            if (whole) {
                const int64_t bh = (br0 + (m0 + m) / group) * H + (int64_t)g * group + (m0 + m) % group;
                if (4 * f < d) store4(reinterpret_cast<T*>(a.out) + bh * d + 4 * f, row_out(acc, l));
                if (a.lse && f == 0) a.lse[bh] = row_lse(top, l);
            } else {
                reinterpret_cast<float4*>(rec + m * D)[f] = acc;
                if (f == 0) {
                    rec[L::kRows * D + 2 * m] = top;
                    rec[L::kRows * D + 2 * m + 1] = l;
                }
            }
        }
        __syncthreads();
    }
    write_empty<T, SPARSE>(cfg, a, plan);
}

// ------------------------------------------------------------------------------ host side
static int at_dim(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }
// Two records for every CTA of any variant, 32 rows each at most.
size_t kv_attend_workspace_bytes(const spin_kv_config& cfg, int, int) {
    const int D = at_dim(cfg.head_dim);
    const size_t G = kAtMostCtas * (size_t)device_sm_count();
    return (G * sizeof(int4) + 255) / 256 * 256 + G * 2 * 32 * (size_t)(D + 2) * sizeof(float);
}

// units of the longest job; CTAs that the GPU holds; whether jobs are divided
static int64_t at_units(const spin_kv_config& cfg, const KvAttendArgs& a) {
    return ((a.list ? a.top_k : cfg.max_slots) + kAtUnit - 1) / kAtUnit;
}
template <int D, int MT, bool SPLIT> static int64_t at_room() {
    const int sms = device_sm_count();
    return at_ctas<D, MT, SPLIT>() * (int64_t)(sms < kAtMostSms ? sms : kAtMostSms);
}
static bool at_split(int64_t jobs, int64_t most, int64_t per, int64_t ctas) {
    // whole jobs: ceil(jobs / ctas) * most units on the busiest CTA; split: jobs * most / ctas
    const int64_t ranks = ctas / per;
    return ranks > 0 && (jobs + ctas - 1) / ctas * most > jobs * most / (ranks * per) + kAtSplitGain;
}

template <typename T, int D, int MT, bool SPARSE>
static cudaError_t launch_at(const spin_kv_config& cfg, const KvAttendArgs& a, cudaStream_t s) {
    constexpr bool SPLIT = std::is_same<T, float>::value;
    using L = AtSmem<D, MT, SPLIT, SPARSE>;
    auto k = kv_attend_kernel<T, D, MT, SPARSE>;
    static std::atomic<uint64_t> allowed;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), L::kBytes, allowed);
    if (e != cudaSuccess) return e;
    const int M = cfg.n_heads / cfg.kv_heads * (SPARSE ? 1 : a.rows);
    AtPlan p;
    p.mchunks = (M + L::kRows - 1) / L::kRows;
    p.n_virtual = SPARSE ? cfg.n_req * a.rows : cfg.n_req;
    p.per = cfg.kv_heads * p.mchunks;
    p.crows = L::kRows;
    const int64_t jobs = (int64_t)p.n_virtual * p.per, most = at_units(cfg, a), ctas = at_room<D, MT, SPLIT>();
    const int64_t ranks = ctas / p.per, most_ranks = p.n_virtual * (most + kAtJobUnits + kAtMinCost - 1) / kAtMinCost;
    p.split = at_split(jobs, most, p.per, ctas);
    const int G = (int)(p.split ? (most_ranks < ranks ? most_ranks : ranks) * p.per : jobs < ctas ? jobs : ctas);
    p.ranks = G / p.per;
    p.by_job = jobs <= G;
    p.owner = reinterpret_cast<int4*>(a.workspace);
    p.rec = a.workspace + ((size_t)kAtMostCtas * device_sm_count() * sizeof(int4) + 255) / 256 * 64;
    e = launch_pdl(k, dim3(G), dim3(kAtThreads), L::kBytes, s, nullptr, 0, cfg, a, p);
    if (e != cudaSuccess || !p.split) return e;
    return launch_pdl(kv_attend_join_kernel<T, D>, dim3(p.by_job ? (unsigned)jobs : G, M < L::kRows ? M : L::kRows),
                      dim3(32 * kJoinWarps), 0, s, nullptr, 0, cfg, a, p, SPARSE ? 1 : a.rows);
}

template <typename T, int D, int MT>
static cudaError_t launch_list(const spin_kv_config& cfg, const KvAttendArgs& a, cudaStream_t s) {
    return a.list ? launch_at<T, D, MT, true>(cfg, a, s) : launch_at<T, D, MT, false>(cfg, a, s);
}

// One row tile (16 query rows of a key/value head) a warp, or two where there are more rows: every
// converted code then feeds two products (64 heads on one key head 396 us, 527 with one tile; four
// rows of 64 heads on 8 119 and 154 us), at two CTAs an SM instead of three.  Short whole jobs that
// are all on the GPU at once take one: a tile is then half the latency (64 requests of 100 to 700
// slots, 64 heads on one: 16 and 19 us); with lists, whose tiles slow each other more, where each
// job has an SM to itself (512 slots each: 4 requests 13 and 14.5 us, 96 requests 23.4 and 22 us).
template <typename T, int D>
static cudaError_t launch_rows(const spin_kv_config& cfg, const KvAttendArgs& a, cudaStream_t s) {
    const int64_t rows = a.list ? 1 : a.rows, M = cfg.n_heads / cfg.kv_heads * rows;
    const int64_t per = cfg.kv_heads * ((M + 15) / 16), jobs = (a.list ? cfg.n_req * (int64_t)a.rows : cfg.n_req) * per;
    const int64_t ctas = at_room<D, 1, std::is_same<T, float>::value>();
    if (M <= 16 || (jobs <= (a.list ? device_sm_count() : ctas) && !at_split(jobs, at_units(cfg, a), per, ctas))) return launch_list<T, D, 1>(cfg, a, s);
    return launch_list<T, D, 2>(cfg, a, s);
}

template <typename T>
static cudaError_t launch_typed(const spin_kv_config& cfg, const KvAttendArgs& a, cudaStream_t s) {
    const int D = at_dim(cfg.head_dim);
    if (D == 256) return launch_list<T, 256, 1>(cfg, a, s);  // (a 256-wide output leaves registers for one tile)
    return D == 128 ? launch_rows<T, 128>(cfg, a, s) : launch_rows<T, 64>(cfg, a, s);
}

cudaError_t launch_kv_attend(const spin_kv_config& cfg, const KvAttendArgs& a, cudaStream_t s) {
    switch (cfg.dtype) {
        case SPIN_DTYPE_F32: return launch_typed<float>(cfg, a, s);
        case SPIN_DTYPE_BF16: return launch_typed<__nv_bfloat16>(cfg, a, s);
        default: return launch_typed<__half>(cfg, a, s);
    }
}

}  // namespace spin
