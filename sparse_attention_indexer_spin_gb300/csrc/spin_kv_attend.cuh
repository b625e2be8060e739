// spin_kv_attend.cuh -- parts of the attention over the 8-bit KV cache: small helpers, the division of
// the work over CTAs, and the join of divided jobs.
//
// What runs once per CTA or segment is kept small in code (loops not unrolled, divisions out of
// line): its instructions are fetched cold, and with everything unrolled a CTA's first tile started
// 8 us after its launch.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "spin_common.cuh"
#include "spin_internal.h"

namespace spin {

constexpr float kAtTop = 12.0f;  // log2 of the largest weight when the reference is set
constexpr float kAtSlack = 3.0f; // a maximum may exceed that by this much before the reference moves
constexpr float kAtFar = 1048576.0f;  // references from here on take care of the exponents' roundings
// The weights' sum l is kept times 2^-20.  A slot adds up to 2^(12 + 3) / vs to l, vs >= 2^-100 as the
// reference counts it: 2^24 slots reach 2^139, times 2^-20 2^119.  The largest weight's slot alone adds 2^12 / vs
// >= 2^-88, so that l never underflows either.
constexpr float kAtSumUnit = 9.5367431640625e-7f;

// ------------------------------------------------------------------------ small helpers
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Value scales that their logarithm stands for: positive and neither tiny nor huge.  The others
// count as 2^-100 .. 2^100 in the reference, times a ratio.
__device__ __forceinline__ bool in_log_range(float v) { return v >= 7.888609e-31f && v <= 1.2676506e30f; }
__device__ __forceinline__ float scale_log2(float v) { return fminf(fmaxf(lg2(fabsf(v)), -100.0f), 100.0f); }

// Four e4m3 codes as two pairs of f16 (exact).
__device__ __forceinline__ void codes_to_f16(uint32_t c, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(c));
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

__device__ __forceinline__ float2 unpack_f16(uint32_t u) {
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

// 16 (or 4) bytes global -> shared, zeros instead where !live.
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool live) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(live ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
template <typename T> __device__ __forceinline__ float to_f(T x);
template <> __device__ __forceinline__ float to_f(float x) { return x; }
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <> __device__ __forceinline__ float to_f(__half x) { return __half2float(x); }

__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__half* p, float4 v) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_f16(v.x, v.y), pack_f16(v.z, v.w));
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// ------------------------------------------------------------------------- work division
// A job is a (request, or with a list request row; key/value head; chunk of query rows), its work a
// row of units of UNIT slots, its cost JOB_UNITS and then its units.  A split launch lays the
// requests' costs end to end and divides them evenly into ranks; `per` CTAs, one for each head and
// chunk, share a rank, so that a page's heads, which lie side by side, are read at about the same
// time.
struct AtPlan {
    int split;      // jobs may be divided over ranks; else CTAs take whole jobs
    int crows;      // query rows in a chunk
    int mchunks;    // chunks of query rows per key/value head
    int per;        // jobs of a request: kv_heads * mchunks
    int n_virtual;  // requests, or with lists request rows
    int ranks;      // gridDim.x / per
    int by_job;     // `owner` has an entry per job, else one per CTA
    float* rec;     // partial results, two records per CTA: crows x D sums, then (reference, l) of each row
    int4* owner;    // a divided job (request, job of the request), its first rank and number of pieces (by_job:
                    // of this job; else: of the job that this CTA begins and does not finish); w = 0: none
};

constexpr int kAtMinCost = 4;      // cost a rank takes at least, in units
constexpr int kAtMostCtas = 3;     // CTAs on an SM
constexpr int kAtMostSms = 512;    // bounds the pieces of a job
constexpr int kAtMostPieces = kAtMostCtas * kAtMostSms;

// Slots of request b's longest row (its own row's with a list); bad lengths count as 0.
__device__ __forceinline__ int row_slots(const KvAttendArgs& a, int64_t br, int max_slots) {
    const int n = a.n_slots[br];
    if (n < 0 || n > max_slots) {
        set_status(a.status, SPIN_STATUS_BAD_N);
        return 0;
    }
    return n;
}

template <bool SPARSE>
__device__ __forceinline__ int virtual_len(const spin_kv_config& cfg, const KvAttendArgs& a, int v) {
    if constexpr (SPARSE) {
        return row_slots(a, v, cfg.max_slots) > 0 ? a.top_k : 0;
    } else {
        int n = 0;
#pragma unroll 1
        for (int r = 0; r < a.rows; ++r) n = max(n, row_slots(a, (int64_t)v * a.rows + r, cfg.max_slots));
        return n;
    }
}

__device__ __forceinline__ int64_t warp_incl_scan64(int64_t v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t t = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += t;
    }
    return v;
}

// Inclusive scan over a CTA of WARPS warps; *total is the sum.
template <int WARPS>
__device__ __forceinline__ int64_t cta_incl_scan64(int64_t v, int64_t* smem, int64_t* total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int64_t s = warp_incl_scan64(v);
    if (lane == 31) smem[w] = s;
    __syncthreads();
    int64_t all = 0;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) {
        if (i < w) s += smem[i];
        all += smem[i];
    }
    __syncthreads();
    *total = all;
    return s;
}

static __device__ __noinline__ int2 div_mod(int a, int b) { return make_int2(a / b, a % b); }
// a / b for 0 <= a, 0 < b (a long division takes some 700 cycles, and few totals need one)
static __device__ __noinline__ int64_t quotient(int64_t a, int64_t b) {
    return (uint64_t)(a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// `total` cut into `ranks` parts that differ by one at most, the longer ones first.
struct AtCut {
    int64_t each, more;   // length of the shorter parts; how many are one longer
    __device__ __forceinline__ void set(int64_t total, int64_t ranks) {
        each = quotient(total, ranks);
        more = total - each * ranks;
    }
    __device__ __forceinline__ int64_t begin(int64_t rank) const { return rank * each + min(rank, more); }
    __device__ __forceinline__ int64_t rank_of(int64_t x) const {
        const int64_t longer = more * (each + 1);
        return x < longer ? quotient(x, each + 1) : more + quotient(x - longer, each);
    }
};

// One segment of a CTA's work: units [u0, u1) of the job (v, g, mc).
struct AtSegment {
    int v, g, mc, len, units, u0, u1;
    int64_t cost0, span;   // split: where the job's cost begins, and its cost
};

// A CTA's walk over its segments.
template <bool SPARSE, int UNIT, int JOB_UNITS> struct AtWalk {
    int64_t total, at, end, ranks, into;
    AtCut cut;
    int job, v, len_v, rank, mine;

    __device__ __forceinline__ static int64_t cost(int len) {
        return len ? (len + UNIT - 1) / UNIT + JOB_UNITS : 0;
    }

    // By the whole CTA of WARPS warps; smem: WARPS + 3 words.
    template <int WARPS>
    __device__ __forceinline__ void start(const spin_kv_config& cfg, const KvAttendArgs& a, const AtPlan& plan, int64_t* smem) {
        constexpr int THREADS = 32 * WARPS;
        const int tid = threadIdx.x;
        const int2 place = div_mod(blockIdx.x, plan.per);
        rank = place.x;
        mine = place.y;
        total = at = end = into = 0;
        job = blockIdx.x;
        v = 0;
        len_v = -1;
        if (!plan.split) return;
        const bool one = plan.n_virtual <= THREADS;  // the first pass has every request's place
        int len = 0;
        int64_t inc = 0, sum;
#pragma unroll 1
        for (int base = 0; base < plan.n_virtual; base += THREADS) {
            const int x = base + tid;
            len = x < plan.n_virtual ? virtual_len<SPARSE>(cfg, a, x) : 0;
            inc = cta_incl_scan64<WARPS>(cost(len), smem, &sum);
            total += sum;
        }
        // every rank that takes part has some cost at least: a divided job's pieces are those of
        // consecutive ranks
        ranks = min((int64_t)plan.ranks, (total + kAtMinCost - 1) / kAtMinCost);
        if (rank < ranks) {
            cut.set(total, ranks);
            at = cut.begin(rank);
            end = cut.begin(rank + 1);
            int64_t before = 0;
#pragma unroll 1
            for (int base = 0; base < plan.n_virtual; base += THREADS) {
                const int x = base + tid;
                if (!one) {
                    len = x < plan.n_virtual ? virtual_len<SPARSE>(cfg, a, x) : 0;
                    inc = before + cta_incl_scan64<WARPS>(cost(len), smem, &sum);
                    before += sum;
                }
                if (inc > at && inc - cost(len) <= at) {
                    smem[WARPS] = x;
                    smem[WARPS + 1] = at - (inc - cost(len));
                    smem[WARPS + 2] = len;
                }
                if (before > at) break;
            }
            __syncthreads();
            v = (int)smem[WARPS];
            into = smem[WARPS + 1];
            len_v = (int)smem[WARPS + 2];
        }
        if (tid == 0 && !plan.by_job) plan.owner[blockIdx.x].w = 0;
    }

    __device__ __forceinline__ bool next(const spin_kv_config& cfg, const KvAttendArgs& a, const AtPlan& plan, AtSegment& s) {
        if (plan.split) {
#pragma unroll 1
            while (at < end) {
#pragma unroll 1
                for (;;) {
                    if (len_v < 0) len_v = virtual_len<SPARSE>(cfg, a, v);
                    if (into < cost(len_v)) break;
                    into = 0;
                    len_v = -1;
                    ++v;
                }
                s.v = v;
                s.len = len_v;
                s.units = (len_v + UNIT - 1) / UNIT;
                s.span = s.units + JOB_UNITS;
                const int2 y = div_mod(mine, plan.mchunks);
                s.g = y.x;
                s.mc = y.y;
                s.cost0 = at - into;
                const int64_t take = min(s.span - into, end - at);
                s.u0 = (int)max((int64_t)0, into - JOB_UNITS);
                s.u1 = (int)max((int64_t)0, into + take - JOB_UNITS);
                at += take;
                into += take;
                if (s.u0 != s.u1) return true;  // else the part ends before the job's first unit
            }
            return false;
        }
#pragma unroll 1
        while (job < plan.n_virtual * plan.per) {
            const int2 x = div_mod(job, plan.per), y = div_mod(x.y, plan.mchunks);
            s.v = x.x;
            s.g = y.x;
            s.mc = y.y;
            job += gridDim.x;
            s.len = virtual_len<SPARSE>(cfg, a, s.v);
            if (s.len == 0) continue;
            s.units = (s.len + UNIT - 1) / UNIT;
            s.u0 = 0;
            s.u1 = s.units;
            return true;
        }
        return false;
    }

    __device__ __forceinline__ bool done(const AtPlan& plan) const {
        return plan.split ? at >= end : job >= plan.n_virtual * plan.per;
    }

    // Once per segment: who joins the pieces of a job that this CTA begins.
    __device__ __forceinline__ void own(const AtPlan& plan, const AtSegment& s) const {
        if (!plan.split || s.u0 != 0) return;
        int4 o = make_int4(s.v, mine, rank, 0);
        if (s.u1 < s.units) {  // up to the rank that holds the end of the job's cost
            o.w = (int)(cut.rank_of(s.cost0 + s.span - 1) - rank) + 1;
        }
        if (plan.by_job) plan.owner[(int64_t)s.v * plan.per + mine] = o;
        else if (o.w) plan.owner[blockIdx.x] = o;
    }

    // The record of a segment that is not a whole job: a CTA has one that begins inside a job, at
    // most, and one that begins a job and does not end it.
    __device__ __forceinline__ static float* record(const AtPlan& plan, const AtSegment& s, int D) {
        return plan.rec + (int64_t)(2 * blockIdx.x + (s.u0 == 0 ? 1 : 0)) * plan.crows * (D + 2);
    }
};

// Requests without any slot: zeros.
template <typename T, bool SPARSE>
__device__ __noinline__ void write_empty(const spin_kv_config& cfg, const KvAttendArgs& a, const AtPlan& plan) {
    const int rows = SPARSE ? 1 : a.rows, H = cfg.n_heads, d = cfg.head_dim;
    for (int x = blockIdx.x; x < plan.n_virtual; x += gridDim.x) {
        if (virtual_len<SPARSE>(cfg, a, x) > 0) continue;
        const int64_t base = (int64_t)x * rows * H;
        for (int64_t e = threadIdx.x; e < (int64_t)rows * H * d / 4; e += blockDim.x)
            store4(reinterpret_cast<T*>(a.out) + base * d + 4 * e, make_float4(0, 0, 0, 0));
        if (a.lse)
            for (int e = threadIdx.x; e < rows * H; e += blockDim.x) a.lse[base + e] = __uint_as_float(0xff800000u);
        if (plan.split && plan.by_job)
            for (int e = threadIdx.x; e < plan.per; e += blockDim.x) plan.owner[(int64_t)x * plan.per + e].w = 0;
    }
}

// lse of a row from its reference and sum.
__device__ __forceinline__ float row_lse(float ref, float l) {
    const float ninf = __uint_as_float(0xff800000u);
    const float lg = l < 1.2676506e30f ? log2f(l * (1.0f / kAtSumUnit)) : log2f(l) + 20.0f;
    return l == 0.0f ? ninf : ((ref == ninf ? 0.0f : ref) + lg) * 0.6931471805599453f;
}

// A row's outputs from its sums: o / l (zeros where there is no weight).  1 / l is normal: l <= 2^119.
__device__ __forceinline__ float4 row_out(const float4 o, float l) {
    if (l == 0.0f) return make_float4(0, 0, 0, 0);
    const float inv = __fdiv_rn(1.0f, l);
    return make_float4(o.x * kAtSumUnit * inv, o.y * kAtSumUnit * inv, o.z * kAtSumUnit * inv, o.w * kAtSumUnit * inv);
}

// Joins the pieces of the jobs that were divided: its first rank's second record, then the first
// records of the ranks after it.  One CTA per job and query row: the pieces' factors first, then
// each warp adds up every fourth piece.  A chain of latencies bounds it (launch, owner, factors,
// pieces): 6.5 us for 64 rows of 57 pieces; a CTA for all rows of a job took 26 us.
constexpr int kJoinWarps = 4;

template <typename T, int D>
__global__ void __launch_bounds__(32 * kJoinWarps)
kv_attend_join_kernel(spin_kv_config cfg, KvAttendArgs a, AtPlan plan, int rows) {
    pdl_wait();
    constexpr int F = D / 32;
    const int ROWS = plan.crows, REC = ROWS * (D + 2);
    __shared__ float s_c[kAtMostPieces], s_w[kAtMostPieces], s_top[kJoinWarps], s_l[kJoinWarps];
    __shared__ __align__(16) float s_acc[kJoinWarps][D];
    const int4 job = plan.owner[blockIdx.x];
    if (job.w == 0) return;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, H = cfg.n_heads, d = cfg.head_dim;
    const int group = H / cfg.kv_heads, g = job.y / plan.mchunks, m0 = job.y % plan.mchunks * ROWS, m = blockIdx.y;
    const int pieces = job.w;
    if (m >= min(ROWS, group * rows - m0)) return;
    const float ninf = __uint_as_float(0xff800000u);
    // CTA c has records 2c and 2c + 1; piece p lies in the first record of rank job.z + p, the first
    // piece in the second of its rank
    const float* rec = plan.rec + (int64_t)2 * (job.z * plan.per + job.y) * REC;
    const int64_t step = (int64_t)2 * plan.per * REC;
    auto at = [&](int p) -> const float* { return rec + (p ? p * step : REC); };
    // a warp's first pieces are on their way while the factors are found
    constexpr int AHEAD = 16 / F;
    float x[AHEAD][F];
    auto load = [&](float (&to)[F], int p) {
        const float* r = at(p) + m * D + lane * F;
        if constexpr (F == 2) {
            const float2 y = *reinterpret_cast<const float2*>(r);
            to[0] = y.x; to[1] = y.y;
        } else {
#pragma unroll
            for (int i = 0; i < F; i += 4) {
                const float4 y = *reinterpret_cast<const float4*>(r + i);
                to[i] = y.x; to[i + 1] = y.y; to[i + 2] = y.z; to[i + 3] = y.w;
            }
        }
    };
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
        if (wid + k * kJoinWarps < pieces) load(x[k], wid + k * kJoinWarps);
    float top = ninf, l = 0.0f;
    for (int p = tid; p < pieces; p += 32 * kJoinWarps) {
        const float2 ml = *reinterpret_cast<const float2*>(at(p) + ROWS * D + 2 * m);
        s_c[p] = ml.x;
        s_w[p] = ml.y;
        top = fmaxf(top, ml.x);
    }
#pragma unroll
    for (int i = 16; i; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
    if (lane == 0) s_top[wid] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, s_top[w]);
    for (int p = tid; p < pieces; p += 32 * kJoinWarps) {
        const float c = s_c[p] == ninf ? 0.0f : ex2(s_c[p] - top);
        s_c[p] = c;
        l = fmaf(c, s_w[p], l);
    }
#pragma unroll
    for (int i = 16; i; i >>= 1) l += __shfl_xor_sync(0xffffffffu, l, i);
    if (lane == 0) s_l[wid] = l;
    __syncthreads();
    l = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) l += s_l[w];
    float acc[F];
#pragma unroll
    for (int i = 0; i < F; ++i) acc[i] = 0.0f;
    for (int base = wid; base < pieces; base += AHEAD * kJoinWarps) {
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int p = base + k * kJoinWarps;
            if (p >= pieces) break;
            const float c = s_c[p];
#pragma unroll
            for (int i = 0; i < F; ++i) acc[i] = fmaf(c, x[k][i], acc[i]);
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int p = base + (AHEAD + k) * kJoinWarps;
            if (p < pieces) load(x[k], p);
        }
    }
#pragma unroll
    for (int i = 0; i < F; ++i) s_acc[wid][lane * F + i] = acc[i];
    __syncthreads();
    const int64_t bh = ((int64_t)job.x * rows + (m0 + m) / group) * H + (int64_t)g * group + (m0 + m) % group;
    for (int f = tid; f < d / 4; f += 32 * kJoinWarps) {
        float4 y = make_float4(0, 0, 0, 0);
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) {
            const float4 x = *reinterpret_cast<const float4*>(&s_acc[w][4 * f]);
            y.x += x.x; y.y += x.y; y.z += x.z; y.w += x.w;
        }
        store4(reinterpret_cast<T*>(a.out) + bh * d + 4 * f, row_out(y, l));
    }
    if (a.lse && tid == 0) a.lse[bh] = row_lse(top, l);
}

}  // namespace spin
