// spin_kv_append.cu -- new keys and values quantised into the paged 8-bit cache (sm_103a).
//
// Per page p that a request's new slots fall in, and per key/value head h:
//   s_old = 0 if the first new slot is the page's slot 0, else scale[p][h]
//   s_new = max(s_old, 2^e),  2^e the smallest power of two with max|x| <= 448 2^e, e >= -126
//   earlier slots: code <- e4m3(code s_old / s_new);   new slots: code = e4m3(x / s_new)
// e4m3 carries its own exponent, so a scale that is only a power of two costs no relative
// precision, and it makes every quotient exact: the single rounding is the one to e4m3 (at
// most half a step, 2^-4 of a normal code), and moving the earlier slots to a larger scale
// loses only what falls below e4m3's smallest subnormal.
//
// Memory bounds it: each new value is read once and its code written once.  Eight ragged prompts of bf16
// tokens, 8 heads x 128, one call among others: 49 us, 6.0 TB/s of the 293 MB.  As a graph launch of its own
// behind an L2 flush, some microseconds of it the launch: 45056 tokens of that shape 53 us (277 MB), f32 92 us,
// 8 x 64 33 us.  Issue slots come next, so maxima are taken two values at a time, a thread divides once for
// its place, and keys and values share a CTA's look-up (81 us before).  A token each for 64 requests: 11 us
// in such a graph, the chain of dependent reads counts -> page -> scale.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "spin_common.cuh"
#include "spin_internal.h"

namespace spin {

// The smallest power of two s >= 2^-126 with amax <= 448 s (0 for amax = 0): 448 = 1.75 2^8, so
// with amax = m 2^k, 1 <= m < 2, it is 2^(k-8) where m <= 1.75, else 2^(k-7).
__device__ __forceinline__ float pow2_scale(float amax) {
    const uint32_t u = __float_as_uint(amax);
    if (u == 0u) return 0.0f;
    int e = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);  // biased exponent of s
    return __uint_as_float((uint32_t)(e < 1 ? 1 : e) << 23);
}

__device__ __forceinline__ void unpack(const uint4 v, float (&x)[4], const float*) {
    x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ void unpack(const uint4 v, float (&x)[8], const __nv_bfloat16*) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack(const uint4 v, float (&x)[8], const __half*) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

// max|x| over a vector and `m` (NaN left out; infinite where one is): the 16-bit types two at a time
__device__ __forceinline__ void abs_max(const uint4 v, float& m, const float*) {
    m = fmaxf(fmaxf(fmaxf(fabsf(__uint_as_float(v.x)), fabsf(__uint_as_float(v.y))),
                    fmaxf(fabsf(__uint_as_float(v.z)), fabsf(__uint_as_float(v.w)))), m);
}
template <typename T2> __device__ __forceinline__ T2 abs_max2(const uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    T2 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __habs2(*reinterpret_cast<const T2*>(&w[i]));
    return __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
}
__device__ __forceinline__ void abs_max(const uint4 v, float& m, const __nv_bfloat16*) {
    const float2 f = __bfloat1622float2(abs_max2<__nv_bfloat162>(v));
    m = fmaxf(m, fmaxf(f.x, f.y));
}
__device__ __forceinline__ void abs_max(const uint4 v, float& m, const __half*) {
    const float2 f = __half22float2(abs_max2<__half2>(v));
    m = fmaxf(m, fmaxf(f.x, f.y));
}

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}

__device__ __forceinline__ float2 values2(uint32_t two_codes) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two_codes, __NV_E4M3);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// One CTA per (request, touched page, head): its at most 64 x head_dim new keys, then values
// (P = 2; P = 1: one CTA for each, where a thread's registers would not hold both), are read once
// into registers (NV 16-byte vectors a thread), reduced to max|x|, and written as codes.
template <typename T, int THREADS, int NV, int P>
__global__ void __launch_bounds__(THREADS, NV * P <= 8 ? 1024 / THREADS : 1)
kv_append_kernel(spin_kv_config cfg, KvAppendArgs a, int each) {
    pdl_begin();
    constexpr int E = 16 / (int)sizeof(T);  // elements per vector
    __shared__ float s_amax[P][THREADS / 32];
    __shared__ int s_pages[THREADS / 32], s_found[5];
    const int tid = threadIdx.x, lane = tid & 31, kv0 = blockIdx.y, h = blockIdx.x % cfg.kv_heads;
    const int kvh = cfg.kv_heads, d = cfg.head_dim;

    int jj = blockIdx.x / kvh, r = 0;  // page jj of request r
    int t0 = 0, cnt = 0, nb = 0;
    // the pages that request x touches (0 where it is refused): its place among the new tokens,
    // its count and its slots before
    auto pages_of = [&](int x, bool reports, int& s0, int& c, int& n) -> int {
        s0 = a.new_start[x];
        const int s1 = a.new_start[x + 1];
        n = a.n_before[x];
        c = s0 < 0 || s1 < s0 ? -1 : s1 - s0;
        if (c < 0 || s1 > a.n_tokens || c > a.max_new || n < 0 || n > cfg.max_slots - c) {
            if (reports) set_status(a.status, SPIN_STATUS_BAD_N);
            return 0;
        }
        return c > 0 ? ((n + c - 1) >> 6) - (n >> 6) + 1 : 0;
    };
    const bool first = h == 0 && kv0 == 0;
    if (each) {  // `each` CTAs for every request's pages
        r = jj / each;
        jj -= r * each;
        if (jj >= pages_of(r, first && jj == 0 && tid == 0, t0, cnt, nb)) return;
    } else {     // the touched pages of all requests laid end to end
        const bool reports = first && jj == 0;  // this CTA looks at every request
        bool found = false;
        for (int base = 0; base < cfg.n_req; base += THREADS) {
            const int x = base + tid;
            int s0, c, n, pages = 0;
            if (x < cfg.n_req) pages = pages_of(x, reports, s0, c, n);
            const int upto = warp_incl_scan(pages);
            if (lane == 31) s_pages[tid >> 5] = upto;
            __syncthreads();
            int lo = upto - pages, all = 0;
#pragma unroll
            for (int w = 0; w < THREADS / 32; ++w) {
                if (w < tid >> 5) lo += s_pages[w];
                all += s_pages[w];
            }
            if (!found && jj >= lo && jj < lo + pages) {
                s_found[0] = x, s_found[1] = jj - lo, s_found[2] = s0, s_found[3] = c, s_found[4] = n;
            }
            __syncthreads();
            if (!found && jj < all) {
                found = true;
                r = s_found[0], jj = s_found[1], t0 = s_found[2], cnt = s_found[3], nb = s_found[4];
            } else if (!found) {
                jj -= all;
            }
            if (found && !reports) break;
        }
        if (!found) return;
    }
    const int j = (nb >> 6) + jj;
    const int64_t page = a.block_table[r * a.bt_stride + j];  // (looked at when the loads are on their way)
    const int s0 = max(nb, j * kBlock), s1 = min(nb + cnt, (j + 1) * kBlock);
    const int at = s0 & 63, m = s1 - s0;

    const int per_row = d / E, row_step = kvh * per_row, nvec = m * per_row;
    // vector e = tid + i THREADS lies in row e / per_row: one division, then steps
    const int row0 = tid / per_row, col0 = tid - row0 * per_row;
    const int rows_i = THREADS / per_row, cols_i = THREADS - rows_i * per_row;
    auto step = [&](int& row, int& col) {
        row += rows_i;
        col += cols_i;
        if (col >= per_row) col -= per_row, ++row;
    };
    uint4 v[P][NV];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const uint4* x = reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(kv0 + p ? a.x[1] : a.x[0]) +
                                                        ((int64_t)(t0 + s0 - nb) * kvh + h) * d);
        int row = row0, col = col0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            v[p][i] = tid + i * THREADS < nvec ? x[row * row_step + col] : make_uint4(0, 0, 0, 0);
            step(row, col);
        }
    }
    if (page < 0 || page >= a.n_pages) {
        if (tid == 0) set_status(a.status, SPIN_STATUS_BAD_PAGE);
        return;
    }
    float old[P];
#pragma unroll
    for (int p = 0; p < P; ++p) old[p] = at ? (kv0 + p ? a.scale[1] : a.scale[0])[page * kvh + h] : 0.0f;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) abs_max(v[p][i], amax, (const T*)nullptr);
        if (amax == __uint_as_float(0x7f800000u)) {  // finite values only
            amax = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float f[E];
                unpack(v[p][i], f, (const T*)nullptr);
#pragma unroll
                for (int k = 0; k < E; ++k)
                    if (fabsf(f[k]) < __uint_as_float(0x7f800000u)) amax = fmaxf(amax, fabsf(f[k]));
            }
        }
        // (non-negative floats order as their bits do)
        amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
        if (lane == 0) s_amax[p][tid >> 5] = amax;
    }
    __syncthreads();
#pragma unroll
    for (int p = 0; p < P; ++p) {
        float amax = s_amax[p][0];
#pragma unroll
        for (int w = 1; w < THREADS / 32; ++w) amax = fmaxf(amax, s_amax[p][w]);
        const float s_new = fmaxf(old[p], pow2_scale(amax));
        // (below 2^-126 there are only zeros, infinities and NaN: they keep their codes under any factor but 0)
        const float inv = s_new >= __uint_as_float(0x00800000u) ? __fdiv_rn(1.0f, s_new) : 1.0f;
        uint8_t* dst = (kv0 + p ? a.pool[1] : a.pool[0]) + (page * kBlock * kvh + h) * d;
        if (tid == 0) (kv0 + p ? a.scale[1] : a.scale[0])[page * kvh + h] = s_new;
        int row = row0, col = col0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (tid + i * THREADS >= nvec) break;
            float f[E];
            unpack(v[p][i], f, (const T*)nullptr);
            uint8_t* o = dst + (at + row) * kvh * d + col * E;
            if constexpr (E == 4) {
                *reinterpret_cast<uint32_t*>(o) = codes4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
            } else {
                *reinterpret_cast<uint2*>(o) = make_uint2(codes4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                                                          codes4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
            }
            step(row, col);
        }
        if (at && s_new != old[p]) {  // the page's earlier slots move to the larger scale
            const float ratio = s_new >= __uint_as_float(0x00800000u) ? __fdiv_rn(old[p], s_new) : 0.0f;
            const int words = d / 4;
            for (int e = tid; e < at * words; e += THREADS) {
                uint32_t* q = reinterpret_cast<uint32_t*>(dst + (int64_t)(e / words) * kvh * d) + e % words;
                const uint32_t c = *q;
                const float2 lo = values2(c & 0xffffu), hi = values2(c >> 16);
                *q = codes4(lo.x * ratio, lo.y * ratio, hi.x * ratio, hi.y * ratio);
            }
        }
    }
}

template <typename T>
static cudaError_t launch_typed(const spin_kv_config& cfg, const KvAppendArgs& a, cudaStream_t s) {
    // pages touched, at most: n slots touch (n + 62) / 64 + 1, one page more than they fill.  Every
    // request gets as many CTAs as the longest may need where that is no more than all can touch (a
    // token or so each, or prompts of one length; one, which checks the counts, where max_new is 0); else
    // a CTA looks its page up (512 requests of 4 tokens: 34 us without, 43 us with the look-up; 64 of 1
    // token: 11 us both).
    int64_t each = ((int64_t)a.max_new + kBlock - 2) / kBlock + 1;
    int64_t pages = a.n_tokens / kBlock + 2 * (int64_t)cfg.n_req;
    if (each * cfg.n_req <= pages) pages = each * cfg.n_req;
    else each = 0;
    if (pages * cfg.kv_heads > 0x7fffffff) return cudaErrorInvalidValue;
    const dim3 both((unsigned)(pages * cfg.kv_heads)), grid(both.x, 2);
    // 64 new slots of a head in a thread's registers; up to 128 bytes a slot a CTA of half the size
    // keeps its threads busy (45056 bf16 tokens, 8 x 64: 33 us, 44 us with 256 threads)
    const int slot_bytes = cfg.head_dim * (int)sizeof(T);
    if (slot_bytes <= 128)
        return launch_pdl(kv_append_kernel<T, 128, 4, 2>, both, dim3(128), 0, s, nullptr, 0, cfg, a, (int)each);
    if (slot_bytes <= 256)
        return launch_pdl(kv_append_kernel<T, 256, 4, 2>, both, dim3(256), 0, s, nullptr, 0, cfg, a, (int)each);
    if (slot_bytes <= 512)
        return launch_pdl(kv_append_kernel<T, 256, 8, 1>, grid, dim3(256), 0, s, nullptr, 0, cfg, a, (int)each);
    if constexpr (sizeof(T) == 4)
        return launch_pdl(kv_append_kernel<T, 256, 16, 1>, grid, dim3(256), 0, s, nullptr, 0, cfg, a, (int)each);
    return cudaErrorInvalidValue;  // not reached: head_dim <= 256
}

cudaError_t launch_kv_append(const spin_kv_config& cfg, const KvAppendArgs& a, cudaStream_t s) {
    switch (cfg.dtype) {
        case SPIN_DTYPE_F32: return launch_typed<float>(cfg, a, s);
        case SPIN_DTYPE_BF16: return launch_typed<__nv_bfloat16>(cfg, a, s);
        default: return launch_typed<__half>(cfg, a, s);
    }
}

}  // namespace spin
