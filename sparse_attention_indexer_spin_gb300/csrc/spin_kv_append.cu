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
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "spin_common.cuh"
#include "spin_internal.h"

namespace spin {

constexpr int kAppThreads = 256;

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

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}

__device__ __forceinline__ float2 values2(uint32_t two_codes) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two_codes, __NV_E4M3);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// One CTA per (request, touched page, head, key or value): its at most 64 x head_dim new
// values are read once into registers (NV 16-byte vectors a thread), reduced to max|x|, and
// written as codes.
template <typename T, int NV>
__global__ void __launch_bounds__(kAppThreads, NV <= 4 ? 5 : 1)
kv_append_kernel(spin_kv_config cfg, KvAppendArgs a) {
    pdl_begin();
    constexpr int E = 16 / (int)sizeof(T);  // elements per vector
    __shared__ float s_amax[kAppThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, kv = blockIdx.y, h = blockIdx.x % cfg.kv_heads;
    const int kvh = cfg.kv_heads, d = cfg.head_dim;

    // The touched pages of all requests are laid end to end; every warp looks up which of them this
    // CTA's is, 32 requests at a time.
    int jj = blockIdx.x / kvh, r = -1;  // page jj of request r
    int64_t t0 = 0, cnt = 0, nb = 0;
    const bool reports = blockIdx.x == 0 && kv == 0 && tid < 32;  // this warp looks at every request
    for (int base = 0; base < cfg.n_req; base += 32) {
        const int x = base + lane;
        int64_t s0 = 0, c = 0, n = 0;
        int pages = 0;
        if (x < cfg.n_req) {
            s0 = a.new_start[x];
            c = a.new_start[x + 1] - s0;
            n = a.n_before[x];
            if (s0 < 0 || c < 0 || s0 + c > a.n_tokens || c > a.max_new || n < 0 || n + c > cfg.max_slots) {
                if (reports) set_status(a.status, SPIN_STATUS_BAD_N);
            } else if (c > 0) {
                pages = (int)(((n + c - 1) >> 6) - (n >> 6)) + 1;
            }
        }
        const int upto = warp_incl_scan(pages);
        const uint32_t here = __ballot_sync(0xffffffffu, upto > jj);
        if (r < 0 && here) {
            const int at = __ffs(here) - 1;
            r = base + at;
            jj -= __shfl_sync(0xffffffffu, upto - pages, at);
            t0 = __shfl_sync(0xffffffffu, s0, at);
            cnt = __shfl_sync(0xffffffffu, c, at);
            nb = __shfl_sync(0xffffffffu, n, at);
            if (!reports) break;
        }
        if (r < 0) jj -= __shfl_sync(0xffffffffu, upto, 31);
    }
    if (r < 0) return;
    const int64_t j = (nb >> 6) + jj;
    const int64_t page = a.block_table[(int64_t)r * a.bt_stride + j];
    if (page < 0 || page >= a.n_pages) {
        if (tid == 0) set_status(a.status, SPIN_STATUS_BAD_PAGE);
        return;
    }
    const int64_t s0 = nb > j * kBlock ? nb : j * kBlock;
    const int64_t s1 = nb + cnt < (j + 1) * kBlock ? nb + cnt : (j + 1) * kBlock;
    const int at = (int)(s0 & 63), m = (int)(s1 - s0);

    const uint4* x = reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(kv ? a.x[1] : a.x[0]) +
                                                    ((t0 + s0 - nb) * kvh + h) * d);
    const int per_row = d / E, row_step = kvh * per_row, nvec = m * per_row;
    float amax = 0.0f;
    uint4 v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = tid + i * kAppThreads;
        v[i] = e < nvec ? x[(int64_t)(e / per_row) * row_step + e % per_row] : make_uint4(0, 0, 0, 0);
    }
    float* scale = (kv ? a.scale[1] : a.scale[0]) + page * kvh + h;
    const float old = at ? *scale : 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float f[E];
        unpack(v[i], f, (const T*)nullptr);
#pragma unroll
        for (int k = 0; k < E; ++k) {
            const float ab = fabsf(f[k]);
            if (ab < __uint_as_float(0x7f800000u)) amax = fmaxf(amax, ab);  // finite values only
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if ((tid & 31) == 0) s_amax[tid >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kAppThreads / 32; ++w) amax = fmaxf(amax, s_amax[w]);

    const float s_new = fmaxf(old, pow2_scale(amax));
    const float inv = s_new >= __uint_as_float(0x00800000u) ? __fdiv_rn(1.0f, s_new) : 0.0f;
    uint8_t* dst = (kv ? a.pool[1] : a.pool[0]) + (page * kBlock * kvh + h) * d;
    if (tid == 0) *scale = s_new;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = tid + i * kAppThreads;
        if (e >= nvec) break;
        float f[E];
        unpack(v[i], f, (const T*)nullptr);
        uint8_t* o = dst + (int64_t)(at + e / per_row) * kvh * d + e % per_row * E;
        if constexpr (E == 4) {
            *reinterpret_cast<uint32_t*>(o) = codes4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
        } else {
            *reinterpret_cast<uint2*>(o) = make_uint2(codes4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                                                      codes4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
        }
    }
    if (at && s_new != old) {  // the page's earlier slots move to the larger scale
        const float ratio = s_new >= __uint_as_float(0x00800000u) ? __fdiv_rn(old, s_new) : 0.0f;
        const int words = d / 4;
        for (int e = tid; e < at * words; e += kAppThreads) {
            uint32_t* p = reinterpret_cast<uint32_t*>(dst + (int64_t)(e / words) * kvh * d) + e % words;
            const uint32_t c = *p;
            const float2 lo = values2(c & 0xffffu), hi = values2(c >> 16);
            *p = codes4(lo.x * ratio, lo.y * ratio, hi.x * ratio, hi.y * ratio);
        }
    }
}

template <typename T>
static cudaError_t launch_typed(const spin_kv_config& cfg, const KvAppendArgs& a, cudaStream_t s) {
    if (a.max_new == 0) return cudaSuccess;
    // pages touched, at most: n slots touch (n + 62) / 64 + 1, one page more than they fill
    const int64_t each = ((int64_t)a.max_new + kBlock - 2) / kBlock + 1;
    const int64_t all = a.n_tokens / kBlock + 2 * (int64_t)cfg.n_req;
    const int64_t pages = each * cfg.n_req < all ? each * cfg.n_req : all;
    if (pages * cfg.kv_heads > 0x7fffffff) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)(pages * cfg.kv_heads), 2);
    const int nv = (kBlock * cfg.head_dim * (int)sizeof(T) + 16 * kAppThreads - 1) / (16 * kAppThreads);
    if (nv <= 4) return launch_pdl(kv_append_kernel<T, 4>, grid, dim3(kAppThreads), 0, s, nullptr, 0, cfg, a);
    if (nv <= 8) return launch_pdl(kv_append_kernel<T, 8>, grid, dim3(kAppThreads), 0, s, nullptr, 0, cfg, a);
    if constexpr (sizeof(T) == 4)
        return launch_pdl(kv_append_kernel<T, 16>, grid, dim3(kAppThreads), 0, s, nullptr, 0, cfg, a);
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
