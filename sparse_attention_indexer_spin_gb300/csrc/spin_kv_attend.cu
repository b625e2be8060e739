// spin_kv_attend.cu -- attention over the paged 8-bit KV cache (sm_103a).
//
// Per query row and head, over the row's set of slots (its context, or the slots of a list):
//   s_i = softmax_scale ks (q . kc_i),  out = sum_i e^{s_i} vs vc_i / sum_i e^{s_i},
//   lse = ln sum_i e^{s_i}
// in one pass, with the running maximum and sum of the softmax.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "spin_common.cuh"
#include "spin_internal.h"

namespace spin {

template <typename T> __device__ __forceinline__ float to_f(T x);
template <> __device__ __forceinline__ float to_f(float x) { return x; }
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <> __device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_f(float x) { return __float2half_rn(x); }

__device__ __forceinline__ float code_value(uint8_t c) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(c, __NV_E4M3);
    return __half2float(*reinterpret_cast<const __half*>(&h));
}

// One warp per (request, row, head): lane l holds dims l, l + 32, ...
template <typename T>
__global__ void __launch_bounds__(32) kv_attend_kernel(spin_kv_config cfg, KvAttendArgs a) {
    pdl_begin();
    const int lane = threadIdx.x, h = blockIdx.x, row = blockIdx.y, b = blockIdx.z;
    const int H = cfg.n_heads, kvh = cfg.kv_heads, d = cfg.head_dim, g = h / (H / kvh);
    const int64_t br = (int64_t)b * a.rows + row;
    int n = a.n_slots[br];
    if (n < 0 || n > cfg.max_slots) {
        if (lane == 0) set_status(a.status, SPIN_STATUS_BAD_N);
        n = 0;
    }
    float q[8], o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c = lane + 32 * i;
        q[i] = c < d ? to_f(reinterpret_cast<const T*>(a.q)[(br * H + h) * d + c]) * cfg.softmax_scale : 0.0f;
        o[i] = 0.0f;
    }
    const float ninf = __uint_as_float(0xff800000u);
    float m = ninf, l = 0.0f;
    const int cnt = a.list ? a.top_k : n;
    for (int t = 0; t < cnt; ++t) {
        int i = t;
        if (a.list) {
            i = a.list[br * a.top_k + t];
            if (i == -1) continue;
            if (i < 0 || i >= n) {
                if (lane == 0) set_status(a.status, SPIN_STATUS_BAD_LIST);
                continue;
            }
        }
        const int64_t page = a.block_table[(int64_t)b * a.bt_stride + (i >> 6)];
        if (page < 0 || page >= a.n_pages) {
            if (lane == 0) set_status(a.status, SPIN_STATUS_BAD_PAGE);
            continue;
        }
        const int64_t at = ((page * kBlock + (i & 63)) * kvh + g) * d;
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (lane + 32 * k < d) s = fmaf(q[k], code_value(a.k_pool[at + lane + 32 * k]), s);
#pragma unroll
        for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= a.k_scale[page * kvh + g];
        const float vs = a.v_scale[page * kvh + g];
        const float mn = fmaxf(m, s), f = m == ninf ? 0.0f : expf(m - mn), p = expf(s - mn);
        m = mn;
        l = l * f + p;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (lane + 32 * k < d) o[k] = o[k] * f + p * vs * code_value(a.v_pool[at + lane + 32 * k]);
    }
    const float inv = m == ninf ? 0.0f : 1.0f / l;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (lane + 32 * k < d) reinterpret_cast<T*>(a.out)[(br * H + h) * d + lane + 32 * k] = from_f<T>(o[k] * inv);
    if (a.lse && lane == 0) a.lse[br * H + h] = m == ninf ? ninf : m + logf(l);
}

size_t kv_attend_workspace_bytes(const spin_kv_config&, int, int) { return 256; }

cudaError_t launch_kv_attend(const spin_kv_config& cfg, const KvAttendArgs& a, cudaStream_t s) {
    const dim3 grid(cfg.n_heads, a.rows, cfg.n_req);
    switch (cfg.dtype) {
        case SPIN_DTYPE_F32: return launch_pdl(kv_attend_kernel<float>, grid, dim3(32), 0, s, nullptr, 0, cfg, a);
        case SPIN_DTYPE_BF16:
            return launch_pdl(kv_attend_kernel<__nv_bfloat16>, grid, dim3(32), 0, s, nullptr, 0, cfg, a);
        default: return launch_pdl(kv_attend_kernel<__half>, grid, dim3(32), 0, s, nullptr, 0, cfg, a);
    }
}

}  // namespace spin
