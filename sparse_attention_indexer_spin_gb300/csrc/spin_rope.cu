// spin_rope.cu -- rotary positions of queries and keys (sm_103a).
//
// A pair (x, y) of a token at position p becomes
//   m (x cos a - y sin a),  m (x sin a + y cos a),   a = 2 pi p f
// with f in turns a position as a 64-bit fraction F = round(2^64 f): the turns of p are the low 64
// bits of p F, whole-number arithmetic that loses nothing however far p is (F's own rounding adds
// p 2^-65 turns).  The signed upper bits as a fraction of half a turn go to sincospi.  Negative
// positions wrap the same way, to the inverse turn.
//
// Memory bounds it: every value is read and written once.  A CTA takes a token, works out each pair's cos and sin
// once for all heads, and moves 16 bytes a thread at a time where sizes and alignment allow it, pairs one by
// one otherwise.  16384 tokens of 40 heads of 128, bf16, out of a wider buffer: 65 us, 5.1 TB/s; 5000 of 17 fp32 heads
// of 192, a third of each turned: 24 us, 5.4 TB/s; 96 of 72 bf16 heads: 4 us, a launch.
#include <cuda_fp16.h>

#include "spin_common.cuh"
#include "spin_internal.h"

namespace spin {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxPairs = 512;   // rot_dim <= 1024

__device__ __forceinline__ float rope_f(float x) { return x; }
__device__ __forceinline__ float rope_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float rope_f(__half x) { return __half2float(x); }
__device__ __forceinline__ void rope_set(float& o, float x) { o = x; }
__device__ __forceinline__ void rope_set(__nv_bfloat16& o, float x) { o = __float2bfloat16_rn(x); }
__device__ __forceinline__ void rope_set(__half& o, float x) { o = __float2half_rn(x); }

template <typename T, int V> struct alignas(V * sizeof(T)) RopeVec {
    T x[V];
};

// V values at a time.  HALF: an item is V pairs, V values of each half; INTERLEAVED: V / 2 pairs side by side (V = 1:
// a pair, two values).  `copies`: the values outside the rotated ones are copied too.  A thread's first item is on
// its way while the angles are worked out.  Eight CTAs an SM, where registers allow (5000 tokens of 17 fp32 heads 24 us,
// 28 with six); two items ahead took 94 us instead of 65 on 16384 tokens of 40 16-bit heads, CTAs that stay and take
// token after token 69 to 97.  These bounds spill a few words a thread (bf16 halves 16 bytes stored and 48 loaded, the others 12 at
// most), which the times include.
template <typename T, int V, bool HALF>
__global__ void __launch_bounds__(kRopeThreads, HALF && V == 8 ? 6 : 8) rope_kernel(spin_rope_config cfg, RopeArgs a, int copies, int heads) {
    pdl_begin();
    __shared__ float2 s_turn[kRopeMaxPairs];
    constexpr int W = HALF || V > 1 ? V : 2;   // values of an interleaved item
    using Vec = RopeVec<T, W>;
    const int pairs = cfg.rot_dim / 2, threads = blockDim.x;
    const int turned = HALF ? pairs / V : cfg.rot_dim / W;        // items of a head that turn
    const int items = turned + (copies ? (cfg.head_dim - cfg.rot_dim) / V : 0);
    const int h0 = threadIdx.x / items, i0 = threadIdx.x - h0 * items;
    const int hs = threads / items, is = threads - hs * items;
    const int64_t t = blockIdx.x;
    struct Place {
        const T* in;
        T* out;
        int it;
    };
    int h = h0, it = i0, row = 0, base = 0;       // the item that comes next; heads before its tensor
    auto place = [&](Place& p) -> bool {
        if (h >= heads) return false;
        while (h - base >= a.rows[row].heads) base += (int)a.rows[row++].heads;
        const spin_rope_rows& r = a.rows[row];
        const int64_t at = (int64_t)(h - base) * cfg.head_dim;
        p.in = reinterpret_cast<const T*>(r.in) + t * r.in_stride + at;
        p.out = reinterpret_cast<T*>(r.out) + t * r.out_stride + at;
        p.it = it;
        h += hs;
        it += is;
        if (it >= items) it -= items, ++h;
        return true;
    };
    // an item's values: two vectors (HALF), or one, in u
    auto fetch = [&](const Place& p, Vec& u, Vec& v) {
        if (p.it >= turned) {
            int x = (p.it - turned) * V;
            if (x >= cfg.rot_first) x += cfg.rot_dim;
            if constexpr (W == V) u = *reinterpret_cast<const Vec*>(p.in + x);
            else u.x[0] = p.in[x];
        } else if constexpr (HALF) {
            const int x = cfg.rot_first + p.it * V;
            u = *reinterpret_cast<const Vec*>(p.in + x);
            v = *reinterpret_cast<const Vec*>(p.in + x + pairs);
        } else {
            const int x = cfg.rot_first + p.it * W;
            if constexpr (V > 1) u = *reinterpret_cast<const Vec*>(p.in + x);
            else u.x[0] = p.in[x], u.x[1] = p.in[x + 1];
        }
    };
    auto finish = [&](const Place& p, const Vec& u, const Vec& v) {
        if (p.it >= turned) {
            int x = (p.it - turned) * V;
            if (x >= cfg.rot_first) x += cfg.rot_dim;
            if constexpr (W == V) *reinterpret_cast<Vec*>(p.out + x) = u;
            else p.out[x] = u.x[0];
        } else if constexpr (HALF) {
            const int x = cfg.rot_first + p.it * V;
            Vec ou, ov;
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float2 cs = s_turn[p.it * V + k];
                const float fu = rope_f(u.x[k]), fv = rope_f(v.x[k]);
                rope_set(ou.x[k], fu * cs.x - fv * cs.y);
                rope_set(ov.x[k], fu * cs.y + fv * cs.x);
            }
            *reinterpret_cast<Vec*>(p.out + x) = ou;
            *reinterpret_cast<Vec*>(p.out + x + pairs) = ov;
        } else {
            const int x = cfg.rot_first + p.it * W;
            Vec o;
#pragma unroll
            for (int k = 0; k < W; k += 2) {
                const float2 cs = s_turn[(p.it * W + k) / 2];
                const float fu = rope_f(u.x[k]), fv = rope_f(u.x[k + 1]);
                rope_set(o.x[k], fu * cs.x - fv * cs.y);
                rope_set(o.x[k + 1], fu * cs.y + fv * cs.x);
            }
            if constexpr (V > 1) *reinterpret_cast<Vec*>(p.out + x) = o;
            else p.out[x] = o.x[0], p.out[x + 1] = o.x[1];
        }
    };
    Place p;
    Vec u, v;
    const int64_t pos = a.positions[t];
    bool more = place(p);
    if (more) fetch(p, u, v);
    for (int i = threadIdx.x; i < pairs; i += threads) {
        const int64_t turns = (int64_t)((uint64_t)pos * a.turns[i]);
        // turns 2^-64 of a turn: half turns in [-1, 1)
        float s, c;
        sincospif(__ll2float_rn(turns) * 1.0842021724855044e-19f, &s, &c);
        s_turn[i] = make_float2(c * cfg.magnitude, s * cfg.magnitude);
    }
    __syncthreads();
    while (more) {
        finish(p, u, v);
        more = place(p);
        if (more) fetch(p, u, v);
    }
}

template <typename T, bool HALF>
static cudaError_t launch_typed(const spin_rope_config& cfg, const RopeArgs& a, cudaStream_t s) {
    constexpr int V = 16 / (int)sizeof(T);
    bool wide = cfg.head_dim % V == 0 && cfg.rot_first % V == 0 && (HALF ? cfg.rot_dim / 2 : cfg.rot_dim) % V == 0;
    int copies = 0;
    for (int i = 0; i < a.n_rows; ++i) {
        const spin_rope_rows& r = a.rows[i];
        wide = wide && (((uintptr_t)r.in | (uintptr_t)r.out) & 15) == 0 && r.in_stride % V == 0 && r.out_stride % V == 0;
        copies |= r.in != r.out;
    }
    if (cfg.rot_dim == cfg.head_dim) copies = 0;
    // A token a CTA, as many threads as make its passes over the items even.
    int64_t heads = 0;
    for (int i = 0; i < a.n_rows; ++i) heads += a.rows[i].heads;
    const int w = wide ? V : 1, turned = HALF ? cfg.rot_dim / 2 / w : cfg.rot_dim / (w > 1 ? w : 2);
    const int64_t work = heads * (turned + (copies ? (cfg.head_dim - cfg.rot_dim) / w : 0));
    const int64_t passes = (work + kRopeThreads - 1) / kRopeThreads, each = (work + passes - 1) / passes;
    const dim3 grid((unsigned)a.n_tokens), block((unsigned)((each + 31) / 32 * 32));
    if (wide) return launch_pdl(rope_kernel<T, V, HALF>, grid, block, 0, s, nullptr, 0, cfg, a, copies, (int)heads);
    return launch_pdl(rope_kernel<T, 1, HALF>, grid, block, 0, s, nullptr, 0, cfg, a, copies, (int)heads);
}

template <typename T>
static cudaError_t launch_layout(const spin_rope_config& cfg, const RopeArgs& a, cudaStream_t s) {
    return cfg.layout == SPIN_ROPE_HALF ? launch_typed<T, true>(cfg, a, s) : launch_typed<T, false>(cfg, a, s);
}

cudaError_t launch_rope(const spin_rope_config& cfg, const RopeArgs& a, cudaStream_t s) {
    switch (cfg.dtype) {
        case SPIN_DTYPE_F32: return launch_layout<float>(cfg, a, s);
        case SPIN_DTYPE_BF16: return launch_layout<__nv_bfloat16>(cfg, a, s);
        default: return launch_layout<__half>(cfg, a, s);
    }
}

}  // namespace spin
