// spin_pages_evict.cu -- eviction of a request's lightest blocks from a paged cache (sm_103a).
//
// A block of 64 slots weighs as much as its heaviest slot (a maximum: the same in any order).  Of a
// request's B blocks the newest and the first ones stay, and of the others the heaviest, equal ones
// in the order of their places; what stays closes ranks.  The blocks' weights become order-preserving
// keys, an exact radix selection finds the lightest key that stays, and the row's entries and the
// slots' weights move down in order.
//
// Memory bounds it: each weight is read (those that stay twice) and written once.  A cluster of up to eight CTAs takes a
// request where its table is not too wide: one launch, all of them reading and moving weights and the first choosing.  Wider
// tables take three launches, their weights read and moved by the whole GPU.
// 96 requests of 20000 to 131072 slots cut to a third (75 MB): 30 us, 2.5 TB/s; by three launches 38.  What is left to the
// copy rate (11 us) is the chain within a request: its weights, the choice by one CTA, the move.  8 requests of up to 2000
// slots: 6 us.
#include "spin_common.cuh"
#include "spin_internal.h"

namespace spin {

constexpr int kEvThreads = 256;
constexpr int kEvSelThreads = 512;
constexpr int kEvPer = 4;          // neighbouring entries of a row that a thread looks at
constexpr int kEvAhead = 4;        // blocks whose weights half a warp has in flight
constexpr int kEvNear = 4096;      // blocks of a table that a cluster takes: their keys in shared memory
constexpr int kEvCluster = 8;      // its CTAs, at most

// Order of the weights: order_key's, NaN above everything.
__device__ __forceinline__ uint32_t weight_key(float x) { return x != x ? 0xffffffffu : order_key(x); }

// A request's blocks, or -1 where its slots are out of range.
__device__ __forceinline__ int evict_blocks(const PageTable& t, int n) {
    return n < 0 || n > t.stride * kBlock ? -1 : (n + kBlock - 1) / kBlock;
}

// Blocks' keys, by all threads of a CTA: half a warp reads a block, four slots a lane.  Blocks first, first + step, ..
// below B, where `first` is this half warp's.
__device__ __forceinline__ void block_keys(const float4* w, int n, int B, int first, int step, uint32_t* keys) {
    const int l16 = threadIdx.x & 15;
    // (whole warps stay together: the other half's block may be the last)
    for (int j0 = first; j0 - (int)((threadIdx.x >> 4) & 1) < B; j0 += step * kEvAhead) {
        float4 x[kEvAhead];
#pragma unroll
        for (int i = 0; i < kEvAhead; ++i) {
            const int j = j0 + i * step;
            x[i] = j < B ? w[(int64_t)j * 16 + l16] : make_float4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kEvAhead; ++i) {
            const int j = j0 + i * step;
            const int64_t left = n - (int64_t)j * kBlock - 4 * l16;
            uint32_t key = 0;
            if (left > 0) key = weight_key(x[i].x);
            if (left > 1) key = max(key, weight_key(x[i].y));
            if (left > 2) key = max(key, weight_key(x[i].z));
            if (left > 3) key = max(key, weight_key(x[i].w));
#pragma unroll
            for (int o = 8; o; o >>= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, o));
            if (l16 == 0 && j < B) keys[j] = key;
        }
    }
}

struct EvictShared {
    int hist[256], scan[33], pick[3];
};

// The choice of a request's blocks by a CTA of kEvSelThreads, m = keep < B of them, and its row's compaction; `key` in shared
// or global memory.
__device__ __forceinline__ void evict_row(const PageTable& t, const PageEvictArgs& a, int r, int n, int B, int keep,
                                          const uint32_t* key, EvictShared& sh) {
    const int tid = threadIdx.x;
    int32_t* row = t.table + (int64_t)r * t.stride;
    int32_t* kept = a.kept + (int64_t)r * t.stride;
    const int last = min(keep, a.n_last), first = min(keep - last, a.n_first);
    const int lo = first, hi = B - last;              // the blocks that are chosen from
    int need = keep - last - first;                   // of them stay; less than hi - lo
    uint32_t prefix = 0, mask = 0;
    if (need > 0) {
        // the lightest key that stays, eight bits at a time
#pragma unroll 1
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (tid < 256) sh.hist[tid] = 0;
            __syncthreads();
            // (weights lie near each other: the first digits of a warp's keys are few, and one lane adds for all that share one)
            for (int j0 = lo; j0 < hi; j0 += kEvSelThreads) {
                const int j = j0 + tid;
                const uint32_t k = j < hi ? key[j] : 0u;
                const int digit = j < hi && (k & mask) == prefix ? (int)((k >> shift) & 255u) : -1;
                const uint32_t same = __match_any_sync(0xffffffffu, digit);
                if (digit >= 0 && (int)(tid & 31) == __ffs(same) - 1) atomicAdd(sh.hist + digit, __popc(same));
            }
            __syncthreads();
            // the digit whose bin holds the need-th largest: counts from the top down, eight bins a lane
            if (tid < 32) {
                int c[8], sum = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) sum += c[i] = sh.hist[255 - 8 * tid - i];
                int above = warp_incl_scan(sum) - sum;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (above < need && need <= above + c[i]) {
                        sh.pick[0] = 255 - 8 * tid - i;
                        sh.pick[1] = need - above;
                        sh.pick[2] = need == above + c[i];
                    }
                    above += c[i];
                }
            }
            __syncthreads();
            prefix |= (uint32_t)sh.pick[0] << shift;
            mask |= 0xffu << shift;
            need = sh.pick[1];
            if (sh.pick[2]) break;   // all keys that begin so stay
        }
    }
    // keys above `prefix` (in its digits) stay, and the first `need` of those equal to it; a thread looks at kEvPer neighbours
    int at = 0, equal = 0;                            // blocks kept, and equal keys, so far
    for (int64_t base = 0; base < t.stride; base += kEvSelThreads * kEvPer) {
        const int64_t j0 = base + tid * kEvPer;
        int32_t e[kEvPer];
#pragma unroll
        for (int i = 0; i < kEvPer; ++i) e[i] = j0 + i < t.stride ? row[j0 + i] : -1;
        uint32_t above = 0, ties = 0;                 // bits of the entries
#pragma unroll
        for (int i = 0; i < kEvPer; ++i) {
            const int64_t j = j0 + i;
            const bool chosen = j >= lo && j < hi;
            const uint32_t k = chosen ? key[j] & mask : 0u;   // (the digits that were looked at)
            if (j < t.stride && (!chosen || k > prefix)) above |= 1u << i;
            if (chosen && need > 0 && k == prefix) ties |= 1u << i;
        }
        // both counts in one scan: 2048 each at most
        int both;
        const int before = block_excl_scan(__popc(above) | __popc(ties) << 16, sh.scan, &both);   // (a barrier: the entries are read)
        int tie = equal + (before >> 16), to = at + (before & 0xffff) + min(max(need - equal, 0), before >> 16);
#pragma unroll
        for (int i = 0; i < kEvPer; ++i) {
            const int64_t j = j0 + i;
            if (j >= t.stride) break;
            const bool stay = (above >> i & 1u) || ((ties >> i & 1u) && tie < need);
            tie += ties >> i & 1u;
            const int32_t page = e[i] >= 0 && e[i] < t.n_pages ? e[i] : -1;
            if (e[i] != page && e[i] != -1) set_status(t.status, SPIN_STATUS_BAD_PAGE);
            if (stay) {
                row[to] = page;
                if (j < B) kept[to] = (int)j;
                ++to;
            } else if (page >= 0) {
                if (atomicSub(t.ref + page, 1) <= 0) {
                    atomicAdd(t.ref + page, 1);
                    set_status(t.status, SPIN_STATUS_BAD_REF);
                }
            }
        }
        at += (both & 0xffff) + min(max(need - equal, 0), both >> 16);
        equal += both >> 16;
    }
    for (int64_t j = at + tid; j < t.stride; j += kEvSelThreads) row[j] = -1;
    for (int64_t j = keep + tid; j < t.stride; j += kEvSelThreads) kept[j] = -1;
    if (tid == 0) a.n_slots[r] = keep ? n - kBlock * (B - keep) : 0;
}

// Weights to their new places, sixteen lanes a block: blocks first, first + step, .. below `end` of the row, n slots long
// now; block j comes from from(j), -1: zeros.
template <typename F>
__device__ __forceinline__ void move_weights(const PageTable& t, const PageEvictArgs& a, int r, int64_t n, int64_t first, int64_t step, int64_t end, F from) {
    const int l16 = threadIdx.x & 15;
    const float4* w = reinterpret_cast<const float4*>(a.weight) + (int64_t)r * t.stride * 16;
    float4* o = reinterpret_cast<float4*>(a.weight_out) + (int64_t)r * t.stride * 16;
    for (int64_t j0 = first; j0 < end; j0 += step * kEvAhead) {
        float4 x[kEvAhead];
#pragma unroll
        for (int i = 0; i < kEvAhead; ++i) {
            const int64_t j = j0 + i * step, b = j < end ? from(j) : -1;
            x[i] = b >= 0 ? w[b * 16 + l16] : make_float4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kEvAhead; ++i) {
            const int64_t j = j0 + i * step, left = n - j * kBlock - 4 * l16;
            if (left < 4) x[i].w = 0.0f;
            if (left < 3) x[i].z = 0.0f;
            if (left < 2) x[i].y = 0.0f;
            if (left < 1) x[i].x = 0.0f;
            if (j < end) o[j * 16 + l16] = x[i];
        }
    }
}

// ------------------------------------------------------------------- a request in a cluster
// All CTAs of the cluster; what they wrote is there for the others.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__global__ void __launch_bounds__(kEvSelThreads) evict_kernel(PageTable t, PageEvictArgs a, uint32_t* keys, int ctas) {
    pdl_begin();
    extern __shared__ uint32_t s_key[];
    __shared__ EvictShared sh;
    const int r = blockIdx.x / ctas, rank = blockIdx.x - r * ctas, tid = threadIdx.x;
    const int n = a.n_slots[r], B = evict_blocks(t, n), keep = a.keep[r];
    const int first = rank * (kEvSelThreads / 16) + (tid >> 4), step = ctas * (kEvSelThreads / 16);
    int32_t* kept = a.kept + (int64_t)r * t.stride;
    if (B < 0 || keep < 0 || keep >= B) {    // (the whole cluster)
        if (B < 0 && tid == 0 && rank == 0) set_status(t.status, SPIN_STATUS_BAD_N);
        for (int64_t j = rank * kEvSelThreads + tid; j < t.stride; j += (int64_t)ctas * kEvSelThreads) kept[j] = j < B ? (int)j : -1;
        move_weights(t, a, r, B < 0 ? t.stride * kBlock : n, first, step, t.stride, [&](int64_t j) { return B < 0 || j < B ? j : -1; });
        return;
    }
    const float4* w = reinterpret_cast<const float4*>(a.weight) + (int64_t)r * t.stride * 16;
    if (ctas == 1) {
        block_keys(w, n, B, first, step, s_key);
        __syncthreads();
    } else {
        keys += (int64_t)r * t.stride;
        block_keys(w, n, B, first, step, keys);
        cluster_sync();
        if (rank == 0) {
            for (int j = tid; j < B; j += kEvSelThreads) s_key[j] = __ldcg(keys + j);
            __syncthreads();
        }
    }
    // the first CTA chooses, the others empty the places behind what stays
    const int64_t n_new = keep ? n - kBlock * (B - keep) : 0;
    if (rank == 0) evict_row(t, a, r, n, B, keep, s_key, sh);
    if (rank || ctas == 1) {
        const int others = max(1, ctas - 1), me = max(0, rank - 1);
        move_weights(t, a, r, n_new, keep + me * (kEvSelThreads / 16) + (tid >> 4), others * (kEvSelThreads / 16), t.stride,
                     [](int64_t) { return (int64_t)-1; });
    }
    if (ctas == 1) __syncthreads();
    else cluster_sync();
    move_weights(t, a, r, n_new, first, step, keep, [&](int64_t j) { return (int64_t)__ldcg(kept + j); });
}

// ----------------------------------------------------------------------- three launches
__global__ void __launch_bounds__(kEvThreads) evict_weigh_kernel(PageTable t, PageEvictArgs a, uint32_t* keys) {
    pdl_begin();
    for (int r = blockIdx.y; r < t.n_req; r += gridDim.y) {
        const int n = a.n_slots[r], B = evict_blocks(t, n), m = a.keep[r];
        if (m < 0 || m >= B) continue;
        block_keys(reinterpret_cast<const float4*>(a.weight) + (int64_t)r * t.stride * 16, n, B,
                   blockIdx.x * (kEvThreads / 16) + threadIdx.x / 16, gridDim.x * (kEvThreads / 16), keys + (int64_t)r * t.stride);
    }
}

__global__ void __launch_bounds__(kEvSelThreads) evict_select_kernel(PageTable t, PageEvictArgs a, const uint32_t* keys) {
    pdl_begin();
    __shared__ EvictShared sh;
    const int r = blockIdx.x, tid = threadIdx.x, n = a.n_slots[r], B = evict_blocks(t, n), keep = a.keep[r];
    __syncthreads();   // every thread has read n_slots
    if (B < 0 || keep < 0 || keep >= B) {
        if (B < 0 && tid == 0) set_status(t.status, SPIN_STATUS_BAD_N);
        for (int64_t j = tid; j < t.stride; j += kEvSelThreads) a.kept[(int64_t)r * t.stride + j] = j < B ? (int)j : -1;
        return;
    }
    evict_row(t, a, r, n, B, keep, keys + (int64_t)r * t.stride, sh);
}

// n_slots are the new ones here.
__global__ void __launch_bounds__(kEvThreads) evict_move_kernel(PageTable t, PageEvictArgs a) {
    pdl_begin();
    for (int r = blockIdx.y; r < t.n_req; r += gridDim.y) {
        const int n = a.n_slots[r];
        const bool bad = evict_blocks(t, n) < 0;
        const int32_t* kept = a.kept + (int64_t)r * t.stride;
        move_weights(t, a, r, bad ? t.stride * kBlock : n, (int64_t)blockIdx.x * (kEvThreads / 16) + threadIdx.x / 16,
                     (int64_t)gridDim.x * (kEvThreads / 16), t.stride, [&](int64_t j) { return bad ? j : (int64_t)kept[j]; });
    }
}

size_t pages_evict_workspace_bytes(int32_t n_req, int64_t bt_stride) {
    return (size_t)n_req * bt_stride * sizeof(uint32_t);
}

cudaError_t launch_pages_evict(const PageTable& t, const PageEvictArgs& a, cudaStream_t s) {
    uint32_t* keys = reinterpret_cast<uint32_t*>(a.workspace);
    if (t.stride <= kEvNear) {
        // as many CTAs a request as the GPU holds at once, four an SM, and each at least 64 blocks
        int ctas = kEvCluster;
        while (ctas > 1 && ((int64_t)t.n_req * ctas > 4 * device_sm_count() || t.stride < 64 * ctas)) ctas /= 2;
        cudaLaunchAttribute at;
        at.id = cudaLaunchAttributeClusterDimension;
        at.val.clusterDim.x = ctas;
        at.val.clusterDim.y = at.val.clusterDim.z = 1;
        return launch_pdl(evict_kernel, dim3(t.n_req * ctas), dim3(kEvSelThreads), t.stride * sizeof(uint32_t), s, &at, ctas > 1 ? 1 : 0, t, a,
                          keys, ctas);
    }
    const int64_t per = kEvThreads / 16 * kEvAhead, gx = (t.stride + per - 1) / per;
    const dim3 grid((unsigned)(gx < 1024 ? gx : 1024), t.n_req);
    cudaError_t e = launch_pdl(evict_weigh_kernel, grid, dim3(kEvThreads), 0, s, nullptr, 0, t, a, keys);
    if (e == cudaSuccess)
        e = launch_pdl(evict_select_kernel, dim3(t.n_req), dim3(kEvSelThreads), 0, s, nullptr, 0, t, a, (const uint32_t*)keys);
    if (e == cudaSuccess) e = launch_pdl(evict_move_kernel, grid, dim3(kEvThreads), 0, s, nullptr, 0, t, a);
    return e;
}

}  // namespace spin
