// spin_pages.cu -- page management of paged caches (sm_103a): re-parenting a batch's block
// tables, releasing pages, making the next slots writable (fresh pages, copies of shared
// ones) and compacting a pool.
//
// The state is a block table and a reference count per page; a page is free while its count
// is 0.  There is no free list: fresh pages are the lowest free ones, found by a scan over the
// counts, so a result depends on the state alone and never on the order of atomics (counts
// are only added to and subtracted from while other threads may).
//
// What bounds it.  Tables and counts are small: a call is a launch and a chain of a few dependent
// reads, and the plans are one CTA, which needs no other CTA's answer (reserve: 24 us for 256
// requests of a token, with its copying launch).  Copies run at the memory's rate:
// 0.44 GB moved in a pool of 1.6 GB, with the release and the plan before it, 155 us.
#include "spin_common.cuh"
#include "spin_internal.h"

namespace spin {

constexpr int kPgThreads = 256;
constexpr int kPlanThreads = 1024;
constexpr int kOwnBlocks = 4;          // blocks of a request that one thread of the plan looks at
constexpr int kPlanPages = 16;         // neighbouring pages a thread of a plan looks at, at a time
constexpr int kCopyBytes = 16 * 1024;  // bytes one CTA copies at a time

// Workspace: a header of 64 words, then prefix [n_req], dst, src and aux [n_pages].
struct PagesWs {
    int32_t* count;   // header word 0: entries of dst and src
    int32_t* live;    // header word 1: pages in use (compaction)
    int32_t* prefix;  // fresh pages wanted by the requests before this one
    int32_t* dst;
    int32_t* src;     // page to copy to dst, -1: none
    int32_t* aux;     // reserve: page the request leaves, -1: none; compaction: rank of a page that moves, -1: free
};

static __host__ __device__ inline int64_t round64(int64_t n) { return (n + 63) & ~(int64_t)63; }

static PagesWs pages_ws(void* ws, int32_t n_req, int64_t n_pages) {
    int32_t* p = reinterpret_cast<int32_t*>(ws);
    PagesWs w;
    w.count = p;
    w.live = p + 1;
    w.prefix = p + 64;
    w.dst = w.prefix + round64(n_req);
    w.src = w.dst + round64(n_pages);
    w.aux = w.src + round64(n_pages);
    return w;
}

size_t pages_workspace_bytes(int32_t n_req, int64_t n_pages) {
    return (size_t)(64 + round64(n_req) + 3 * round64(n_pages)) * sizeof(int32_t);
}

// A table entry as a page, or -1 (BAD_PAGE for anything else outside the pool).
__device__ __forceinline__ int32_t page_of(int32_t e, const PageTable& t) {
    if (e >= 0 && e < t.n_pages) return e;
    if (e != -1) set_status(t.status, SPIN_STATUS_BAD_PAGE);
    return -1;
}

// One use less of a page; a count that was already 0 stays there.
__device__ __forceinline__ void release(int32_t page, const PageTable& t) {
    if (atomicSub(t.ref + page, 1) <= 0) {
        atomicAdd(t.ref + page, 1);
        set_status(t.status, SPIN_STATUS_BAD_REF);
    }
}

// ---------------------------------------------------------------------------------- fork
// One thread per entry of the new table.  In place, a row that changes never serves as a
// source (checked through `parent`), so the rows read are not written.
__global__ void __launch_bounds__(kPgThreads)
pages_fork_kernel(PageTable t, const int32_t* table_in, const int32_t* parent) {
    pdl_begin();
    const bool in_place = table_in == t.table;
    for (int r = blockIdx.y; r < t.n_req; r += gridDim.y) {
        int p = parent[r];
        if (in_place && p == r) continue;
        bool bad = p < -1 || p >= t.n_req;
        if (in_place && !bad && p >= 0) bad = parent[p] != p;
        if (bad) {
            if (threadIdx.x == 0 && blockIdx.x == 0) set_status(t.status, SPIN_STATUS_BAD_PARENT);
            if (in_place) continue;
            p = -1;
        }
        for (int64_t j = (int64_t)blockIdx.x * kPgThreads + threadIdx.x; j < t.stride; j += (int64_t)gridDim.x * kPgThreads) {
            const int32_t old = page_of(table_in[r * t.stride + j], t);
            const int32_t now = p < 0 ? -1 : p == r ? old : page_of(table_in[p * t.stride + j], t);
            t.table[r * t.stride + j] = now;
            if (now != old) {
                if (now >= 0) atomicAdd(t.ref + now, 1);
                if (old >= 0) release(old, t);
            }
        }
    }
}

// ---------------------------------------------------------------------------------- free
__global__ void __launch_bounds__(kPgThreads) pages_free_kernel(PageTable t, const int32_t* keep) {
    pdl_begin();
    for (int r = blockIdx.y; r < t.n_req; r += gridDim.y) {
        const int k = keep[r];
        if (k < 0) continue;
        const int64_t first = (k >> 6) + ((k & 63) != 0);
        for (int64_t j = first + (int64_t)blockIdx.x * kPgThreads + threadIdx.x; j < t.stride;
             j += (int64_t)gridDim.x * kPgThreads) {
            const int32_t e = t.table[r * t.stride + j];
            if (e == -1) continue;
            const int32_t old = page_of(e, t);
            t.table[r * t.stride + j] = -1;
            if (old >= 0) release(old, t);
        }
    }
}

// ------------------------------------------------------------------------------- reserve
// Pages p0 .. p0 + kPlanPages - 1 as bits: those that exist, those in use.
__device__ __forceinline__ uint32_t pages_there(const PageTable& t, int64_t p0) {
    const int64_t n = t.n_pages - p0;
    return n <= 0 ? 0u : n >= kPlanPages ? (1u << kPlanPages) - 1 : (1u << n) - 1;
}
__device__ __forceinline__ uint32_t used_pages(const PageTable& t, int64_t p0) {
    int ref[kPlanPages];
#pragma unroll
    for (int i = 0; i < kPlanPages; ++i) ref[i] = p0 + i < t.n_pages ? t.ref[p0 + i] : 0;
    uint32_t used = 0;
#pragma unroll
    for (int i = 0; i < kPlanPages; ++i) used |= (uint32_t)(ref[i] > 0) << i;
    return used;
}

struct Span {
    int64_t j0, j1;   // blocks [j0, j1) the next slots fall in
    bool partial;     // the first of them already holds some of the request's slots
    bool bad;
};

__device__ __forceinline__ Span span_of(int32_t n, int32_t add, int64_t stride) {
    Span s{0, 0, false, n < 0 || add < 0};
    if (s.bad || add == 0) return s;
    s.j0 = n >> 6;
    s.j1 = ((int64_t)n + add + 63) >> 6;
    s.partial = (n & 63) != 0;
    s.bad = s.j1 > stride;
    if (s.bad) s.j1 = s.j0;
    return s;
}

// Whether a block needs a fresh page; *old is the page it has (-1: none).
__device__ __forceinline__ bool needs_page(const PageTable& t, int64_t at, int32_t* old) {
    *old = page_of(t.table[at], t);
    return *old < 0 || t.ref[*old] > 1;
}

// Calls f(r, span, fresh) for every request, with the number of blocks of its span that need a fresh page.
// A span of more than kOwnBlocks blocks is counted by its whole warp, four blocks a lane at a time
// (a prompt of 131072 slots: 51 us, 420 us by one thread).  Up to 1024 requests lane l of warp w has
// request 32 l + w, so that a few long prompts fall to as many warps; above, a warp's requests are
// neighbours, whose lengths are read together (4096 single tokens: 37 us, 60 us spread out).
template <typename F>
__device__ __forceinline__ void each_request(const PageTable& t, const int32_t* n_slots, const int32_t* n_new, F f) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    for (int base = 0; base < t.n_req; base += kPlanThreads) {
        const int r = base + (t.n_req <= kPlanThreads ? 32 * lane + wid : (int)threadIdx.x);
        Span sp{0, 0, false, false};
        if (r < t.n_req) sp = span_of(n_slots[r], n_new[r], t.stride);
        const bool by_warp = sp.j1 - sp.j0 > kOwnBlocks;
        int fresh = 0;
        int32_t old;
        if (!by_warp)
            for (int64_t j = sp.j0; j < sp.j1; ++j) fresh += needs_page(t, r * t.stride + j, &old);
        for (uint32_t todo = __ballot_sync(0xffffffffu, by_warp); todo; todo &= todo - 1) {
            const int from = __ffs(todo) - 1;
            const int64_t at = (int64_t)__shfl_sync(0xffffffffu, r, from) * t.stride;
            const int64_t j0 = __shfl_sync(0xffffffffu, sp.j0, from), j1 = __shfl_sync(0xffffffffu, sp.j1, from);
            int n = 0;
#pragma unroll 4
            for (int64_t j = j0 + lane; j < j1; j += 32) n += needs_page(t, at + j, &old);
            n = __reduce_add_sync(0xffffffffu, n);
            if (lane == from) fresh = n;
        }
        f(r, sp, fresh);
    }
}

// The plan, by one CTA: (1) count each request's fresh pages and their prefix, (2) list the
// lowest free pages, (3) hand them out, (4) move the reference counts.  Every decision in (3)
// reads the counts as they were at the start; only (4) changes them.
__global__ void __launch_bounds__(kPlanThreads)
pages_reserve_kernel(PageTable t, const int32_t* n_slots, const int32_t* n_new, int32_t* granted, PagesWs w) {
    pdl_begin();
    __shared__ int s_scan[33];
    __shared__ int s_given;
    const int tid = threadIdx.x, lane = tid & 31;
    constexpr int kMost = 1 << 30;  // prefix sums saturate here (n_pages <= 2^30)
    int carry = 0, sum;
    if (tid == 0) s_given = 0;
    each_request(t, n_slots, n_new, [&](int r, const Span& sp, int fresh) {
        if (r >= t.n_req) return;
        if (sp.bad) set_status(t.status, SPIN_STATUS_BAD_N);
        w.prefix[r] = fresh;
    });
    __syncthreads();
    for (int base = 0; base < t.n_req; base += kPlanThreads) {
        const int r = base + tid;
        const int pre = block_excl_scan(r < t.n_req ? w.prefix[r] : 0, s_scan, &sum);
        if (r < t.n_req) w.prefix[r] = min(kMost, carry + pre);
        carry = min(kMost, carry + sum);
    }
    const int total = carry;
    int found = 0;
    for (int64_t base = 0; base < t.n_pages && found < total; base += kPlanThreads * kPlanPages) {
        const int64_t p0 = base + (int64_t)tid * kPlanPages;
        const uint32_t free_pages = ~used_pages(t, p0) & pages_there(t, p0);
        int rank = found + block_excl_scan(__popc(free_pages), s_scan, &sum);
        for (uint32_t f = free_pages; f && rank < total; f &= f - 1) w.dst[rank++] = (int32_t)(p0 + __ffs(f) - 1);
        found += sum;
    }
    found = min(found, total);
    __syncthreads();
    each_request(t, n_slots, n_new, [&](int r, const Span& sp, int fresh) {
        bool serve = false;
        int k = 0;
        if (r < t.n_req) {
            k = w.prefix[r];
            const bool ok = fresh == 0 || (int64_t)k + fresh <= found;
            granted[r] = ok && !sp.bad;
            if (!ok) set_status(t.status, SPIN_STATUS_NO_PAGES);
            serve = ok && fresh > 0;
            if (serve) atomicMax(&s_given, k + fresh);
        }
        auto give = [&](int64_t at, const Span& s, int64_t j, int32_t old, int to) {
            t.table[at + j] = w.dst[to];
            w.aux[to] = old;
            w.src[to] = old >= 0 && s.partial && j == s.j0 ? old : -1;
        };
        const bool by_warp = serve && sp.j1 - sp.j0 > kOwnBlocks;
        int32_t old;
        if (serve && !by_warp)
            for (int64_t j = sp.j0; j < sp.j1; ++j)
                if (needs_page(t, r * t.stride + j, &old)) give(r * t.stride, sp, j, old, k++);
        for (uint32_t todo = __ballot_sync(0xffffffffu, by_warp); todo; todo &= todo - 1) {
            const int from = __ffs(todo) - 1;
            const int64_t at = (int64_t)__shfl_sync(0xffffffffu, r, from) * t.stride;
            Span s;
            s.j0 = __shfl_sync(0xffffffffu, sp.j0, from);
            s.j1 = __shfl_sync(0xffffffffu, sp.j1, from);
            s.partial = __shfl_sync(0xffffffffu, (int)sp.partial, from);
            int to = __shfl_sync(0xffffffffu, k, from);
            for (int64_t j4 = s.j0; j4 < s.j1; j4 += 128) {
                bool needs[4];
                int32_t olds[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t j = j4 + 32 * i + lane;
                    needs[i] = j < s.j1 && needs_page(t, at + j, &olds[i]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t m = __ballot_sync(0xffffffffu, needs[i]);
                    if (needs[i]) give(at, s, j4 + 32 * i + lane, olds[i], to + __popc(m & ((1u << lane) - 1)));
                    to += __popc(m);
                }
            }
        }
    });
    __syncthreads();
    const int given = s_given;
    for (int k = tid; k < given; k += kPlanThreads) {
        t.ref[w.dst[k]] = 1;
        if (w.aux[k] >= 0) release(w.aux[k], t);
    }
    if (tid == 0) *w.count = given;
}

// ------------------------------------------------------------------------------- compact
// The plan, by one CTA: the number L of pages in use, the used pages from L on (src) and the
// free ones below L (dst), both ascending, and the new id of every page from L on (aux; -1 for a free
// one).  There are as many of the ones as of the others, so a page's new id is the dst of its rank.
__global__ void __launch_bounds__(kPlanThreads) pages_compact_kernel(PageTable t, int32_t* n_live, PagesWs w) {
    pdl_begin();
    __shared__ int s_scan[33];
    const int tid = threadIdx.x;
    int cnt = 0, live;
#pragma unroll 8
    for (int64_t p = tid; p < t.n_pages; p += kPlanThreads) cnt += t.ref[p] > 0;
    block_excl_scan(cnt, s_scan, &live);
    int holes = 0, moves = 0, sum;
    for (int64_t base = 0; base < t.n_pages; base += kPlanThreads * kPlanPages) {
        const int64_t p0 = base + (int64_t)tid * kPlanPages;
        const uint32_t there = pages_there(t, p0), used = used_pages(t, p0);
        const int64_t below = live - p0;  // the first of them lie below L
        const uint32_t low = below <= 0 ? 0u : below >= kPlanPages ? ~0u : (1u << below) - 1;
        // (both counts in one scan: at most 16384 each)
        const int both = block_excl_scan(__popc(~used & low & there) | __popc(used & ~low) << 16, s_scan, &sum);
        int rank = holes + (both & 0xffff);
        for (uint32_t f = ~used & low & there; f; f &= f - 1) w.dst[rank++] = (int32_t)(p0 + __ffs(f) - 1);
        rank = moves + (both >> 16);
        for (uint32_t f = ~low & there; f; f &= f - 1) {
            const int64_t p = p0 + __ffs(f) - 1;
            const bool move = used >> (p - p0) & 1u;
            if (move) w.src[rank] = (int32_t)p;
            w.aux[p] = move ? rank++ : -1;
        }
        holes += sum & 0xffff;
        moves += sum >> 16;
    }
    if (tid == 0) {
        *w.count = moves;
        *w.live = live;
        *n_live = live;
    }
}

// ------------------------------------------------------------------------------- copying
// Pages src[k] -> dst[k] of every pool, in chunks of kCopyBytes.  No source is a destination, so that the
// copies can be repeated for other pools (spin_pages_copy).  After a compaction's plan (REMAP) the table
// entries and reference counts follow first.
template <bool REMAP>
__global__ void __launch_bounds__(kPgThreads) pages_copy_kernel(PageTable t, PagePoolSet pools, PagesWs w, int chunks) {
    pdl_begin();
    if constexpr (REMAP) {
        const int64_t me = (int64_t)blockIdx.x * kPgThreads + threadIdx.x, all = (int64_t)gridDim.x * kPgThreads;
        const int live = *w.live, moves = *w.count;
        for (int64_t i = me; i < (int64_t)t.n_req * t.stride; i += all) {
            const int32_t e = page_of(t.table[i], t);
            if (e < live) continue;
            const int32_t rank = w.aux[e];
            if (rank >= 0) t.table[i] = w.dst[rank];
            else set_status(t.status, SPIN_STATUS_BAD_REF);
        }
        for (int64_t k = me; k < moves; k += all) {
            t.ref[w.dst[k]] = t.ref[w.src[k]];
            t.ref[w.src[k]] = 0;
        }
    }
    const int64_t items = min((int64_t)max(*w.count, 0), t.n_pages) * chunks;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const int k = (int)(it / chunks);
        int c = (int)(it % chunks);
        const int32_t src = w.src[k], dst = w.dst[k];
        if (src == -1) continue;
        if (src < 0 || src >= t.n_pages || dst < 0 || dst >= t.n_pages) {  // (no plan in this workspace)
            set_status(t.status, SPIN_STATUS_BAD_PAGE);
            continue;
        }
        int p = 0;
        for (;; ++p) {
            const int n = (int)((pools.pool[p].page_bytes + kCopyBytes - 1) / kCopyBytes);
            if (c < n) break;
            c -= n;
        }
        const int64_t bytes = pools.pool[p].page_bytes, off = (int64_t)c * kCopyBytes;
        const int n = (int)(bytes - off < kCopyBytes ? bytes - off : kCopyBytes);
        const char* from = (const char*)pools.pool[p].data + src * bytes + off;
        char* to = (char*)pools.pool[p].data + dst * bytes + off;
        if ((((uintptr_t)pools.pool[p].data | (uintptr_t)bytes) & 15) == 0) {
            uint4 v[kCopyBytes / 16 / kPgThreads];
#pragma unroll
            for (int i = 0; i < kCopyBytes / 16 / kPgThreads; ++i) {
                const int e = (int)threadIdx.x + i * kPgThreads;
                if (e * 16 < n) v[i] = reinterpret_cast<const uint4*>(from)[e];
            }
#pragma unroll
            for (int i = 0; i < kCopyBytes / 16 / kPgThreads; ++i) {
                const int e = (int)threadIdx.x + i * kPgThreads;
                if (e * 16 < n) reinterpret_cast<uint4*>(to)[e] = v[i];
            }
        } else {
            for (int e = threadIdx.x; e * 4 < n; e += kPgThreads)
                reinterpret_cast<uint32_t*>(to)[e] = reinterpret_cast<const uint32_t*>(from)[e];
        }
    }
}

static int copy_chunks(const PagePoolSet& pools) {
    int64_t n = 0;
    for (int i = 0; i < pools.n; ++i) n += (pools.pool[i].page_bytes + kCopyBytes - 1) / kCopyBytes;
    return (int)n;
}

static dim3 table_grid(const PageTable& t) {
    const int64_t x = (t.stride + kPgThreads - 1) / kPgThreads;
    return dim3((unsigned)(x < 64 ? x : 64), (unsigned)t.n_req);
}

cudaError_t launch_pages_fork(const PageTable& t, const int32_t* table_in, const int32_t* parent, cudaStream_t s) {
    return launch_pdl(pages_fork_kernel, table_grid(t), dim3(kPgThreads), 0, s, nullptr, 0, t, table_in, parent);
}

cudaError_t launch_pages_free(const PageTable& t, const int32_t* keep, cudaStream_t s) {
    return launch_pdl(pages_free_kernel, table_grid(t), dim3(kPgThreads), 0, s, nullptr, 0, t, keep);
}

template <bool REMAP>
static cudaError_t launch_copy(const PageTable& t, const PagePoolSet& pools, const PagesWs& w, cudaStream_t s) {
    const int chunks = copy_chunks(pools);
    if (chunks == 0 && !REMAP) return cudaSuccess;
    return launch_pdl(pages_copy_kernel<REMAP>, dim3(8 * device_sm_count()), dim3(kPgThreads), 0, s, nullptr, 0, t, pools,
                      w, chunks);
}

cudaError_t launch_pages_reserve(const PageTable& t, const int32_t* n_slots, const int32_t* n_new,
                                 const PagePoolSet& pools, int32_t* granted, void* ws, cudaStream_t s) {
    const PagesWs w = pages_ws(ws, t.n_req, t.n_pages);
    cudaError_t e = launch_pdl(pages_reserve_kernel, dim3(1), dim3(kPlanThreads), 0, s, nullptr, 0, t, n_slots, n_new,
                               granted, w);
    return e != cudaSuccess ? e : launch_copy<false>(t, pools, w, s);
}

cudaError_t launch_pages_copy(const PageTable& t, const PagePoolSet& pools, void* ws, cudaStream_t s) {
    return launch_copy<false>(t, pools, pages_ws(ws, t.n_req, t.n_pages), s);
}

cudaError_t launch_pages_compact(const PageTable& t, const PagePoolSet& pools, int32_t* n_live, void* ws,
                                 cudaStream_t s) {
    const PagesWs w = pages_ws(ws, t.n_req, t.n_pages);
    cudaError_t e = launch_pdl(pages_compact_kernel, dim3(1), dim3(kPlanThreads), 0, s, nullptr, 0, t, n_live, w);
    return e != cudaSuccess ? e : launch_copy<true>(t, pools, w, s);
}

}  // namespace spin
