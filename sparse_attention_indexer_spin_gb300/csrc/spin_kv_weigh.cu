// spin_kv_weigh.cu -- the attention weight that cached slots gather from few new tokens, decoded ones (sm_103a).
//
//   w[r][i] <- decay w[r][i] + sum_{t, h: i <= before + t} exp(s_{t,h,i} - lse[t][h]),
//   s = softmax_scale ks (q . kc_i)
// The log-sum of a row is known, so there is no running maximum: with the row's constants
//   c = log2(e) softmax_scale 2^-k,  b = -log2(e) lse
// a weight is 2^(c ks (q 2^k . kc_i) + b), one product, one fused multiply-add and one exponential.
//
// The keys of the context are read once, and they are what it has to move.  The contexts of all requests are laid end to
// end in units of 16 slots and cut into equal parts, one for each CTA.  A unit's heads go to the CTA's warps in turn: neighbouring
// heads' keys, which lie side by side, are read together (against a unit a warp: 63.8 -> 62.0 us), and the warps' sums meet
// in shared memory every few units.  A warp's keys come by cp.async into a place where each lane reads what it copied
// itself, two heads ahead (one ahead in registers: 75 us; three: 70, as fewer CTAs fit), the first ones while the query
// rows are made (66.2 -> 64.5).  Products are mma.sync m16n8k16 of 16 keys with the request's query rows, which lie in shared
// memory as f16, scaled by a power of two per row as in the attention (two f16 terms for fp32).  A slot's sum is taken in an
// order that depends on the sizes alone: no atomics.
// 64 requests of one token and up to 8192 slots, 32 heads on 8 of 128, bf16: 62 us for 271 MB, 4.4 TB/s.  What is left to the
// copy rate (40 us): issue is 57 % active, with most stalls fixed latencies of dependent instructions (conversion, product,
// exponential) in 20 warps an SM, as many as the registers hold; and the start and end of the parts.
// Beyond kWgMostRows query rows of a key head the tcgen05 kernel of spin_kv_weigh_tc.cu is taken: the same contexts with
// 32 rows 144 us here and 190 there, with 64 rows 264 here and 200 there.
#include <algorithm>

#include "spin_kv_chunk.cuh"

namespace spin {

constexpr int kWgThreads = 128;
constexpr int kWgMostRows = 32;         // query rows of a key head, at most
constexpr int kWgUnit = 16;             // slots of a unit: the rows of a product
constexpr int kWgNear = 256;            // requests whose places every CTA works out (a launch less: 64 of them 25.7 us, else 29.5; 256 75 and 78)
constexpr int kWgSmem = 228 * 1024;     // shared memory of an SM's CTAs, which cost 1024 each beside their own
constexpr int kWgRowBytes = 32 * 1024;  // shared memory for query rows; more heads take turns
template <int D> constexpr int wg_ctas() { return D == 256 ? 3 : 5; }   // CTAs on an SM
template <int D> constexpr int wg_ahead() { return D == 256 ? 2 : D == 128 ? 2 : 4; }   // heads' keys on their way to a warp
// a warp's place for one of them: 16 bytes and a scale for each lane's pieces
template <int D> constexpr int wg_stage() { return 16 * D + 128; }

__device__ __forceinline__ uint32_t lds_u32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ void wg_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Workspace: {first token, count, slots before} of every request, and the units before it.
struct WeighWs {
    int4* req;
    int64_t* begin;   // [requests + 1]
};
static __host__ __device__ inline int wg_dim(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }
static size_t wg_round(size_t n) { return (n + 255) & ~(size_t)255; }
static WeighWs weigh_ws(void* ws, const spin_kv_config& cfg) {
    char* p = reinterpret_cast<char*>(ws);
    WeighWs w;
    w.req = reinterpret_cast<int4*>(p);
    w.begin = reinterpret_cast<int64_t*>(p + wg_round((size_t)cfg.n_req * sizeof(int4)));
    return w;
}
static bool few_rows(const spin_kv_config& cfg, int max_new) {
    return (int64_t)max_new * (cfg.n_heads / cfg.kv_heads) <= kWgMostRows;
}
size_t kv_weigh_workspace_bytes(const spin_kv_config& cfg, int64_t n_tokens, int max_new) {
    if (!few_rows(cfg, max_new)) return kv_weigh_tc_workspace_bytes(cfg, n_tokens);
    return wg_round((size_t)cfg.n_req * sizeof(int4)) + wg_round(((size_t)cfg.n_req + 1) * sizeof(int64_t));
}

// Requests' checked ranges and the units before each, by a CTA; returns the units of all.
template <int THREADS>
__device__ __forceinline__ int64_t place_requests(const spin_kv_config& cfg, const KvChunkArgs& a, const WeighWs& w, int* s_max, int64_t* s_scan) {
    int64_t before_all = 0;
    for_requests<THREADS>(cfg, a, s_max, [&](int x, int s0, int count, int before) {
        const int64_t units = count ? (before + count + kWgUnit - 1) / kWgUnit : 0;
        int64_t sum;
        const int64_t inc = cta_incl_scan64<THREADS / 32>(units, s_scan, &sum);
        if (x < cfg.n_req) {
            w.req[x] = make_int4(s0, count, before, 0);
            w.begin[x] = before_all + inc - units;
        }
        before_all += sum;
    });
    return before_all;
}

__global__ void __launch_bounds__(1024) weigh_plan_kernel(spin_kv_config cfg, KvChunkArgs a, WeighWs w) {
    pdl_begin();
    __shared__ int s_max[32];
    __shared__ int64_t s_scan[32];
    const int64_t all = place_requests<1024>(cfg, a, w, s_max, s_scan);
    if (threadIdx.x == 0) w.begin[cfg.n_req] = all;
}

// A query row in shared memory: D f16 (or two times D) and 16 bytes that spread the rows over the banks.
template <int D, bool SPLIT> struct WgRow {
    static constexpr int BYTES = D * 2 * (SPLIT ? 2 : 1) + 16;
};

// near: few requests, whose places every CTA works out for itself (a launch less); else w has them.
template <typename T, int D>
__global__ void __launch_bounds__(kWgThreads, wg_ctas<D>())
weigh_kernel(const __grid_constant__ spin_kv_config cfg, const __grid_constant__ KvChunkArgs a, WeighWs w, int tiles, int heads_once, int near) {
    pdl_wait();
    constexpr bool SPLIT = std::is_same<T, float>::value;
    constexpr int C = D / 64, L = D / 16, RB = WgRow<D, SPLIT>::BYTES, AHEAD = wg_ahead<D>();
    // the warps' keys, then rows of heads_once heads, then their constants
    extern __shared__ __align__(16) unsigned char smem_all[];
    const uint32_t keys = smem_u32(smem_all);
    unsigned char* smem = smem_all + kWgThreads / 32 * AHEAD * wg_stage<D>();
    const int M8 = tiles * 8;                                // rows of a head, padded
    float4* s_row = reinterpret_cast<float4*>(smem + (size_t)heads_once * M8 * RB);
    constexpr int WARPS = kWgThreads / 32;
    __shared__ float s_sum[2][WARPS][WARPS][kWgUnit];
    __shared__ int s_req, s_max[kWgThreads / 32];
    __shared__ int64_t s_scan[kWgThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, g8 = lane >> 2, t4 = lane & 3;
    const int kvh = cfg.kv_heads, d = cfg.head_dim, H = cfg.n_heads, G = H / kvh;
    if (near) {
        w.begin = reinterpret_cast<int64_t*>(s_row + (size_t)heads_once * M8);
        w.req = reinterpret_cast<int4*>(w.begin + ((cfg.n_req + 2) & ~1));
        const int64_t all = place_requests<kWgThreads>(cfg, a, w, s_max, s_scan);
        if (tid == 0) w.begin[cfg.n_req] = all;
        __syncthreads();
    }
    AtCut cut;
    const int64_t total = w.begin[cfg.n_req];
    cut.set(total, gridDim.x);
    const int64_t at = cut.begin(blockIdx.x), end = cut.begin(blockIdx.x + 1);
    if (at >= end) return;
    for (int x = tid; x < cfg.n_req; x += kWgThreads)
        if (w.begin[x] <= at && at < w.begin[x + 1]) s_req = x;
    __syncthreads();
    int64_t from = at;
    for (int r = s_req; from < end; ++r) {
        const int64_t b0 = w.begin[r], b1 = w.begin[r + 1];
        if (b1 <= from) continue;
        const int u0 = (int)(from - b0), u1 = (int)(min(end, b1) - b0);   // this request's units
        from = b0 + u1;
        const int4 me = w.req[r];
        const int n = me.z + me.y, M = me.y * G;
        const int32_t* table = a.block_table + (int64_t)r * a.bt_stride;
        for (int h0 = 0; h0 < kvh; h0 += heads_once) {
            const int heads = min(heads_once, kvh - h0);
            // ---- this warp's units, and their heads one after another: the first keys are read while the rows are made,
            // the next ones while these multiply
            auto page_of = [&](int u) -> int { return u < u1 ? table[u >> 2] : -1; };
            // (a lane's pieces lie where it alone reads them: nothing but its own copies has to be waited for)
            auto load = [&](uint32_t to, int page, int u, int g) {
                const bool ok = page >= 0 && page < a.n_pages;
                cp4(to + 16 * D + 4 * lane, a.k_scale + (ok ? (int64_t)page * kvh + g : 0), ok);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int slot = u * kWgUnit + g8 + 8 * y;
                    const uint8_t* src = a.k_pool + (((int64_t)(ok ? page : 0) * kBlock + (slot & 63)) * kvh + g) * d;
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        const int dim = 64 * c + 16 * t4;
                        const bool live = ok && slot < n && dim < d;
                        cp16(to + 512 * (2 * c + y) + 16 * lane, src + (live ? dim : 0), live);
                    }
                }
            };
            // Where the copies are, some heads ahead of the products: the warps take a unit's heads in turn, so that
            // they read neighbouring bytes together, and with few heads the next units'.
            int lu = u0, lg = wid;
            auto skip = [&](int& u, int& g) {    // to the unit that an index behind its heads falls in
                while (g >= heads) g -= heads, ++u;
            };
            skip(lu, lg);
            int lpage = page_of(lu);
            auto load_next = [&](uint32_t to) {
                if (lu < u1) {
                    load(to, lpage, lu, h0 + lg);
                    const int page = lu >> 2;
                    lg += WARPS;
                    skip(lu, lg);
                    if (lu >> 2 != page) lpage = page_of(lu);
                }
                cp_commit();
            };
            const uint32_t ring = keys + wid * AHEAD * wg_stage<D>();
#pragma unroll
            for (int x = 0; x < AHEAD; ++x) load_next(ring + x * wg_stage<D>());
            __syncthreads();
            // ---- query rows: D / 16 lanes each, 16 values a lane, made f16
            for (int i0 = 0; i0 < heads * M8; i0 += kWgThreads / L) {
                const int i = i0 + tid / L, ch = tid % L, g = h0 + i / M8, m = i % M8;
                const bool in = i < heads * M8, live = in && m < M;
                const int t = live ? m / G : 0, h = live ? g * G + m - t * G : 0;
                const int64_t th = (int64_t)(me.x + t) * H + h;
                constexpr int QN = (int)sizeof(T);
                uint4 v[QN];
#pragma unroll
                for (int y = 0; y < QN; ++y)
                    v[y] = live && 16 * ch < d ? reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(a.q) + th * d + 16 * ch)[y]
                                               : make_uint4(0, 0, 0, 0);
                float x[16], amax = 0.0f;
#pragma unroll
                for (int y = 0; y < 16; ++y) {
                    x[y] = to_f(reinterpret_cast<const T*>(v)[y]);
                    amax = fmaxf(amax, fabsf(x[y]));
                }
#pragma unroll
                for (int o = L / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                // amax in [2^k, 2^(k+1)) -> [2^14, 2^15); 2^(14 - k) within [2^-113, 2^126]
                const int k = max(-112, (int)(__float_as_uint(amax) >> 23) - 127);
                const float f = __uint_as_float((uint32_t)(127 + 14 - k) << 23);
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int y = 0; y < 8; ++y) {
                    hi[y] = pack_f16(x[2 * y] * f, x[2 * y + 1] * f);
                    const float2 z = unpack_f16(hi[y]);
                    lo[y] = SPLIT ? pack_f16(x[2 * y] * f - z.x, x[2 * y + 1] * f - z.y) : 0u;
                }
                if (in) {
                    uint4* to = reinterpret_cast<uint4*>(smem + (size_t)i * RB + 32 * ch);
                    to[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    to[1] = make_uint4(hi[4], hi[5], hi[6], hi[7]);
                    if constexpr (SPLIT) {
                        to[D / 8] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                        to[D / 8 + 1] = make_uint4(lo[4], lo[5], lo[6], lo[7]);
                    }
                    if (ch == 0) {
                        const float lse = live ? a.lse[th] : __uint_as_float(0xff800000u);
                        // a row of no weight sees no slot
                        const int seen = lse == __uint_as_float(0xff800000u) ? 0 : me.z + t + 1;
                        s_row[i] = make_float4(__uint_as_float((uint32_t)max(1, 127 - 14 + k) << 23) * (cfg.softmax_scale * 1.4426950408889634f),
                                               -1.4426950408889634f * lse, __int_as_float(seen), 0.0f);
                    }
                }
            }
            __syncthreads();

            // ---- weights
            float sum[2] = {0.0f, 0.0f};
            auto head = [&](uint32_t stage, int u, int g) {
                cp_wait<AHEAD - 1>();
                uint32_t kf[C][4][4];                     // [64 dims][step][fragment]
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const uint4 y0 = lds128(stage + 1024 * c + 16 * lane), y1 = lds128(stage + 1024 * c + 512 + 16 * lane);
                    const uint32_t x0[4] = {y0.x, y0.y, y0.z, y0.w}, x1[4] = {y1.x, y1.y, y1.z, y1.w};
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        codes_to_f16(x0[s], kf[c][s][0], kf[c][s][2]);
                        codes_to_f16(x1[s], kf[c][s][1], kf[c][s][3]);
                    }
                }
                const float scale = __uint_as_float(lds_u32(stage + 16 * D + 4 * lane));
                load_next(stage);
                float part[2] = {0.0f, 0.0f};
#pragma unroll 1
                for (int m0 = 0; m0 < M8; m0 += 8) {
                    float part_of[C][4], acc[4];   // (a chain of products for each 64 dimensions: half the wait for the last)
#pragma unroll
                    for (int c = 0; c < C; ++c)
#pragma unroll
                        for (int x = 0; x < 4; ++x) part_of[c][x] = 0.0f;
                    const unsigned char* q = smem + (size_t)(g * M8 + m0 + g8) * RB + 32 * t4;
#pragma unroll
                    for (int z = 0; z < (SPLIT ? 2 : 1); ++z)
#pragma unroll
                        for (int c = 0; c < C; ++c) {
                            const uint4 y0 = *reinterpret_cast<const uint4*>(q + z * D * 2 + 128 * c);
                            const uint4 y1 = *reinterpret_cast<const uint4*>(q + z * D * 2 + 128 * c + 16);
                            wg_mma(part_of[c], kf[c][0], y0.x, y0.y);
                            wg_mma(part_of[c], kf[c][1], y0.z, y0.w);
                            wg_mma(part_of[c], kf[c][2], y1.x, y1.y);
                            wg_mma(part_of[c], kf[c][3], y1.z, y1.w);
                        }
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        acc[x] = part_of[0][x];
#pragma unroll
                        for (int c = 1; c < C; ++c) acc[x] += part_of[c][x];
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float4 cst = s_row[g * M8 + m0 + 2 * t4 + i];
                        const int seen = __float_as_int(cst.z);
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const float p = ex2(fmaf(acc[2 * y + i] * scale, cst.x, cst.y));
                            if (u * kWgUnit + g8 + 8 * y < seen) part[y] += p;
                        }
                    }
                }
                sum[0] += part[0];
                sum[1] += part[1];
            };
            int x = 0, turn = 0, u = u0, g = wid;    // this warp's next unit and head
            skip(u, g);
            for (int base = u0; base < u1; base += WARPS, turn ^= 1) {
                // as many units as warps: their sums meet in shared memory
                for (int k = 0; k < WARPS; ++k) {
                    sum[0] = sum[1] = 0.0f;
                    while (u == base + k && u < u1) {
                        head(ring + x * wg_stage<D>(), u, g);
                        x = x + 1 == AHEAD ? 0 : x + 1;
                        g += WARPS;
                        skip(u, g);
                    }
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        sum[y] += __shfl_xor_sync(0xffffffffu, sum[y], 1);
                        sum[y] += __shfl_xor_sync(0xffffffffu, sum[y], 2);
                        if (t4 == 0) s_sum[turn][k][wid][g8 + 8 * y] = sum[y];
                    }
                }
                __syncthreads();
                const int at = base + wid;
                if (at < u1) {
                    const int page = page_of(at), slot = at * kWgUnit + lane;
                    const bool ok = page >= 0 && page < a.n_pages;
                    if (!ok && lane == 0) set_status(a.status, SPIN_STATUS_BAD_PAGE);
                    if (ok && lane < kWgUnit && slot < n) {
                        float all = 0.0f;
#pragma unroll
                        for (int w = 0; w < WARPS; ++w) all += s_sum[turn][wid][w][lane];
                        float* o = a.weight + (int64_t)r * a.bt_stride * kBlock + slot;
                        // the first heads' sum joins the old weight, the others' what is there by now
                        if (h0) *o += all;
                        else *o = slot < me.z && a.decay != 0.0f ? fmaf(a.decay, *o, all) : all;
                    }
                }
            }
        }
    }
    pdl_trigger();
}

template <typename T, int D>
static cudaError_t launch_dim(const spin_kv_config& cfg, const KvChunkArgs& a, cudaStream_t s) {
    constexpr int RB = WgRow<D, std::is_same<T, float>::value>::BYTES;
    const WeighWs w = weigh_ws(a.workspace, cfg);
    const bool near = cfg.n_req <= kWgNear;
    cudaError_t e = cudaSuccess;
    if (!near || a.max_new == 0) e = launch_pdl(weigh_plan_kernel, dim3(1), dim3(1024), 0, s, nullptr, 0, cfg, a, w);
    if (e != cudaSuccess || a.max_new == 0) return e;
    const int tiles = (a.max_new * (cfg.n_heads / cfg.kv_heads) + 7) / 8, per = tiles * 8 * (RB + 16);
    const int heads = std::min(cfg.kv_heads, std::max(1, kWgRowBytes / per));
    const int ring = kWgThreads / 32 * wg_ahead<D>() * wg_stage<D>();
    const int smem = ring + heads * per + (near ? (cfg.n_req + 2) * 8 + cfg.n_req * 16 : 0);
    static std::atomic<uint64_t> allowed;
    auto k = weigh_kernel<T, D>;
    e = allow_smem(reinterpret_cast<const void*>(k), ring + std::max(kWgRowBytes, kWgMostRows * (RB + 16)) + 24 * kWgNear + 16, allowed);
    if (e != cudaSuccess) return e;
    const int64_t most = (int64_t)cfg.n_req * ((cfg.max_slots + kWgUnit - 1) / kWgUnit), ctas = (int64_t)std::min(wg_ctas<D>(), kWgSmem / (smem + 1024)) * device_sm_count();
    return launch_pdl(k, dim3((unsigned)std::min(most, ctas)), dim3(kWgThreads), smem, s, nullptr, 0, cfg, a, w, tiles, heads, near ? 1 : 0);
}

template <typename T>
static cudaError_t launch_typed(const spin_kv_config& cfg, const KvChunkArgs& a, cudaStream_t s) {
    switch (wg_dim(cfg.head_dim)) {
        case 64: return launch_dim<T, 64>(cfg, a, s);
        case 128: return launch_dim<T, 128>(cfg, a, s);
        default: return launch_dim<T, 256>(cfg, a, s);
    }
}

cudaError_t launch_kv_weigh(const spin_kv_config& cfg, const KvChunkArgs& a, cudaStream_t s) {
    if (!few_rows(cfg, a.max_new)) return launch_kv_weigh_tc(cfg, a, s);
    switch (cfg.dtype) {
        case SPIN_DTYPE_F32: return launch_typed<float>(cfg, a, s);
        case SPIN_DTYPE_BF16: return launch_typed<__nv_bfloat16>(cfg, a, s);
        default: return launch_typed<__half>(cfg, a, s);
    }
}

}  // namespace spin
