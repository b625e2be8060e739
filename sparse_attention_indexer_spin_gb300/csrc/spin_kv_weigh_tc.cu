// spin_kv_weigh_tc.cu -- the attention weight that cached slots gather from many new tokens, on tcgen05 (sm_103a).
//
//   w[r][i] <- decay w[r][i] + sum_{t, h: i <= before + t} exp(s_{t,h,i} - lse[t][h]),
//   s = softmax_scale ks (q . kc_i)
// The log-sum of a row is known, so there is no running maximum: with the row's constants
//   c = log2(e) softmax_scale 2^-k,  b = -log2(e) lse
// a weight is 2^(c ks (q 2^k . kc_i) + b).  A slot sums over rows and heads, so the product is taken with the slots as
// its rows: S = K Q^T puts a slot in each lane of tensor memory and 128 query rows in its columns, and a thread adds up
// its lane: no shuffles, no atomics, an order that depends on the sizes alone.
//
// Launches: a plan (requests' row tiles, slot tiles and their costs), the queries' row tiles (f16, scaled by a power of two
// per row, in the swizzled form that the product reads, with the rows' constants), the products, and the join of the slot
// tiles that were divided.  A unit is 128 slots of a request: for every key head, its codes become f16 in shared memory
// once and meet the row tiles that see them.  The units' costs are laid end to end and cut into equal parts, one for
// each CTA.  Warps: eight add up weights (two groups, row tiles in turn), six convert codes, one copies row tiles
// (cp.async.bulk), one issues products.
//
// What bounds it: a row tile's chain.  A row tile takes a CTA about 1700 cycles, where its product needs 512 and its
// exponentials as many; each of the two groups so takes 3400 for 128 weights a thread: loads from tensor memory, constants
// from shared memory (a value that all lanes read costs it as much as 32 of their own, so rows that share a power of two spare
// half), exponentials, sums, one behind the other.  The exponentials' pipe is 31 % active, the tensor pipe 31 %, issue 32 %.
// Four groups (80 registers, 130 us), units of 256 slots (129) and loads of the next 32 columns ahead (135: registers that
// do not fit go to L2) were slower.  (32 bytes a thread are spilled as it is.)
// Measured (32 heads on 8 of 128, bf16): 1024 tokens behind 8192 slots 116 us, 0.63 PFLOP/s and 2.5 10^12 weights a second;
// 4 x 32 tokens behind up to 32000 slots (f16, 64 heads on 8) 84 us, 0.40 PFLOP/s.
#include "spin_kv_tc.cuh"

namespace spin {

constexpr int kWtThreads = 512;
constexpr int kWtConvWarps = 6, kWtFirstConv = 8, kWtLoader = 14, kWtIssuer = 15;
constexpr int kWtSlots = 128;      // slots of a unit: the lanes of tensor memory
constexpr int kWtAcc = 4;          // accumulators in tensor memory
// Key tiles whose scales are kept.  A stage of keys is filled again when the products of two key tiles before have
// ended, and those were issued when the weights of all but the last four row tiles had been added: six are in use at most.
constexpr int kWtRing = 8;
constexpr int kWtKeyCost = 4;      // what a key head's codes cost beside its row tiles, in row tiles
constexpr int kWtMinCost = 4;
constexpr int kWtMostSms = 512;

template <int D, bool SPLIT> struct WtShape {
    static constexpr int RT = D == 256 ? 64 : 128;               // query rows of a row tile
    static constexpr int NSTK = D == 256 && SPLIT ? 1 : 2;       // stages of keys
    static constexpr int NSTQ = D == 64 ? 4 : D == 128 && !SPLIT ? 4 : 2;   // of row tiles
    static constexpr uint32_t K_BYTES = kWtSlots * D * 2;
    static constexpr uint32_t Q_TERM = RT * D * 2, Q_BYTES = Q_TERM * (SPLIT ? 2 : 1);
    static constexpr uint32_t C_BYTES = RT * 12;                 // the rows' b, their c, the slots they see
    static constexpr uint32_t COLS = kWtAcc * RT;                // 512, or 256
    static constexpr uint32_t HDR = 12 * 1024;
    static constexpr uint32_t BYTES = HDR + NSTK * K_BYTES + NSTQ * Q_BYTES + 1024;   // (slack for 1024-byte alignment)
};

struct WtPlan {
    int64_t* head;     // {row tiles, units, cost of all units}
    int4* req;         // {first token, count, slots before, first row tile}
    int* ubase;        // first unit of a request
    int2* rt;          // {request, first row} of a row tile
    int* least;        // [key heads][row tiles]: the fewest slots that a row of the tile sees
    float* same;       // [key heads][row tiles]: the rows' c where it is the same for all, else 0
    int2* unit;        // {request, slot tile}
    int64_t* begin;    // cost of the units before
    int2* owner;       // per CTA: the divided unit that it begins: {unit, pieces}
    float* rec;        // per CTA: two records of 128 sums
    unsigned char* q;  // [key heads][row tiles] images
    unsigned char* c;  // [key heads][row tiles] constants
    int rt_cap;
    int64_t u_cap;
    int ranks;
};

struct WtJob {
    int unit, req, j, before, count, rt0, nrt, first;   // rt0: the request's first row tile; rows see the unit from tile `first` on
    int g0, r0, g1, r1;                                  // row tiles [r0, ..) of head g0 to [.., r1) of head g1
    int begins, whole;
    int64_t cost0, cost;
};

struct WtWalk {
    int64_t at, end, into;
    int u;
    AtCut cut;
    __device__ __forceinline__ static int64_t ranks_of(const WtPlan& p, int64_t total) {
        return min((int64_t)p.ranks, (total + kWtMinCost - 1) / kWtMinCost);
    }
    __device__ __forceinline__ void start(const WtPlan& p, int unit, int64_t off, int64_t total) {
        cut.set(total, ranks_of(p, total));
        at = cut.begin(blockIdx.x);
        end = cut.begin(blockIdx.x + 1);
        u = unit;
        into = off;
    }
    __device__ __noinline__ bool next(const WtPlan& p, int kv_heads, int group, int rows, WtJob& j) {
        while (at < end) {
            const int64_t cost = p.begin[u + 1] - p.begin[u];
            if (into >= cost) {
                into = 0;
                ++u;
                continue;
            }
            const int64_t take = min(cost - into, end - at), per = cost / kv_heads, p0 = into, p1 = into + take;
            j.cost0 = at - into;
            j.cost = cost;
            at += take;
            into += take;
            const int tiles = (int)per - kWtKeyCost;
            j.g0 = (int)(p0 / per);
            j.r0 = (int)max((int64_t)0, p0 - j.g0 * per - kWtKeyCost);
            j.g1 = (int)((p1 - 1) / per);
            j.r1 = (int)max((int64_t)0, p1 - j.g1 * per - kWtKeyCost);
            if (j.r1 == 0) {   // nothing of the last head: up to the end of the one before
                --j.g1;
                j.r1 = tiles;
            }
            // nothing but (a part of) what a head's codes cost: the record of such a piece stays zero
            if (j.g1 < j.g0 || (j.g1 == j.g0 && j.r1 <= j.r0)) continue;
            const int2 x = p.unit[u];
            const int4 q = p.req[x.x];
            j.unit = u, j.req = x.x, j.j = x.y, j.before = q.z, j.count = q.y, j.rt0 = q.w;
            j.nrt = (int)(((int64_t)q.y * group + rows - 1) / rows);
            j.first = j.nrt - tiles;
            j.begins = j.g0 == 0 && j.r0 == 0;
            j.whole = j.begins && p1 == cost;
            return true;
        }
        return false;
    }
};

struct WtRole {
    WtWalk walk;
    WtJob job;
    int more;
};

struct WtHdr {
    uint64_t kfull[2], kempty[2];
    uint64_t qfull[4], qempty[4];
    uint64_t tfull[kWtAcc], tempty[kWtAcc], cfull[kWtAcc];
    uint64_t scale[kWtRing];  // a key tile's scales
    uint64_t half[2], sum[2]; // the second group's sums are there; the first has added them (units in turn)
    uint64_t jdone[5], jready[5];
    uint64_t fin;
    uint32_t tmem_base;
    int abort_flag, unit;
    int64_t into;
    float ks[kWtRing][2];
    float part[2][kWtSlots];
    WtRole role[5];           // the two groups, the converters, the loader, the issuer
};
static_assert(sizeof(WtHdr) <= 4096, "the header fits before the constants");

// ------------------------------------------------------------------------------- the plan
template <int ROWS>
__global__ void __launch_bounds__(1024) weigh_tc_plan_kernel(spin_kv_config cfg, KvChunkArgs a, WtPlan p) {
    pdl_begin();
    __shared__ int s_int[33];
    __shared__ int64_t s_scan[32];
    const int tid = threadIdx.x, G = cfg.n_heads / cfg.kv_heads;
    int n_rt = 0, n_units = 0;
    for_requests<1024>(cfg, a, s_int, [&](int x, int s0, int count, int before) {
        int total;
        const int at = n_rt + block_excl_scan((int)(((int64_t)count * G + ROWS - 1) / ROWS), s_int, &total);
        n_rt += total;
        const int ua = n_units + block_excl_scan(count ? (before + count + kWtSlots - 1) / kWtSlots : 0, s_int, &total);
        n_units += total;
        if (x < cfg.n_req) {
            p.req[x] = make_int4(s0, count, before, at);
            p.ubase[x] = ua;
        }
    });
    for (int r = tid; r < p.ranks; r += 1024) p.owner[r] = make_int2(0, 0);
    __syncthreads();
    n_rt = min(n_rt, p.rt_cap);
    n_units = (int)min((int64_t)n_units, p.u_cap);
    for (int k = tid; k < n_rt; k += 1024) {
        int lo = 0, hi = cfg.n_req - 1;   // the last request whose row tiles begin at or before k
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (p.req[mid].w <= k) lo = mid; else hi = mid - 1;
        }
        p.rt[k] = make_int2(lo, (k - p.req[lo].w) * ROWS);
    }
    int64_t before = 0;
    for (int base = 0; base < n_units; base += 1024) {
        const int k = base + tid;
        int64_t cost = 0;
        if (k < n_units) {
            int lo = 0, hi = cfg.n_req - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (p.ubase[mid] <= k) lo = mid; else hi = mid - 1;
            }
            const int4 q = p.req[lo];
            const int j = k - p.ubase[lo];
            p.unit[k] = make_int2(lo, j);
            const int64_t t = max(0, j * kWtSlots - q.z);     // the first token that sees the unit
            const int64_t tiles = ((int64_t)q.y * G + ROWS - 1) / ROWS - t * G / ROWS;
            cost = (tiles + kWtKeyCost) * cfg.kv_heads;
        }
        int64_t sum;
        const int64_t inc = cta_incl_scan64<32>(cost, s_scan, &sum);
        if (k < n_units) p.begin[k] = before + inc - cost;
        before += sum;
    }
    if (tid == 0) {
        p.begin[n_units] = before;
        p.head[0] = n_rt;
        p.head[1] = n_units;
        p.head[2] = before;
    }
}

// ------------------------------------------------------------------------------- row tiles
// D / 16 lanes a row, 16 values each.  Rows whose largest values are within 2^8 of each other share a power of two, and so
// c (an addition's constant is then all that a column needs); others have their own.
constexpr int kWtRowThreads = 512;
template <typename T, int D>
__global__ void __launch_bounds__(kWtRowThreads) weigh_tc_rows_kernel(spin_kv_config cfg, KvChunkArgs a, WtPlan p) {
    pdl_begin();
    constexpr bool SPLIT = std::is_same<T, float>::value;
    using S = WtShape<D, SPLIT>;
    constexpr int L = D / 16, PER = kWtRowThreads / L, RT = S::RT, N = (RT + PER - 1) / PER, QN = (int)sizeof(T);
    __shared__ int s_least, s_low, s_high;
    const int g = blockIdx.y, H = cfg.n_heads, G = H / cfg.kv_heads, d = cfg.head_dim, ch = threadIdx.x % L;
    const int n_rt = (int)p.head[0];
    for (int k = blockIdx.x; k < n_rt; k += gridDim.x) {
        if (threadIdx.x == 0) s_least = 0x7fffffff, s_low = 0x7fffffff, s_high = -0x7fffffff;
        __syncthreads();
        const int2 x = p.rt[k];
        const int4 rq = p.req[x.x];
        const int64_t tile = (int64_t)g * p.rt_cap + k;
        unsigned char* image = p.q + tile * S::Q_BYTES;
        float* cst = reinterpret_cast<float*>(p.c + tile * S::C_BYTES);
        uint4 v[N][QN];
        int own[N];      // the exponent of a row's largest value
        int64_t th[N];   // the row, -1: none
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int m = n * PER + threadIdx.x / L;
            const uint32_t R = (uint32_t)x.y + m, token = R / (uint32_t)G;
            const bool live = m < RT && token < (uint32_t)rq.y;
            th[n] = live ? ((int64_t)rq.x + token) * H + (int64_t)g * G + (R - token * G) : -1;
#pragma unroll
            for (int y = 0; y < QN; ++y)
                v[n][y] = live && 16 * ch < d ? reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(a.q) + th[n] * d + 16 * ch)[y]
                                              : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float amax = 0.0f;
#pragma unroll
            for (int y = 0; y < 16; ++y) amax = fmaxf(amax, fabsf(to_f(reinterpret_cast<const T*>(v[n])[y])));
#pragma unroll
            for (int o = L / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            // amax in [2^e, 2^(e+1)) -> [2^14, 2^15); 2^(14 - e) within [2^-113, 2^126]
            own[n] = max(-112, (int)(__float_as_uint(amax) >> 23) - 127);
            if (ch == 0 && amax > 0.0f) {     // (a row of zeros is at home anywhere)
                atomicMin(&s_low, own[n]);
                atomicMax(&s_high, own[n]);
            }
        }
        __syncthreads();
        const bool same = s_low == 0x7fffffff || s_high - s_low <= 8;   // (s_low as it was set: only zeros)
        const int common = s_low == 0x7fffffff ? 0 : s_high;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int m = n * PER + threadIdx.x / L;
            if (m >= RT) break;
            const int e = same ? common : own[n];
            const float f = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
            if (ch == 0) {
                const uint32_t token = ((uint32_t)x.y + m) / (uint32_t)G;
                const float lse = th[n] >= 0 ? a.lse[th[n]] : __uint_as_float(0xff800000u);
                // a row of no weight sees no slot, so that nothing of it is added whatever the keys are
                const int seen = lse == __uint_as_float(0xff800000u) ? 0 : rq.z + (int)token + 1;
                const float c = __uint_as_float((uint32_t)max(1, 127 - 14 + e) << 23) * (cfg.softmax_scale * 1.4426950408889634f);
                cst[m] = seen ? -1.4426950408889634f * lse : __uint_as_float(0xff800000u);
                cst[RT + m] = c;
                reinterpret_cast<int*>(cst)[2 * RT + m] = seen;
                atomicMin(&s_least, seen);
                if (m == 0) p.same[tile] = same ? c : 0.0f;   // (c = 0 is told to be different: the same outcome)
            }
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int y = 0; y < 8; ++y) {
                const float u = to_f(reinterpret_cast<const T*>(v[n])[2 * y]) * f, w = to_f(reinterpret_cast<const T*>(v[n])[2 * y + 1]) * f;
                hi[y] = pack_f16(u, w);
                const float2 z = unpack_f16(hi[y]);
                lo[y] = SPLIT ? pack_f16(u - z.x, w - z.y) : 0u;
            }
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                unsigned char* to = image + (ch >> 2) * (RT * 128) + m * 128 + (((2 * (ch & 3) + y) ^ (m & 7)) << 4);
                *reinterpret_cast<uint4*>(to) = make_uint4(hi[4 * y], hi[4 * y + 1], hi[4 * y + 2], hi[4 * y + 3]);
                if constexpr (SPLIT)
                    *reinterpret_cast<uint4*>(to + S::Q_TERM) = make_uint4(lo[4 * y], lo[4 * y + 1], lo[4 * y + 2], lo[4 * y + 3]);
            }
        }
        __syncthreads();
        if (threadIdx.x == 0) p.least[tile] = s_least;
        __syncthreads();
    }
}

// A slot's new weight from its sum; slots without a page keep theirs.
__device__ __forceinline__ void set_weight(const KvChunkArgs& a, int req, int slot, int before, int count, float sum) {
    if (slot >= before + count) return;
    const int page = a.block_table[(int64_t)req * a.bt_stride + (slot >> 6)];
    if (page < 0 || page >= a.n_pages) return;
    float* o = a.weight + (int64_t)req * a.bt_stride * kBlock + slot;
    *o = slot < before && a.decay != 0.0f ? fmaf(a.decay, *o, sum) : sum;
}

// ---------------------------------------------------------------------------- the kernel
template <int D, bool SPLIT>
__global__ void __launch_bounds__(kWtThreads, 1)
weigh_tc_kernel(const __grid_constant__ spin_kv_config cfg, const __grid_constant__ KvChunkArgs a,
                const __grid_constant__ WtPlan plan) {
    using S = WtShape<D, SPLIT>;
    constexpr int RT = S::RT, NSTK = S::NSTK, NSTQ = S::NSTQ;
    extern __shared__ unsigned char smem_raw[];
    pdl_wait();
    unsigned char* smem = reinterpret_cast<unsigned char*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    WtHdr* hdr = reinterpret_cast<WtHdr*>(smem);
    unsigned char* sC = smem + 4096;     // constants of the row tiles in the accumulators
    const uint32_t sK = smem_u32(smem) + S::HDR, sQ = sK + NSTK * S::K_BYTES;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int kvh = cfg.kv_heads, G = cfg.n_heads / kvh, d = cfg.head_dim;

    const int64_t total = plan.head[2], ranks = WtWalk::ranks_of(plan, total);
    if ((int64_t)blockIdx.x >= ranks) return;
    if (wid == kWtIssuer) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&hdr->tmem_base)),
                     "r"(S::COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&hdr->kfull[i], 32 * kWtConvWarps);
            mbar_init(&hdr->kempty[i], 1);
            mbar_init(&hdr->half[i], 128);
            mbar_init(&hdr->sum[i], 128);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&hdr->qfull[i], 1);
            mbar_init(&hdr->qempty[i], 1);
        }
        for (int i = 0; i < kWtRing; ++i) mbar_init(&hdr->scale[i], 2);
        for (int i = 0; i < kWtAcc; ++i) {
            mbar_init(&hdr->tfull[i], 1);
            mbar_init(&hdr->tempty[i], 128);
            mbar_init(&hdr->cfull[i], 1);
        }
        for (int r = 0; r < 5; ++r) {
            mbar_init(&hdr->jdone[r], r < 2 ? 128 : r == 2 ? 32 * kWtConvWarps : 32);
            mbar_init(&hdr->jready[r], 1);
        }
        mbar_init(&hdr->fin, 1);
        hdr->abort_flag = 0;
        fence_barrier_init();
    }
    // (a piece in the middle of a unit may hold no row tile: it adds zero)
    if (tid < kWtSlots) plan.rec[(int64_t)2 * blockIdx.x * kWtSlots + tid] = 0.0f;
    {   // the unit that this CTA's part begins in
        AtCut cut;
        cut.set(total, ranks);
        const int64_t at = cut.begin(blockIdx.x), n = plan.head[1];
        for (int64_t k = tid; k < n; k += kWtThreads) {
            const int64_t b = plan.begin[k];
            if (b <= at && at < plan.begin[k + 1]) {
                hdr->unit = (int)k;
                hdr->into = at - b;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = hdr->tmem_base;
    if (tid < 5) hdr->role[tid].walk.start(plan, hdr->unit, hdr->into, total);
    __syncthreads();
    auto fail_wait = [&]() {
        hdr->abort_flag = 1;
        set_status(a.status, SPIN_STATUS_TIMEOUT);
    };
    // by whole warps, which go on together
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        if (__all_sync(0xffffffffu, mbar_wait(bar, parity & 1u, &hdr->abort_flag))) return true;
        fail_wait();
        return false;
    };
    // The n-th job of role r, by all its warps; `first`: the warp whose lane 0 moves the role on.
    auto next_job = [&](int r, uint32_t n, bool first) -> bool {
        WtRole& role = hdr->role[r];
        mbar_arrive(&hdr->jdone[r]);   // the last one's fields have been read
        if (first) {
            if (!wait(&hdr->jdone[r], n)) return false;
            if (lane == 0) {
                role.more = role.walk.next(plan, kvh, G, RT, role.job);
                mbar_arrive(&hdr->jready[r]);
            }
            __syncwarp();
        }
        return wait(&hdr->jready[r], n) && role.more;
    };
    bool ok = true;
    uint32_t it = 0, kt = 0, n_job = 0;   // row tiles, key tiles, jobs so far

    if (wid < kWtFirstConv) {
        // =============================================================== weights: a slot each
        const int grp = wid >> 2, m = tid & 127;
        const uint32_t lanes = tmem + ((uint32_t)((wid & 3) * 32) << 16);
        const WtJob& job = hdr->role[grp].job;
        while (ok && next_job(grp, n_job, (wid & 3) == 0)) {
            const int g0 = job.g0, g1 = job.g1, slot0 = job.j * kWtSlots, slot = slot0 + m;
            float sum = 0.0f;
            for (int g = g0; ok && g <= g1; ++g, ++kt) {
                if (!(ok = wait(&hdr->scale[kt % kWtRing], kt / kWtRing))) break;
                const float ks = hdr->ks[kt % kWtRing][m >> 6];
                const int r_end = g == g1 ? job.r1 : job.nrt - job.first;
                const int* least = plan.least + (int64_t)g * plan.rt_cap + job.rt0 + job.first;
                const float* same = plan.same + (int64_t)g * plan.rt_cap + job.rt0 + job.first;
                const int rows = (int)min((int64_t)0x7fffffff, (int64_t)job.count * G);
                float part = 0.0f;
                int r = g == g0 ? job.r0 : 0;
                // this group's next row tile, and what is known of it, read ahead
                int ahead = r + ((int)(it & 1) != grp), l_next = ahead < r_end ? least[ahead] : 0;
                float c_next = ahead < r_end ? same[ahead] : 0.0f;
                for (; r < r_end; ++r, ++it) {
                    if ((int)(it & 1) != grp) continue;
                    const uint32_t acc = it % kWtAcc;
                    const bool border = slot0 + kWtSlots > l_next;
                    const float c_same = c_next;
                    if (r + 2 < r_end) {
                        l_next = least[r + 2];
                        c_next = same[r + 2];
                    }
                    const int cols = min(RT, rows - (job.first + r) * RT);
                    if (!(ok = wait(&hdr->cfull[acc], it / kWtAcc) && wait(&hdr->tfull[acc], it / kWtAcc))) break;
                    tc_fence_after();
                    const uint32_t tS = lanes + acc * RT;
                    const float* cb = reinterpret_cast<const float*>(sC + acc * S::C_BYTES);
                    const float* cc = cb + RT;
                    const int* seen = reinterpret_cast<const int*>(cb + 2 * RT);
                    float2 add[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                    const float2 ck = make_float2(c_same * ks, c_same * ks);
                    // (an overflow of c ks is no score's: keys of zero score 0 whatever their scale)
                    const bool plain = !border && c_same != 0.0f && fabsf(ck.x) < __uint_as_float(0x7f800000u);
                    // (a value that all lanes read costs the shared memory as much as 32 of their own: a common c spares half)
                    auto weights = [&](const float (&s)[32], int c0) {
                        if (plain) {
#pragma unroll
                            for (int x = 0; x < 32; x += 4) {
                                const float4 b = *reinterpret_cast<const float4*>(cb + c0 + x);
                                const float2 e0 = fma2(make_float2(s[x], s[x + 1]), ck, make_float2(b.x, b.y));
                                const float2 e1 = fma2(make_float2(s[x + 2], s[x + 3]), ck, make_float2(b.z, b.w));
                                add[0] = add2(add[0], make_float2(ex2(e0.x), ex2(e0.y)));
                                add[1] = add2(add[1], make_float2(ex2(e1.x), ex2(e1.y)));
                            }
                        } else {
#pragma unroll
                            for (int x = 0; x < 32; x += 2) {
                                const float p0 = ex2(fmaf(s[x] * ks, cc[c0 + x], cb[c0 + x])), p1 = ex2(fmaf(s[x + 1] * ks, cc[c0 + x + 1], cb[c0 + x + 1]));
                                add[0].x += slot < seen[c0 + x] ? p0 : 0.0f;
                                add[0].y += slot < seen[c0 + x + 1] ? p1 : 0.0f;
                            }
                        }
                    };
#pragma unroll 1
                    for (int c0 = 0; c0 < cols; c0 += 32) {
                        float s[32];
                        tm_ld32(tS + c0, s);
                        tm_wait32(s);
                        weights(s, c0);
                    }
                    tc_fence_before();
                    mbar_arrive(&hdr->tempty[acc]);
                    part += (add[0].x + add[0].y) + (add[1].x + add[1].y);
                }
                sum += part;
            }
            if (!ok) break;
            // the groups' sums together: the second's through shared memory
            const uint32_t b = n_job & 1;
            if (grp == 1) {
                if (n_job >= 2 && !wait(&hdr->sum[b], (n_job >> 1) - 1)) break;
                hdr->part[b][m] = sum;
                mbar_arrive(&hdr->half[b]);
            } else {
                if (!wait(&hdr->half[b], n_job >> 1)) break;
                sum += hdr->part[b][m];
                mbar_arrive(&hdr->sum[b]);
                if (job.whole) {
                    set_weight(a, job.req, slot, job.before, job.count, sum);
                } else {
                    plan.rec[(int64_t)(2 * blockIdx.x + job.begins) * kWtSlots + m] = sum;
                    if (job.begins && m == 0)
                        plan.owner[blockIdx.x] = make_int2(
                            job.unit, (int)(hdr->role[0].walk.cut.rank_of(job.cost0 + job.cost - 1) - blockIdx.x) + 1);
                }
            }
            ++n_job;
        }
    } else if (wid < kWtLoader) {
        // ===================================================================== converters
        constexpr int CH = D / 16, RPI = 32 / CH, NG = kWtSlots / RPI;   // chunks of a row; rows of an instruction; groups of them
        constexpr int CW = kWtConvWarps, N = (NG + CW - 1) / CW;         // a warp takes groups cw, cw + CW, ...
        const int ct = tid - kWtFirstConv * 32, cw = ct >> 5, x = lane % CH, sub = lane / CH;
        const int slot_bytes = kvh * d;
        const bool in_row = 16 * x < d;
        const int odd = (x >> 2) & 1, c2 = 2 * (x & 3);
        const uint32_t to = (uint32_t)(x >> 2) * (kWtSlots * 128) + (uint32_t)sub * 128;
        const uint32_t at0 = (uint32_t)(((c2 + odd) ^ sub) << 4), at1 = (uint32_t)(((c2 + 1 - odd) ^ sub) << 4);
        const WtJob& job = hdr->role[2].job;
        while (ok && next_job(2, n_job, cw == 0)) {
            const int len = job.before + job.count, g0 = job.g0, g1 = job.g1, j0 = job.j;
            int pg[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int block = 2 * j0 + h;
                const int p = block * kBlock < len ? a.block_table[(int64_t)job.req * a.bt_stride + block] : -2;   // -2: behind the context
                pg[h] = p >= 0 && p < a.n_pages ? p : -1;
                if (p != -2 && pg[h] < 0 && ct == 0) set_status(a.status, SPIN_STATUS_BAD_PAGE);
            }
            auto load = [&](uint4 (&v)[N], int g) {
                const uint8_t* src[2];
                int rows[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    src[h] = a.k_pool + (int64_t)max(pg[h], 0) * (kBlock * slot_bytes) + (int64_t)g * d + (in_row ? 16 * x : 0) + sub * slot_bytes;
                    rows[h] = pg[h] >= 0 && in_row ? min(kBlock, len - j0 * kWtSlots - kBlock * h) - sub : 0;
                }
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const int r = RPI * (cw + CW * n), in = r & (kBlock - 1);
                    const bool up = r >= kBlock;
                    v[n] = load_codes((up ? src[1] : src[0]) + in * slot_bytes, r < kWtSlots && in < (up ? rows[1] : rows[0]));
                }
            };
            uint4 v[2][N];
            float ks = 0.0f;
            auto scales = [&](int g) {
                const int p = ct ? pg[1] : pg[0];
                if (ct < 2) ks = p >= 0 ? a.k_scale[(int64_t)p * kvh + g] : 0.0f;
            };
            load(v[0], g0);
            scales(g0);
            auto head = [&](uint4 (&now)[N], uint4 (&next)[N], int g) {
                const uint32_t st = kt % NSTK;
                if (g < g1) load(next, g + 1);
                // the stage is free (and the scales' entry: see kempty)
                if (!(ok = wait(&hdr->kempty[st], (kt / NSTK) ^ 1u))) return;
                if (ct < 2) {
                    hdr->ks[kt % kWtRing][ct] = ks;
                    mbar_arrive(&hdr->scale[kt % kWtRing]);
                }
                __syncwarp();
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const int r = RPI * (cw + CW * n);
                    if (NG % CW && r >= kWtSlots) break;
                    const uint32_t line = sK + st * S::K_BYTES + to + (uint32_t)r * 128, sw = (uint32_t)(r & 7) << 4;
                    store_codes(line + (at0 ^ sw), line + (at1 ^ sw), odd, now[n]);
                }
                fence_async_smem();
                mbar_arrive(&hdr->kfull[st]);
                ++kt;
                if (g < g1) scales(g + 1);
            };
            for (int g = g0; ok && g <= g1; g += 2) {
                head(v[0], v[1], g);
                if (ok && g < g1) head(v[1], v[0], g + 1);
            }
            ++n_job;
        }
    } else if (wid == kWtLoader) {
        // ============================================================= loader of row tiles
        const WtJob& job = hdr->role[3].job;
        uint32_t tiles = 0, csts = 0;   // copies asked for
        while (ok && next_job(3, n_job, true)) {
            const int g0 = job.g0, g1 = job.g1;
            for (int g = g0; ok && g <= g1; ++g) {
                const int r_end = g == g1 ? job.r1 : job.nrt - job.first;
                const int64_t tile0 = (int64_t)g * plan.rt_cap + job.rt0 + job.first;
                for (int r = g == g0 ? job.r0 : 0; r < r_end; ++r, ++it) {
                    const uint32_t st = it % NSTQ, acc = it % kWtAcc;
                    if (!(ok = wait(&hdr->qempty[st], (it / NSTQ) ^ 1u))) break;
                    if (elect_one()) {
                        mbar_arrive_expect_tx(&hdr->qfull[st], S::Q_BYTES);
                        bulk_g2s(smem + S::HDR + NSTK * S::K_BYTES + st * S::Q_BYTES, plan.q + (tile0 + r) * S::Q_BYTES, S::Q_BYTES,
                                 &hdr->qfull[st]);
                    }
                    __syncwarp();
                    ++tiles;
                    if (!(ok = wait(&hdr->tempty[acc], (it / kWtAcc) ^ 1u))) break;
                    if (elect_one()) {
                        mbar_arrive_expect_tx(&hdr->cfull[acc], S::C_BYTES);
                        bulk_g2s(sC + acc * S::C_BYTES, plan.c + (tile0 + r) * S::C_BYTES, S::C_BYTES, &hdr->cfull[acc]);
                    }
                    __syncwarp();
                    ++csts;
                }
            }
            ++n_job;
        }
        // never leave with copies in flight: the last fill of every stage (waits that nothing cuts short but time)
        for (uint32_t i = 0; i < NSTQ && i < tiles; ++i) {
            const uint32_t x = tiles - 1 - i;
            if (!mbar_wait(&hdr->qfull[x % NSTQ], (x / NSTQ) & 1u, nullptr)) set_status(a.status, SPIN_STATUS_TIMEOUT);
        }
        for (uint32_t i = 0; i < kWtAcc && i < csts; ++i) {
            const uint32_t x = csts - 1 - i;
            if (!mbar_wait(&hdr->cfull[x % kWtAcc], (x / kWtAcc) & 1u, nullptr)) set_status(a.status, SPIN_STATUS_TIMEOUT);
        }
    } else {
        // ========================================================================= issuer
        constexpr uint32_t A_REGION = kWtSlots * 128, B_REGION = RT * 128;
        const int ksteps = d / 16;
        bool issued = false;
        const WtJob& job = hdr->role[4].job;
        while (ok && next_job(4, n_job, true)) {
            const int g0 = job.g0, g1 = job.g1;
            const int64_t rows = (int64_t)job.count * G;
            for (int g = g0; ok && g <= g1; ++g, ++kt) {
                const uint32_t sk = kt % NSTK;
                if (!(ok = wait(&hdr->kfull[sk], kt / NSTK))) break;
                const int r_end = g == g1 ? job.r1 : job.nrt - job.first;
                for (int r = g == g0 ? job.r0 : 0; r < r_end; ++r, ++it) {
                    const uint32_t sq = it % NSTQ, acc = it % kWtAcc;
                    if (!(ok = wait(&hdr->qfull[sq], it / NSTQ) && wait(&hdr->tempty[acc], (it / kWtAcc) ^ 1u))) break;
                    tc_fence_after();
                    const int n = (int)min((int64_t)RT, rows - (int64_t)(job.first + r) * RT);
                    const uint32_t idesc = idesc_mma(0u, (uint32_t)((n + 15) & ~15), 128);
                    if (elect_one()) {
                        const uint64_t a0 = smem_desc_sw128(sK + sk * S::K_BYTES);
#pragma unroll
                        for (int z = 0; z < (SPLIT ? 2 : 1); ++z) {
                            const uint64_t b0 = smem_desc_sw128(sQ + sq * S::Q_BYTES + z * S::Q_TERM);
#pragma unroll
                            for (int k = 0; k < D / 16; ++k)
                                if (k < ksteps)
                                    tc_mma_f16(tmem + acc * RT, a0 + (uint64_t)((k >> 2) * (A_REGION >> 4) + 2 * (k & 3)),
                                               b0 + (uint64_t)((k >> 2) * (B_REGION >> 4) + 2 * (k & 3)), idesc, (z | k) ? 1u : 0u);
                        }
                        tc_commit(&hdr->qempty[sq]);
                        tc_commit(&hdr->tfull[acc]);
                    }
                    issued = true;
                    __syncwarp();
                }
                if (!ok) break;
                if (elect_one()) tc_commit(&hdr->kempty[sk]);
                __syncwarp();
            }
            ++n_job;
        }
        if (issued) {   // every product has ended before tensor memory is released
            if (elect_one()) tc_commit(&hdr->fin);
            __syncwarp();
            if (!mbar_wait(&hdr->fin, 0u, nullptr)) set_status(a.status, SPIN_STATUS_TIMEOUT);
        }
    }
    pdl_trigger();
    tc_fence_before();
    __syncthreads();
    if (wid == kWtIssuer) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::COLS) : "memory");
    }
}

// The divided units: the first piece lies in the second record of the CTA that begins the unit, the others in the
// first records of the CTAs after it.
__global__ void __launch_bounds__(kWtSlots) weigh_tc_join_kernel(spin_kv_config cfg, KvChunkArgs a, WtPlan p) {
    pdl_begin();
    const int2 o = p.owner[blockIdx.x];
    if (o.y == 0) return;
    const int m = threadIdx.x;
    const float* rec = p.rec + (int64_t)2 * blockIdx.x * kWtSlots + m;
    float sum = rec[kWtSlots];
    for (int i = 1; i < o.y; ++i) sum += rec[(int64_t)2 * i * kWtSlots];
    const int2 x = p.unit[o.x];
    const int4 q = p.req[x.x];
    set_weight(a, x.x, x.y * kWtSlots + m, q.z, q.y, sum);
}

// ------------------------------------------------------------------------------ host side
static int wt_dim(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }
static int wt_sms() {
    const int n = device_sm_count();
    return n < kWtMostSms ? n : kWtMostSms;
}

static size_t wt_layout(const spin_kv_config& cfg, int64_t n_tokens, void* ws, WtPlan* out) {
    const int D = wt_dim(cfg.head_dim), RT = D == 256 ? 64 : 128, terms = cfg.dtype == SPIN_DTYPE_F32 ? 2 : 1;
    const int64_t G = cfg.n_heads / cfg.kv_heads, rt = n_tokens * G / RT + cfg.n_req;
    const int64_t units = (int64_t)cfg.n_req * ((cfg.max_slots + kWtSlots - 1) / kWtSlots);
    const size_t sms = (size_t)wt_sms();
    char* c = reinterpret_cast<char*>(ws);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char* x = c + at;
        at += (bytes + 255) & ~(size_t)255;
        return x;
    };
    WtPlan p;
    p.head = reinterpret_cast<int64_t*>(take(24));
    p.req = reinterpret_cast<int4*>(take((size_t)cfg.n_req * sizeof(int4)));
    p.ubase = reinterpret_cast<int*>(take((size_t)cfg.n_req * sizeof(int)));
    p.rt = reinterpret_cast<int2*>(take((size_t)rt * sizeof(int2)));
    p.least = reinterpret_cast<int*>(take((size_t)rt * cfg.kv_heads * sizeof(int)));
    p.same = reinterpret_cast<float*>(take((size_t)rt * cfg.kv_heads * sizeof(float)));
    p.unit = reinterpret_cast<int2*>(take((size_t)units * sizeof(int2)));
    p.begin = reinterpret_cast<int64_t*>(take((size_t)(units + 1) * sizeof(int64_t)));
    p.owner = reinterpret_cast<int2*>(take(sms * sizeof(int2)));
    p.rec = reinterpret_cast<float*>(take(sms * 2 * kWtSlots * sizeof(float)));
    p.q = reinterpret_cast<unsigned char*>(take((size_t)rt * cfg.kv_heads * RT * D * 2 * terms));
    p.c = reinterpret_cast<unsigned char*>(take((size_t)rt * cfg.kv_heads * RT * 12));
    p.rt_cap = (int)rt;
    p.u_cap = units;
    p.ranks = (int)sms;
    if (out) *out = p;
    return at;
}

size_t kv_weigh_tc_workspace_bytes(const spin_kv_config& cfg, int64_t n_tokens) { return wt_layout(cfg, n_tokens, nullptr, nullptr); }

template <typename T, int D>
static cudaError_t launch_dim(const spin_kv_config& cfg, const KvChunkArgs& a, cudaStream_t s) {
    constexpr bool SPLIT = std::is_same<T, float>::value;
    using S = WtShape<D, SPLIT>;
    static std::atomic<uint64_t> allowed;
    auto k = weigh_tc_kernel<D, SPLIT>;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), S::BYTES, allowed);
    if (e != cudaSuccess) return e;
    WtPlan p;
    wt_layout(cfg, a.n_tokens, a.workspace, &p);
    e = launch_pdl(weigh_tc_plan_kernel<S::RT>, dim3(1), dim3(1024), 0, s, nullptr, 0, cfg, a, p);
    if (e != cudaSuccess || a.max_new == 0) return e;
    e = launch_pdl(weigh_tc_rows_kernel<T, D>, dim3(p.rt_cap < 4096 ? p.rt_cap : 4096, cfg.kv_heads), dim3(kWtRowThreads), 0, s, nullptr, 0, cfg, a, p);
    if (e == cudaSuccess) e = launch_pdl(k, dim3(p.ranks), dim3(kWtThreads), S::BYTES, s, nullptr, 0, cfg, a, p);
    if (e == cudaSuccess) e = launch_pdl(weigh_tc_join_kernel, dim3(p.ranks), dim3(kWtSlots), 0, s, nullptr, 0, cfg, a, p);
    return e;
}

template <typename T>
static cudaError_t launch_typed(const spin_kv_config& cfg, const KvChunkArgs& a, cudaStream_t s) {
    switch (wt_dim(cfg.head_dim)) {
        case 64: return launch_dim<T, 64>(cfg, a, s);
        case 128: return launch_dim<T, 128>(cfg, a, s);
        default: return launch_dim<T, 256>(cfg, a, s);
    }
}

cudaError_t launch_kv_weigh_tc(const spin_kv_config& cfg, const KvChunkArgs& a, cudaStream_t s) {
    switch (cfg.dtype) {
        case SPIN_DTYPE_F32: return launch_typed<float>(cfg, a, s);
        case SPIN_DTYPE_BF16: return launch_typed<__nv_bfloat16>(cfg, a, s);
        default: return launch_typed<__half>(cfg, a, s);
    }
}

}  // namespace spin
