// spin_kv_prefill.cu -- attention of ragged chunks of new tokens over the paged 8-bit KV cache (sm_103a).
//
// Per new token and head, over the slots up to the token's own:
//   s_i = softmax_scale ks (q . kc_i),  out = sum_i e^{s_i} vs vc_i / sum_i e^{s_i},  lse = ln sum_i e^{s_i}
// in one pass over the slots, with the running maximum and sum of the softmax.  The numbers are
// spin_kv_attend's (see there): exponents in base 2, a reference that follows max(t_i + log2 vs_i) - 9 and moves
// only when a weight (or a page's sum) would leave f16's range, weights times value scale rounded to f16, queries
// scaled by a power of two per row and rounded to f16; for fp32 both as two f16 terms.
//
// Shape.  A job is a key/value head of a chunk of a request's query rows (token by token, the heads of the group
// side by side): 256 rows as two tiles of 128, or one tile.  The codes of two pages (one where heads are wider
// than 128) become f16 in shared memory once for all the job's rows, and tcgen05.mma multiplies:
//   S = Q K^T   both from shared memory, into tensor memory
//   O += P V    P written over S in tensor memory by the threads that hold the rows, V as it lies (N-major)
// Warps: four per row tile hold a row a thread (scores, weights, and the rare rescaling of O); six (ten beside
// one row tile) convert codes; one works out the jobs, and one
// thread issues the products.  Two row tiles take turns, one's products running
// while the other's weights are computed; a single one has two buffers of scores instead.
//
// The jobs' costs are laid end to end by a planning launch and cut into equal parts, one for each CTA; the pieces of
// divided jobs are joined by a last launch.
//
// What bounds it: a chain, not a pipe.  A tile of 128 slots and 256 rows takes about 3700 cycles where its products need
// 2048 (64 cycles an instruction of 128 x 128 x 16, measured alone): a row tile's scores have to end (517 cycles, and 300
// until a waiting warp knows), its two pages become weights (about 1000 cycles each: tensor memory, exponentials at 8 a
// cycle and quarter, packing, tensor memory), and the last page's product has to end before the next scores may overwrite the
// weights (258 and 300).  With two row tiles all of tensor memory is taken (scores 2 x 128 columns, sums 2 x 128), so
// that scores cannot be a tile ahead.  How the issuing loop is laid out counts: with the row tiles unrolled 951 -> 857 us at
// 2048 tokens behind 32768 slots (ragged prompts 145 -> 152: a loop twice as long, whose code is fetched cold).  Slower there (from 951): the next scores page by page (1357:
// 128 x 64 x 16 takes 48 cycles, not 32, and the issuing thread waits for room after four instructions); eight warps a row
// tile, half a tile's slots each (1388: 80 registers a thread, and what does not fit comes from L2, as 201 KB of shared
// memory leave little first-level cache); the second page's scores loaded while the first page's weights are stored (1075: the
// page's code twice).  Leaving out row tiles without a row: turns 269 -> 256, prompts 145 -> 160 in the loop before; in this one
// the long chunk, which has no such tile, 857 -> 938.  No instance spills a register; the code of a job's start and end is fetched cold, and what is
// added there shows in short jobs (prompts 157 -> 160 us with the sums that leave tensor memory and the second factor of zero keys).
// Measured (bf16, 32 heads on 8 of 128): 2048 tokens behind 32768 slots 855 us, 1.33 PFLOP/s (0.68 of the measured
// product rate); 8 ragged prompts of 100 to 2048 tokens 160 us, 0.39 PFLOP/s: short jobs, whose queries, first scores and
// outputs nothing overlaps, on the diagonal, where half a tile's products are masked.  16 turns of 5 to 32 tokens behind up to
// 32000 slots (f16, 64 heads on 8) 239 us, 0.52 PFLOP/s counted in rows that are there: row tiles are partly filled.
#include "spin_kv_chunk.cuh"
#include "spin_kv_tc.cuh"

namespace spin {

constexpr int kPfRows = 128;       // rows of a row tile: the lanes of tensor memory
constexpr int kPfRing = 8;         // tiles whose scales are kept (see kempty)
constexpr int kPfThreads = 512;    // 16 warps: four for each row tile, one planner, one issuer, the rest converters
constexpr int kPfIssuer = kPfThreads / 32 - 1, kPfPlanner = kPfIssuer - 1;
constexpr int kPfJobs = 4;         // jobs worked out ahead
// What starting a job costs, in tiles of slots: one value for all shapes (prompts of many short jobs, turns on long contexts:
// 2 161, 276 us; 4 151, 251; 5 154, 247; 7 155, 242).
constexpr int kPfJobUnits = 7;
// Cost a CTA takes at least, in tiles of slots.  Less than a job's start: in small calls a part may lie within one and hold no tile
// (its CTA works out no job and leaves).
constexpr int kPfMinCost = 4;
constexpr int kPfMostSms = 512;
// Slots whose products tensor memory adds up (half as many more at a job's end) before the sums leave it for a record that is
// added to with rounding to nearest.  Tensor memory's own additions, one for 16 slots (two for fp32), cut off: 2^-24 of the sum
// each on average, all in one direction.  Without this a CTA's 2^20 slots of one sign came out 0.1 % short, 2^24 7 %.
__host__ __device__ constexpr int pf_fold(bool split) { return split ? 4096 : 32768; }
constexpr float kPfTop = 9.0f;     // log2 of the largest weight when the reference is set: 64 of them are within f16
constexpr float kPfSlack = 6.0f;   // a maximum may exceed that by this much before the reference moves

template <typename T, int D, int NQ> struct PfShape {
    static constexpr bool SPLIT = std::is_same<T, float>::value;
    static constexpr int BN = D == 256 ? 64 : 128, HALVES = BN / kBlock;   // slots, pages of a tile
    static constexpr int SB = NQ == 2 ? 1 : 2;                  // buffers of scores
    static constexpr int NST = D == 64 ? 4 : D == 256 && SPLIT ? 1 : 2;    // stages of codes as f16
    static constexpr int CW = 14 - 4 * NQ, CONV = 32 * CW;      // converting warps, threads
    static constexpr uint32_t Q_TILE = kPfRows * D * 2;         // a row tile's queries (one f16 term)
    static constexpr uint32_t Q_BYTES = NQ * Q_TILE * (SPLIT ? 2 : 1);
    static constexpr uint32_t KV = BN * D * 2;                  // keys, or values, of a stage
    static constexpr uint32_t COLS = NQ * (SB * BN + D) > 256 ? 512 : 256;
    static constexpr int FOLD = pf_fold(SPLIT) / BN;            // tiles between two of those, a power of two
    static constexpr uint32_t HDR = 4096;
    static constexpr uint32_t BYTES = HDR + Q_BYTES + NST * 2 * KV + 1024;   // (slack for 1024-byte alignment)
};

// ------------------------------------------------------------------------------- the plan
struct PfPlan {
    int64_t* head;      // {chunks, cost of all jobs}
    int64_t* begin;     // [chunks + 1] cost of the chunks before, for one key head
    int4* chunk;        // {request, first row of the chunk, longest row's slots, slots before the new tokens}
    int2* tokens;       // {first token, count} of the chunk's request
    int4* owner;        // per CTA: the divided job that it begins: {chunk, key head, pieces, 0}
    float* rec;         // two records per CTA: rows x D sums, then (reference, sum) of each row
    float* fold;        // per CTA: D x rows sums that left tensor memory (where contexts are long enough)
    int* base;          // [requests + 1] chunks before
    int most;           // chunks that fit
    int ranks;          // CTAs that may work
};

// --------------------------------------------------------------------------- a CTA's jobs
struct PfJob {
    int more;        // 0: there is none
    int req, g, row0, len, before, t0, count, units, u0, u1, chunk;
    int pieces;      // of a divided job, where it begins
};

struct PfWalk {
    int64_t at, end, into;
    int k, g;
    AtCut cut;

    __device__ __forceinline__ void start(const PfPlan& p, int chunk, int64_t off, int kv_heads, int64_t total) {
        cut.set(total, pf_ranks(p, total));
        at = cut.begin(blockIdx.x);
        end = cut.begin(blockIdx.x + 1);
        k = chunk;
        const int64_t cost = p.begin[k + 1] - p.begin[k];
        g = (int)quotient(off, cost);
        into = off - g * cost;
    }
    __device__ __forceinline__ static int64_t pf_ranks(const PfPlan& p, int64_t total) {
        return min((int64_t)p.ranks, (total + kPfMinCost - 1) / kPfMinCost);
    }
    template <int BN> __device__ __noinline__ void next(const PfPlan& p, int kv_heads, PfJob& j) {
        j.more = 0;
        while (at < end) {
            const int4 c = p.chunk[k];
            const int2 t = p.tokens[k];
            const int units = (c.z + BN - 1) / BN;
            const int64_t cost = units + kPfJobUnits;
            if (into >= cost) {
                into = 0;
                if (++g == kv_heads) g = 0, ++k;
                continue;
            }
            const int64_t take = min(cost - into, end - at), cost0 = at - into;
            j.u0 = (int)max((int64_t)0, into - kPfJobUnits);
            j.u1 = (int)max((int64_t)0, into + take - kPfJobUnits);
            at += take;
            into += take;
            if (j.u0 == j.u1) continue;   // the part ends before the job's first tile
            j.req = c.x, j.row0 = c.y, j.len = c.z, j.before = c.w, j.t0 = t.x, j.count = t.y, j.units = units, j.g = g,
            j.chunk = k;
            // up to the CTA that holds the end of the job's cost
            j.pieces = j.u0 == 0 && j.u1 < units ? (int)(cut.rank_of(cost0 + cost - 1) - blockIdx.x) + 1 : 0;
            j.more = 1;
            return;
        }
    }
};

struct alignas(16) PfScale {   // what a page's scales mean for its slots' weights; live: the page is there
    float ks, lv, iv, ratio;
    int live, odd, pad[2];
};

struct PfHdr {
    uint64_t kfull[4], kempty[4], vfull[4], vempty[4];
    uint64_t qready[2];   // a job's queries are in shared memory (128 threads)
    // (row tile, tiles in turn: a barrier tells a phase from the next one only)
    uint64_t sfull[2][2]; // scores are in tensor memory
    uint64_t pready[2][2][2];   // a page's weights are in tensor memory (128 threads)
    uint64_t padone[2][2];   // O has the first page's
    uint64_t pvdone[2][2];   // O has the tile's
    uint64_t scale[kPfRing];
    uint64_t cdone[2];    // a job's codes are converted (jobs in turn)
    uint64_t epi[2];      // a job's outputs are out (jobs in turn)
    uint64_t jready[kPfJobs], jdone[kPfJobs];   // a job is there; every warp has read it
    uint64_t fin;
    uint32_t tmem_base;
    int abort_flag;
    uint32_t tiles;       // whose codes the converters have begun with: what moves while a job goes on
    int64_t into;
    int chunk;
    PfScale sc[kPfRing][2];
    PfJob job[kPfJobs];   // (in shared memory: registers are few, and local memory is far beside this much of it)
    alignas(16) int nan[2][256];   // jobs in turn: per dimension, the first slot of a NaN that only some rows see
};
static_assert(sizeof(PfHdr) <= 4096, "the header fits");
static_assert(offsetof(PfHdr, nan) % 16 == 0 && offsetof(PfHdr, sc) % 16 == 0, "read 16 bytes at a time");

// k of a row's largest value in [2^k, 2^(k+1)), which is scaled to [2^14, 2^15); 2^(14 - k) within [2^-113, 2^126].
__device__ __forceinline__ int pow2_of(float amax) { return max(-112, (int)(__float_as_uint(amax) >> 23) - 127); }

__host__ __device__ inline int pf_dim(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }

// One CTA: chunks of every request, then each chunk's row range and cost.
constexpr int kPfNear = 1024;   // requests whose places the plan keeps in shared memory

template <int ROWS, int BN>
__global__ void __launch_bounds__(1024) prefill_plan_kernel(spin_kv_config cfg, KvChunkArgs a, PfPlan p) {
    pdl_begin();
    __shared__ int s_int[33], s_base[kPfNear];
    __shared__ int64_t s_scan[32];
    __shared__ int3 s_req[kPfNear];   // {first token, count, slots before}
    const int tid = threadIdx.x, G = cfg.n_heads / cfg.kv_heads;
    const bool near = cfg.n_req <= kPfNear;
    int n_chunks = 0;
    for_requests<1024>(cfg, a, s_int, [&](int x, int s0, int count, int before) {
        const int64_t c = ((int64_t)count * G + ROWS - 1) / ROWS;
        int total;
        const int at = n_chunks + block_excl_scan((int)c, s_int, &total);
        if (near) {
            s_base[x] = at;
            s_req[x] = make_int3(s0, count, before);
        } else if (x < cfg.n_req) {
            p.base[x] = at;
        }
        n_chunks += total;
    });
    for (int r = tid; r < p.ranks; r += 1024) p.owner[r] = make_int4(0, 0, 0, 0);
    __syncthreads();
    n_chunks = min(n_chunks, p.most);   // (not more: requests that were counted do not share tokens)
    const int* at = near ? s_base : p.base;
    int64_t before = 0;
    for (int base = 0; base < n_chunks; base += 1024) {
        const int k = base + tid;
        int64_t cost = 0;
        if (k < n_chunks) {
            int lo = 0, hi = cfg.n_req - 1;   // the last request whose chunks begin at or before k
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (at[mid] <= k) lo = mid; else hi = mid - 1;
            }
            int3 r;
            if (near) r = s_req[lo];
            else r = make_int3(a.new_start[lo], a.new_start[lo + 1] - a.new_start[lo], a.n_before[lo]);
            const int row0 = (k - at[lo]) * ROWS;
            const int last = min(r.y - 1, (int)(((uint32_t)row0 + ROWS - 1) / (uint32_t)G));
            const int len = r.z + last + 1;
            p.chunk[k] = make_int4(lo, row0, len, r.z);
            p.tokens[k] = make_int2(r.x, r.y);
            cost = (len + BN - 1) / BN + kPfJobUnits;
        }
        int64_t sum;
        const int64_t inc = cta_incl_scan64<32>(cost, s_scan, &sum);
        if (k < n_chunks) p.begin[k] = before + inc - cost;
        before += sum;
    }
    if (tid == 0) {
        p.begin[n_chunks] = before;
        p.head[0] = n_chunks;
        p.head[1] = before * cfg.kv_heads;
    }
}

// A page's weights over its scores: f16 pairs, or for fp32 the two terms of 32 slots side by side.
template <bool SPLIT> __device__ __forceinline__ void store_weights(uint32_t tS, const float (&s)[kBlock]) {
#pragma unroll
    for (int y = 0; y < kBlock; y += 32) {
        uint32_t w[16], e[16];
#pragma unroll
        for (int x = 0; x < 16; ++x) {
            w[x] = pack_f16(s[y + 2 * x], s[y + 2 * x + 1]);
            if constexpr (SPLIT) {
                const float2 f = unpack_f16(w[x]);
                e[x] = pack_f16(s[y + 2 * x] - f.x, s[y + 2 * x + 1] - f.y);
            }
        }
        if constexpr (SPLIT) {
            tm_st16(tS + y, w);
            tm_st16(tS + y + 16, e);
        } else {
            tm_st16(tS + y / 2, w);
        }
    }
}

// A row's sums leave tensor memory for the record (`again`: which has some, under factor f).  Out of line, and the loop over
// tiles inside one over stretches: with this code in the loop a single row tile took 4 to 7 % longer for every tile (one token
// on 2^20 slots a CTA, bf16: 9.8 ms without it, 10.5 in the loop, 10.1 here; fp32, eight times as often: 13.7, 15.0, 14.7).
template <int ROWS> __device__ __noinline__ void fold_sums(uint32_t tO, int d, float* to, bool again, float f) {
#pragma unroll 1
    for (int c = 0; c < d; c += 16, to += 16 * ROWS) {
        float o[16], y[16];
        const uint32_t none[16] = {};
#pragma unroll
        for (int x = 0; x < 16; ++x) y[x] = again ? to[x * ROWS] : 0.0f;
        tm_ld16(tO + c, o);
        tm_st16(tO + c, none);
#pragma unroll
        for (int x = 0; x < 16; ++x) to[x * ROWS] = again ? fmaf(y[x], f, o[x]) : o[x];
    }
    tm_wait_st();
}

// ---------------------------------------------------------------------------- the kernel
template <typename T, int D, int NQ>
__global__ void __launch_bounds__(kPfThreads, 1)
prefill_kernel(const __grid_constant__ spin_kv_config cfg, const __grid_constant__ KvChunkArgs a,
               const __grid_constant__ PfPlan plan) {
    using S = PfShape<T, D, NQ>;
    constexpr bool SPLIT = S::SPLIT;
    constexpr int BN = S::BN, HALVES = S::HALVES, SB = S::SB, NST = S::NST, ROWS = NQ * kPfRows;
    extern __shared__ unsigned char smem_raw[];
    pdl_wait();
    unsigned char* smem = reinterpret_cast<unsigned char*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    PfHdr* hdr = reinterpret_cast<PfHdr*>(smem);
    const uint32_t sQ = smem_u32(smem) + S::HDR, sKV = sQ + S::Q_BYTES;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, wg = wid >> 2;
    const int H = cfg.n_heads, kvh = cfg.kv_heads, G = H / kvh, d = cfg.head_dim;
    const float ninf = __uint_as_float(0xff800000u);

    // ------------------------------------------------------------------------------ set-up
    const int n_chunks = (int)plan.head[0];
    const int64_t total = plan.head[1];
    if ((int64_t)blockIdx.x >= PfWalk::pf_ranks(plan, total)) return;   // (the CTAs from here on have no part)
    if (wid == kPfIssuer) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&hdr->tmem_base)),
                     "r"(S::COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else if (tid == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(&hdr->kfull[i], S::CONV);
            mbar_init(&hdr->vfull[i], S::CONV);
            mbar_init(&hdr->kempty[i], 1);
            mbar_init(&hdr->vempty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&hdr->qready[i], kPfRows);
            mbar_init(&hdr->sfull[i][0], 1);
            mbar_init(&hdr->sfull[i][1], 1);
            for (int h = 0; h < 2; ++h) {
                mbar_init(&hdr->pready[i][h][0], kPfRows);
                mbar_init(&hdr->pready[i][h][1], kPfRows);
                mbar_init(&hdr->padone[i][h], 1);
            }
            mbar_init(&hdr->pvdone[i][0], 1);
            mbar_init(&hdr->pvdone[i][1], 1);
            mbar_init(&hdr->cdone[i], S::CONV);
            mbar_init(&hdr->epi[i], NQ * kPfRows);
        }
        for (int i = 0; i < kPfRing; ++i) mbar_init(&hdr->scale[i], HALVES);
        for (int i = 0; i < kPfJobs; ++i) {
            mbar_init(&hdr->jready[i], 1);
            mbar_init(&hdr->jdone[i], NQ * kPfRows + S::CONV + 32);
        }
        mbar_init(&hdr->fin, 1);
        hdr->abort_flag = 0;
        hdr->tiles = 0;
        fence_barrier_init();
    }
    {   // the chunk that this CTA's part begins in
        AtCut cut;
        cut.set(total, PfWalk::pf_ranks(plan, total));
        const int64_t at = cut.begin(blockIdx.x);
        for (int k = tid; k < n_chunks; k += kPfThreads) {
            const int64_t b = plan.begin[k] * kvh;
            if (b <= at && at < plan.begin[k + 1] * kvh) {
                hdr->chunk = k;
                hdr->into = at - b;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = hdr->tmem_base;
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

    auto job_there = [&](uint32_t n) -> bool { return wait(&hdr->jready[n % kPfJobs], n / kPfJobs) && hdr->job[n % kPfJobs].more; };
    auto job_read = [&](uint32_t n) { mbar_arrive(&hdr->jdone[n % kPfJobs]); };

    if (wg < NQ) {
        // ================================================================= rows: a thread each
        const int i = wg, m = tid & 127;
        const uint32_t lanes = tmem + ((uint32_t)((wid & 3) * 32) << 16);
        const uint32_t tO = lanes + (uint32_t)(NQ * SB * BN + i * D);
        uint32_t it = 0, n_job = 0;
        bool ok = true;
        // 16-byte vectors of a row (of queries, of outputs); rows that an instruction of the warp moves; vectors of a lane
        constexpr int VB = 16 / (int)sizeof(T), LPR = D / VB, RPI = LPR < 32 ? 32 / LPR : 1, VPL = LPR < 32 ? 1 : LPR / 32;
        constexpr int NI = 32 / RPI, NB = 16 / VPL < NI ? 16 / VPL : NI;   // instructions for the warp's 32 rows; in flight
        const uint32_t tile = sQ + (uint32_t)i * S::Q_TILE * (SPLIT ? 2u : 1u);
        // byte b of a row's line: regions of 128 bytes a row, 16-byte chunks swizzled as the product reads them
        auto line = [&](int row, int b) -> uint32_t {
            return tile + (uint32_t)(b >> 7) * (kPfRows * 128) + (uint32_t)row * 128 + (uint32_t)((((b >> 4) ^ row) & 7) << 4) + (b & 15);
        };
        const int w0 = (wid & 3) * 32, sub = lane / (LPR < 32 ? LPR : 32), vec = lane % LPR;   // the warp's first row; this lane's place
        while (ok && job_there(n_job)) {
            const PfJob& job = hdr->job[n_job % kPfJobs];
            // ---- queries: scaled by a power of two and rounded to f16, as swizzled rows of 64 values
            const uint32_t R = (uint32_t)job.row0 + i * kPfRows + m;   // (below 2^31 + 256)
            const uint32_t token = R / (uint32_t)G;
            const bool mine = token < (uint32_t)job.count;
            const int row = mine ? (int)((job.t0 + token) * (uint32_t)H + job.g * G + (R - token * G)) : -1;   // (below 2^31)
            const int lim = mine ? job.before + (int)token + 1 : job.len;
            const uint32_t token0 = (R - m) / (uint32_t)G;       // the tile's shortest row
            const int lim0 = token0 < (uint32_t)job.count ? job.before + (int)token0 + 1 : job.len;
            float amax = 0.0f;
            if constexpr (!SPLIT) {
                // copied as they are, the warp's rows one after another, then made f16 in their places, a row a thread
                // (small loops: this code runs once a job and is fetched cold)
#pragma unroll 4
                for (int n = 0; n < NI; ++n) {
                    const int from = RPI * n + sub, r = __shfl_sync(0xffffffffu, row, from);
                    const bool live = r >= 0 && vec * VB < d;
                    cp16(line(w0 + from, 16 * vec), reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(a.q) + (int64_t)max(r, 0) * d) + (live ? vec : 0), live);
                }
                cp_commit();
                cp_wait<0>();
                __syncwarp();
                uint32_t most = 0;
#pragma unroll 4
                for (int x = 0; x < LPR; ++x) {
                    const uint4 v = lds128(line(m, 16 * x));
                    most = abs_max2(abs_max2(abs_max2(abs_max2(most, v.x, (const T*)nullptr), v.y, (const T*)nullptr), v.z, (const T*)nullptr), v.w,
                                    (const T*)nullptr);
                }
                amax = abs_max_of(most, (const T*)nullptr);
                const float f = __uint_as_float((uint32_t)(127 + 14 - pow2_of(amax)) << 23);
#pragma unroll 4
                for (int x = 0; x < LPR; ++x) {
                    const uint32_t at = line(m, 16 * x);
                    const uint4 v = lds128(at);
                    const T* y = reinterpret_cast<const T*>(&v);
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(pack_f16(to_f(y[0]) * f, to_f(y[1]) * f)),
                                 "r"(pack_f16(to_f(y[2]) * f, to_f(y[3]) * f)), "r"(pack_f16(to_f(y[4]) * f, to_f(y[5]) * f)),
                                 "r"(pack_f16(to_f(y[6]) * f, to_f(y[7]) * f))
                                 : "memory");
                }
            } else {
                // the warp's rows one after another, 16 bytes a lane
                const T* q = reinterpret_cast<const T*>(a.q);
#pragma unroll 1
                for (int n0 = 0; n0 < NI; n0 += NB) {
                    uint4 v[NB][VPL];
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        const int r = __shfl_sync(0xffffffffu, row, RPI * (n0 + n) + sub);
#pragma unroll
                        for (int y = 0; y < VPL; ++y) {
                            const bool live = r >= 0 && (vec + 32 * y) * VB < d;
                            v[n][y] = live ? __ldg(reinterpret_cast<const uint4*>(q + (int64_t)r * d) + vec + 32 * y) : make_uint4(0, 0, 0, 0);
                        }
                    }
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        float x[VPL][VB], most = 0.0f;
#pragma unroll
                        for (int y = 0; y < VPL; ++y)
#pragma unroll
                            for (int z = 0; z < VB; ++z) {
                                x[y][z] = to_f(reinterpret_cast<const T*>(&v[n][y])[z]);
                                most = fmaxf(most, fabsf(x[y][z]));
                            }
#pragma unroll
                        for (int o = (LPR < 32 ? LPR : 32) / 2; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
                        const float theirs = __shfl_sync(0xffffffffu, most, (lane % RPI) * (LPR < 32 ? LPR : 32));
                        if (lane / RPI == n0 + n) amax = theirs;
                        const float f = __uint_as_float((uint32_t)(127 + 14 - pow2_of(most)) << 23);
                        const int at = w0 + RPI * (n0 + n) + sub;
#pragma unroll
                        for (int y = 0; y < VPL; ++y) {
                            uint32_t hi[VB / 2], lo[VB / 2];
#pragma unroll
                            for (int z = 0; z < VB / 2; ++z) {
                                const float u = x[y][2 * z] * f, w = x[y][2 * z + 1] * f;
                                hi[z] = pack_f16(u, w);
                                const float2 h = unpack_f16(hi[z]);
                                lo[z] = pack_f16(u - h.x, w - h.y);
                            }
                            const uint32_t to = line(at, (vec + 32 * y) * VB * 2);
                            asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(to), "r"(hi[0]), "r"(hi[1]) : "memory");
                            asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(to + S::Q_TILE), "r"(lo[0]), "r"(lo[1]) : "memory");
                        }
                    }
                }
            }
            const float qs = __uint_as_float((uint32_t)max(1, 127 - 14 + pow2_of(amax)) << 23) * (cfg.softmax_scale * 1.4426950408889634f);
            fence_async_smem();
            tc_fence_before();   // (the last job's O has been read)
            mbar_arrive(&hdr->qready[i]);

            // ---- weights, tile by tile
            float mx = ninf, l = 0.0f;
            bool far = false, primed = false;   // a reference of kAtFar or more; every row of the warp has one
            const int u0 = job.u0, u1 = job.u1;
            float held = ninf;    // the reference of the sums that left
            for (int u = u0, stop = u0; stop < u1;) {
                if (u != u0) {
                    // the sums so far leave tensor memory
                    if (!(ok = wait(&hdr->pvdone[i][(it - 1) & 1], (it - 1) >> 1))) break;
                    tc_fence_after();
                    fold_sums<ROWS>(tO, d, plan.fold + (int64_t)blockIdx.x * ROWS * D + i * kPfRows + m, u - u0 > S::FOLD,
                                    mx == ninf ? 1.0f : ex2(held - mx));
                    held = mx;
                }
                stop = u1 - u >= S::FOLD + S::FOLD / 2 ? u + S::FOLD : u1;
                for (; u < stop; ++u, ++it) {
                    if (!(ok = wait(&hdr->scale[it % kPfRing], it / kPfRing) && wait(&hdr->sfull[i][it & 1], it >> 1))) break;
                    tc_fence_after();
                    bool broke = false;
#pragma unroll 1
                    for (int h = 0; h < HALVES; ++h) {
                        const uint32_t tS = lanes + (uint32_t)((SB * i + it % SB) * BN + kBlock * h);
                        const PfScale& sc = hdr->sc[it % kPfRing][h];
                        const int slot0 = u * BN + kBlock * h, n = sc.live ? lim - slot0 : 0;   // slots of the page that the row sees
                        const float lv = sc.lv;
                        const bool border = !sc.live || slot0 + kBlock > lim0;    // (lim0: the same for the row tile)
                        float c = qs * sc.ks, slack = kPfSlack;
                        if (primed && !border && !far && !sc.odd) {
                            // Every row has a reference, and most pages do not exceed it: their weights are taken at once.  A
                            // sum that f16 holds says that none of them left its range; else the page is done again below.
                            // (c may be infinite here: scores that are not below zero leave the range then.)
                            float s[kBlock];
                            tm_ld32(tS, s);
                            tm_ld32(tS + 32, s + 32);
                            const float2 cc = make_float2(c, c), bb = make_float2(lv - mx, lv - mx);
                            float2 add[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                            uint32_t w[SPLIT ? 1 : 32];
                            auto weights = [&](int y) {
#pragma unroll
                                for (int x = y; x < y + 32; x += 2) {
                                    const float2 e = fma2(make_float2(s[x], s[x + 1]), cc, bb);
                                    s[x] = ex2(e.x);
                                    s[x + 1] = ex2(e.y);
                                    add[(x >> 1) & 1] = add2(add[(x >> 1) & 1], make_float2(s[x], s[x + 1]));
                                    if constexpr (!SPLIT) w[x >> 1] = pack_f16(s[x], s[x + 1]);
                                }
                            };
                            tm_wait32(s);
                            tm_wait32(s + 32);
                            weights(0);
                            weights(32);
                            const float sum = (add[0].x + add[0].y) + (add[1].x + add[1].y);
                            if (__all_sync(0xffffffffu, sum <= 60000.0f)) {
                                l = fmaf(sum, sc.iv, l);
                                if constexpr (SPLIT) {
                                    store_weights<SPLIT>(tS, s);
                                } else {
                                    tm_st16(tS, w);
                                    tm_st16(tS + 16, w + 16);
                                }
                                tm_wait_st();
                                tc_fence_before();
                                mbar_arrive(&hdr->pready[i][h][it & 1]);
                                continue;
                            }
                            slack = 0.0f;
                        }
                        float s[kBlock];
                        tm_ld32(tS, s);
                        tm_ld32(tS + 32, s + 32);
                        tm_wait32(s);
                        tm_wait32(s + 32);
                        // an overflow of the factors' product is no score's (keys of zero score 0 whatever their scale): then one by one
                        const bool huge = fabsf(c) == __uint_as_float(0x7f800000u);
                        if (border || huge) {
                            if (huge) c = qs;
#pragma unroll 1
                            for (int both = huge; both >= 0; --both) {
                                const float a = both ? sc.ks : c;
#pragma unroll
                                for (int x = 0; x < kBlock; ++x) s[x] = x < n ? s[x] * a : ninf;
                            }
                            c = 1.0f;
                        }
                        float top = ninf;
                        if (c < 0.0f) {     // (the same for all rows: the signs of the scales)
#pragma unroll
                            for (int x = 0; x < kBlock; ++x) top = fmaxf(top, -s[x]);
                        } else {
                            float t[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                            for (int x = 4; x < kBlock - 4; x += 8) {
#pragma unroll
                                for (int y = 0; y < 4; ++y) t[y] = max3(t[y], s[x + y], s[x + 4 + y]);
                            }
#pragma unroll
                            for (int y = 0; y < 4; ++y) t[y] = fmaxf(t[y], s[kBlock - 4 + y]);
                            top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
                        }
                        top = top * fabsf(c) + lv;
                        top -= kPfTop;
                        if (__any_sync(0xffffffffu, top > mx + slack)) {
                            const float now = fmaxf(mx, top);
                            const float f = now == ninf ? 1.0f : ex2(mx - now);
                            mx = now;
                            primed = __all_sync(0xffffffffu, mx != ninf);
                            l *= f;
                            far = __any_sync(0xffffffffu, far || (now != ninf && fabsf(now) >= kAtFar));
                            if (u != u0 || h) {
                                // O holds the pages before: the last one's product has to be there
                                if (!(ok = h ? wait(&hdr->padone[i][it & 1], it >> 1)
                                             : wait(&hdr->pvdone[i][(it - 1) & 1], (it - 1) >> 1))) {
                                    broke = true;
                                    break;
                                }
                                tc_fence_after();
                                if (__any_sync(0xffffffffu, f != 1.0f)) {
#pragma unroll 1
                                    for (int c = 0; c < D; c += 16) {
                                        float o[16];
                                        tm_ld16(tO + c, o);
                                        uint32_t w[16];
#pragma unroll
                                        for (int x = 0; x < 16; ++x) w[x] = __float_as_uint(o[x] * f);
                                        tm_st16(tO + c, w);
                                    }
                                }
                            }
                        }
                        const float ref = mx == ninf ? 0.0f : mx;
                        float bias = lv - ref;
                        if (far) {   // the exponents, rounded as the maximum was and bounded
#pragma unroll
                            for (int x = 0; x < kBlock; ++x) {
                                const float e = __fsub_rn(__fadd_rn(__fmul_rn(s[x], c), lv), ref);
                                s[x] = e > kPfTop + kPfSlack ? kPfTop + kPfSlack : e;   // (NaN stays)
                            }
                            c = 1.0f;
                            bias = 0.0f;
                        }
                        float2 add[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                        const float2 cc = make_float2(c, c), bb = make_float2(bias, bias);
#pragma unroll
                        for (int x = 0; x < kBlock; x += 2) {
                            const float2 e = fma2(make_float2(s[x], s[x + 1]), cc, bb);
                            s[x] = ex2(e.x);
                            s[x + 1] = ex2(e.y);
                            add[(x >> 1) & 1] = add2(add[(x >> 1) & 1], make_float2(s[x], s[x + 1]));
                        }
                        l = fmaf((add[0].x + add[0].y) + (add[1].x + add[1].y), sc.iv, l);
                        if (sc.odd) {  // zero, negative, tiny, huge or NaN: the ratio of scale and power of two, for the
                                       // slots that the row sees (0 x inf and 0 x NaN would reach the others)
                            const float f = sc.ratio;
#pragma unroll
                            for (int x = 0; x < kBlock; ++x) s[x] = x < n ? s[x] * f : 0.0f;
                        }
                        store_weights<SPLIT>(tS, s);
                        tm_wait_st();
                        tc_fence_before();
                        mbar_arrive(&hdr->pready[i][h][it & 1]);
                    }
                    if (broke) break;
                }
                if (!ok) break;
            }
            if (!ok) break;

            // ---- outputs, or the record of a piece
            if (!wait(&hdr->pvdone[i][(it - 1) & 1], (it - 1) >> 1) || !wait(&hdr->cdone[n_job & 1], n_job >> 1)) break;
            tc_fence_after();
            const bool whole = job.u0 == 0 && job.u1 == job.units;
            if (job.pieces && tid == 0) plan.owner[blockIdx.x] = make_int4(job.chunk, job.g, job.pieces, 0);
            float* rec = plan.rec + (int64_t)(2 * blockIdx.x + (job.u0 == 0)) * ROWS * (D + 2);
            const int at_row = i * kPfRows + m;
            const int4* nan = reinterpret_cast<const int4*>(hdr->nan[n_job & 1]);
            const float inv = l == 0.0f ? 0.0f : kAtSumUnit * __fdiv_rn(1.0f, l);
            // Through the queries' place (their products have ended), a row's line by its thread, then the warp's lines
            // one after another, 16 bytes a lane; sums of a piece in 32 bits, half a row at a time where a line holds that.
            const int rounds = whole || SPLIT ? 1 : 2, cols = D / rounds;
            const bool folded = u1 - u0 >= S::FOLD + S::FOLD / 2;
            const float* left = plan.fold + (int64_t)blockIdx.x * ROWS * D + at_row;
            held = mx == ninf ? 1.0f : ex2(held - mx);    // the factor of the sums that left
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += cols) {
#pragma unroll 1
                for (int c = c0; c < c0 + cols && c < d; c += 32) {
                    float o[32];
                    __syncwarp();
                    tm_ld32(tO + c, o);
                    tm_wait32(o);
                    if (folded) {
#pragma unroll
                        for (int h = 0; h < 32; h += 16) {
                            if (c + h >= d) break;
                            float y[16];
#pragma unroll
                            for (int x = 0; x < 16; ++x) y[x] = left[(c + h + x) * ROWS];
#pragma unroll
                            for (int x = 0; x < 16; ++x) o[h + x] = fmaf(y[x], held, o[h + x]);
                        }
                    }
#pragma unroll
                    for (int x = 0; x < 32; x += 4) {
                        const int4 first = nan[(c + x) / 4];
                        if (first.x < lim) o[x] = __uint_as_float(0x7fffffffu);
                        if (first.y < lim) o[x + 1] = __uint_as_float(0x7fffffffu);
                        if (first.z < lim) o[x + 2] = __uint_as_float(0x7fffffffu);
                        if (first.w < lim) o[x + 3] = __uint_as_float(0x7fffffffu);
                    }
                    if (whole) {
#pragma unroll
                        for (int x = 0; x < 32; ++x) o[x] = l == 0.0f ? 0.0f : o[x] * inv;   // (no weight: zeros, whatever the values were)
                    }
                    if (whole && !SPLIT) {
#pragma unroll
                        for (int x = 0; x < 32; x += 8) {
                            uint32_t w[4];
#pragma unroll
                            for (int z = 0; z < 4; ++z) w[z] = pack2(o[x + 2 * z], o[x + 2 * z + 1], (const T*)nullptr);
                            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(line(m, (c + x) * 2)), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                                         "r"(w[3])
                                         : "memory");
                        }
                    } else {
#pragma unroll
                        for (int x = 0; x < 32; x += 4)
                            asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(line(m, (c - c0 + x) * 4)), "f"(o[x]), "f"(o[x + 1]),
                                         "f"(o[x + 2]), "f"(o[x + 3])
                                         : "memory");
                    }
                }
                __syncwarp();
                // (a vector holds VB outputs, or four sums)
#pragma unroll 4
                for (int n = 0; n < NI; ++n) {
                    const int from = RPI * n + sub, r = __shfl_sync(0xffffffffu, row, from);
#pragma unroll
                    for (int y = 0; y < VPL; ++y) {
                        const int at = vec + 32 * y;
                        const uint4 x = lds128(line(w0 + from, 16 * at));
                        if (r < 0) continue;
                        if (whole) {
                            if (at * VB < d) *(reinterpret_cast<uint4*>(reinterpret_cast<T*>(a.out) + (int64_t)r * d) + at) = x;
                        } else if (c0 + at * 4 < d) {
                            *reinterpret_cast<uint4*>(rec + (i * kPfRows + w0 + from) * D + c0 + at * 4) = x;
                        }
                    }
                }
                __syncwarp();
            }
            if (mine) {
                if (!whole) {
                    float* ml = rec + (int64_t)ROWS * D + 2 * at_row;
                    ml[0] = mx;
                    ml[1] = l;
                } else if (a.lse) {
                    a.lse[row] = row_lse(mx, l);
                }
            }
            job_read(n_job);
            mbar_arrive(&hdr->epi[n_job & 1]);
            ++n_job;
        }
        if (!ok) fail_wait();
    } else if (wid < kPfPlanner) {
        // ===================================================================== converters
        constexpr int CH = D / 16, RPI = 32 / CH, NG = BN / RPI;     // chunks of a row; rows of an instruction; groups of them
        constexpr int CW = S::CW, N = (NG + CW - 1) / CW;            // a warp takes groups cw, cw + CW, ...
        const int ct = tid - NQ * 128, cw = ct >> 5, x = lane % CH, sub = lane / CH;
        const int slot_bytes = kvh * d;
        const bool in_row = 16 * x < d;
        // where this lane's chunk goes: its region, and its two places in a row's line under the swizzle
        const int odd = (x >> 2) & 1, c2 = 2 * (x & 3);
        const uint32_t to = (uint32_t)(x >> 2) * (BN * 128) + (uint32_t)sub * 128;
        const uint32_t at0 = (uint32_t)(((c2 + odd) ^ sub) << 4), at1 = (uint32_t)(((c2 + 1 - odd) ^ sub) << 4);
        uint32_t it = 0, n_job = 0;
        bool ok = true;
        while (job_there(n_job)) {
            const PfJob& job = hdr->job[n_job % kPfJobs];
            int* nan = hdr->nan[n_job & 1];   // (the planner cleared it)
            const int u1 = job.u1, len = job.len, g = job.g;
            const int shortest = job.before + job.row0 / G + 1;   // slots that every row sees
            const int32_t* table = a.block_table + (int64_t)job.req * a.bt_stride;
            const int64_t lane_src = (int64_t)g * d + (in_row ? 16 * x : 0) + sub * slot_bytes;
            auto page_of = [&](int u, int h) -> int {
                const int block = u * HALVES + h;
                return u < u1 && block * kBlock < len ? table[block] : -2;   // -2: behind the context
            };
            auto checked = [&](int p) -> int {
                if (p >= 0 && p < a.n_pages) return p;
                if (p != -2 && ct == 0) set_status(a.status, SPIN_STATUS_BAD_PAGE);
                return -1;
            };
            auto load = [&](uint4 (&v)[N], const uint8_t* pool, const int (&pg)[HALVES], int u) {
                const uint8_t* src[HALVES];
                int rows[HALVES];    // of the page that are there, for this lane
#pragma unroll
                for (int h = 0; h < HALVES; ++h) {
                    src[h] = pool + (int64_t)max(pg[h], 0) * (kBlock * slot_bytes) + lane_src;
                    rows[h] = pg[h] >= 0 && in_row ? min(kBlock, len - u * BN - kBlock * h) - sub : 0;
                }
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const int r = RPI * (cw + CW * n), in = r & (kBlock - 1);
                    const bool up = HALVES == 2 && r >= kBlock;
                    const bool live = (NG % CW == 0 || r < BN) && in < (up ? rows[HALVES - 1] : rows[0]);
                    v[n] = load_codes((up ? src[HALVES - 1] : src[0]) + in * slot_bytes, live);
                }
            };
            auto store = [&](const uint4 (&v)[N], uint32_t tile) {
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const int r = RPI * (cw + CW * n);
                    if (NG % CW && r >= BN) break;
                    const uint32_t line = tile + to + (uint32_t)r * 128, sw = (uint32_t)(r & 7) << 4;
                    store_codes(line + (at0 ^ sw), line + (at1 ^ sw), odd, v[n]);
                }
            };
            int next[HALVES], pg[HALVES];
#pragma unroll
            for (int h = 0; h < HALVES; ++h) {
                pg[h] = checked(page_of(job.u0, h));
                next[h] = page_of(job.u0 + 1, h);
            }
            uint4 kv[N], vv[N];
            float ks = 0.0f, vs = 0.0f;
            int mine = -1;
            auto load_scales = [&]() {
                if (ct < HALVES) {
                    mine = HALVES == 2 && ct ? pg[HALVES - 1] : pg[0];
                    ks = mine >= 0 ? a.k_scale[(int64_t)mine * kvh + g] : 0.0f;
                    vs = mine >= 0 ? a.v_scale[(int64_t)mine * kvh + g] : 1.0f;
                }
            };
            load(kv, a.k_pool, pg, job.u0);
            load_scales();
            for (int u = job.u0; u < u1; ++u, ++it) {
                const uint32_t st = it % NST, ph = it / NST;
                const uint32_t sK = sKV + st * 2 * S::KV, sV = sK + S::KV;
                load(vv, a.v_pool, pg, u);
                // the stage, and with it the ring's entry (see kempty's commit), is free
                if (!(ok = wait(&hdr->kempty[st], ph ^ 1u))) break;
                if (ct < HALVES) {
                    PfScale& e = hdr->sc[it % kPfRing][ct];
                    const bool strange = !in_log_range(vs);
                    const float lv = scale_log2(vs);
                    e.ks = ks;
                    e.lv = lv;
                    e.iv = kAtSumUnit * (strange ? ex2(-lv) : __frcp_rn(vs));
                    e.ratio = strange ? vs * ex2(-lv) : 1.0f;
                    e.live = mine >= 0;
                    e.odd = strange;
                    if (ct == 0) *(volatile uint32_t*)&hdr->tiles = it + 1;
                    mbar_arrive(&hdr->scale[it % kPfRing]);
                }
                __syncwarp();
                store(kv, sK);
                fence_async_smem();
                mbar_arrive(&hdr->kfull[st]);
                if (u + 1 < u1) {
#pragma unroll
                    for (int h = 0; h < HALVES; ++h) {
                        pg[h] = checked(next[h]);
                        next[h] = page_of(u + 2, h);
                    }
                    load(kv, a.k_pool, pg, u + 1);
                    load_scales();
                }
                if ((u + 1) * BN > shortest) {
                    // NaN codes that some rows see and others do not would reach the others as 0 x NaN: they leave the
                    // tile, and the first one's slot of each dimension is kept
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        uint32_t w[4] = {vv[n].x, vv[n].y, vv[n].z, vv[n].w}, any = 0;
#pragma unroll
                        for (int y = 0; y < 4; ++y) any |= (w[y] & 0x7f7f7f7fu) + 0x01010101u;
                        if (any & 0x80808080u) {
                            const int slot = u * BN + RPI * (cw + CW * n) + sub;
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                const uint32_t b = ((w[y] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;   // bytes that are NaN
                                w[y] &= ~((b >> 7) * 0xffu);
#pragma unroll 1
                                for (uint32_t z = b; z; z &= z - 1) atomicMin(nan + 16 * x + 4 * y + ((__ffs(z) - 1) >> 3), slot);
                            }
                            vv[n] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                    __syncwarp();
                }
                if (!(ok = wait(&hdr->vempty[st], ph ^ 1u))) break;
                store(vv, sV);
                fence_async_smem();
                mbar_arrive(&hdr->vfull[st]);
            }
            if (!ok) break;
            job_read(n_job);
            mbar_arrive(&hdr->cdone[n_job & 1]);
            ++n_job;
        }
    } else if (wid == kPfPlanner) {
        // ======================================================================== planner
        PfWalk walk;
        walk.start(plan, hdr->chunk, hdr->into, kvh, total);
        for (uint32_t n = 0;; ++n) {
            PfJob& job = hdr->job[n % kPfJobs];
            if (!wait(&hdr->jdone[n % kPfJobs], (n / kPfJobs) ^ 1u)) break;
            // the outputs of the job before last are out: its list of NaN begins anew for this one.  All of a job may pass
            // meanwhile (2^24 slots of 256 fp32 dimensions: 0.73 s at full clocks, near a wait's limit of 1 s), so that this
            // wait's limit begins anew while tiles go on.
            if (n >= 2 && !__all_sync(0xffffffffu, mbar_wait_while(&hdr->epi[n & 1], ((n >> 1) - 1) & 1u, &hdr->abort_flag, &hdr->tiles))) {
                fail_wait();
                break;
            }
            for (int e = lane; e < D; e += 32) hdr->nan[n & 1][e] = 0x7fffffff;
            __syncwarp();
            if (lane == 0) {
                walk.next<BN>(plan, kvh, job);
                mbar_arrive(&hdr->jready[n % kPfJobs]);
            }
            __syncwarp();
            if (!job.more) break;
        }
    } else {
        // ========================================================================= issuer
        {
            constexpr uint32_t REGION = kPfRows * 128;    // a row tile's 64 columns of queries
            const uint32_t idesc_s = idesc_mma(0u, BN, 128);
            const uint32_t idesc_o = idesc_mma(0u, (uint32_t)d, 128) | (1u << 16);   // B is N-major
            const int ksteps = d / 16;
            uint32_t it = 0, n_job = 0;
            bool ok = true, issued = false;
            auto scores = [&](int i, uint32_t t) {    // S of row tile i for the tile of iteration t
                const uint64_t b0 = smem_desc_sw128(sKV + (t % NST) * 2 * S::KV);
#pragma unroll
                for (int z = 0; z < (SPLIT ? 2 : 1); ++z) {
                    const uint64_t a0 = smem_desc_sw128(sQ + (uint32_t)(i * (SPLIT ? 2 : 1) + z) * S::Q_TILE);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        if (k < ksteps) tc_mma_f16(tmem + (uint32_t)((SB * i + t % SB) * BN), a0 + (uint64_t)((k >> 2) * (REGION >> 4) + 2 * (k & 3)),
                                   b0 + (uint64_t)((k >> 2) * (BN * 128 >> 4) + 2 * (k & 3)), idesc_s, (z | k) ? 1u : 0u);
                }
                tc_commit(&hdr->sfull[i][t & 1]);
            };
            auto weighted = [&](int i, uint32_t t, int h, bool first) {   // O of row tile i gains a page's values
                const uint64_t b0 = smem_desc_sw128_mn(sKV + (t % NST) * 2 * S::KV + S::KV, BN * 128) + (uint64_t)(h * (8192 >> 4));
                const uint32_t o = tmem + (uint32_t)(NQ * SB * BN + i * D), p0 = tmem + (uint32_t)((SB * i + t % SB) * BN + kBlock * h);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint64_t b = b0 + (uint64_t)(k * (2048 >> 4));
                    const uint32_t acc = !first || k ? 1u : 0u;
                    if constexpr (SPLIT) {
                        const uint32_t p = p0 + 32 * (k >> 1) + 8 * (k & 1);
                        tc_mma_f16_ta(o, p, b, idesc_o, acc);
                        tc_mma_f16_ta(o, p + 16, b, idesc_o, 1u);
                    } else {
                        tc_mma_f16_ta(o, p0 + 8 * k, b, idesc_o, acc);
                    }
                }
            };
            while (ok && job_there(n_job)) {
                const PfJob& job = hdr->job[n_job % kPfJobs];
                const int u0 = job.u0, u1 = job.u1;
                job_read(n_job);
                // the first scores: the buffers of the job before are free when its rows have let the next queries in
                for (int t = 0; t < SB && ok && u0 + t < u1; ++t) {
                    const uint32_t x = it + t;
                    if (!(ok = wait(&hdr->kfull[x % NST], x / NST))) break;
#pragma unroll 1
                    for (int i = 0; i < NQ && ok; ++i) {
                        if (t == 0 && !(ok = wait(&hdr->qready[i], n_job))) break;
                        tc_fence_after();
                        if (elect_one()) scores(i, x);
                        issued = true;
                        __syncwarp();
                    }
                    if (!ok) break;
                    if (elect_one()) tc_commit(&hdr->kempty[x % NST]);
                    __syncwarp();
                }
                // row tile by row tile: its weights' products, then its next scores, so that the row tiles are half a
                // turn apart and one's products run while the other's weights are computed
                for (int u = u0; ok && u < u1; ++u, ++it) {
                    const uint32_t st = it % NST, nx = it + SB;
#pragma unroll
                    for (int i = 0; i < NQ; ++i) {
                        if (!ok) break;
                        for (int h = 0; h < HALVES; ++h) {
                            if (!(ok = wait(&hdr->pready[i][h][it & 1], it >> 1) && (i || h || wait(&hdr->vfull[st], it / NST)))) break;
                            tc_fence_after();
                            if (elect_one()) {
                                weighted(i, it, h, u == u0 && h == 0);
                                tc_commit(h == HALVES - 1 ? &hdr->pvdone[i][it & 1] : &hdr->padone[i][it & 1]);
                                if (i == NQ - 1 && h == HALVES - 1) tc_commit(&hdr->vempty[st]);
                            }
                            __syncwarp();
                        }
                        if (ok && u + SB < u1) {
                            // the weights lie in the scores' columns: the next scores there wait for the product that
                            // reads them
                            if (!(ok = (i || wait(&hdr->kfull[nx % NST], nx / NST)) && wait(&hdr->pvdone[i][it & 1], it >> 1))) break;
                            tc_fence_after();
                            if (elect_one()) {
                                scores(i, nx);
                                if (i == NQ - 1) tc_commit(&hdr->kempty[nx % NST]);
                            }
                            __syncwarp();
                        }
                    }
                }
                ++n_job;
            }
            if (issued) {   // every product has ended before tensor memory is released
                if (elect_one()) tc_commit(&hdr->fin);
                __syncwarp();
                if (!mbar_wait(&hdr->fin, 0u, nullptr)) set_status(a.status, SPIN_STATUS_TIMEOUT);
            }
        }
    }
    pdl_trigger();
    tc_fence_before();
    __syncthreads();
    if (wid == kPfIssuer) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::COLS) : "memory");
    }
}

// Joins the pieces of divided jobs, four rows a warp.  The first piece lies in the second record of the CTA that begins
// the job, the others in the first records of the CTAs after it.
constexpr int kPfJoinWarps = 8, kPfJoinRows = 4;
template <typename T, int D, int NQ>
__global__ void __launch_bounds__(32 * kPfJoinWarps) prefill_join_kernel(spin_kv_config cfg, KvChunkArgs a, PfPlan plan) {
    pdl_begin();
    constexpr int ROWS = NQ * kPfRows, F = D / 32, N = kPfJoinRows;
    const int4 o = plan.owner[blockIdx.x];
    if (o.z == 0) return;
    const int lane = threadIdx.x & 31, m0 = (blockIdx.y * kPfJoinWarps + (threadIdx.x >> 5)) * N;
    const int H = cfg.n_heads, G = H / cfg.kv_heads, d = cfg.head_dim;
    const int4 c = plan.chunk[o.x];
    const int2 t = plan.tokens[o.x];
    constexpr int REC = ROWS * (D + 2);
    const float* rec = plan.rec + (int64_t)2 * blockIdx.x * REC;
    auto at = [&](int p) { return rec + (p ? (int64_t)2 * p * REC : (int64_t)REC); };
    const float ninf = __uint_as_float(0xff800000u);
    float top[N];
#pragma unroll
    for (int n = 0; n < N; ++n) top[n] = ninf;
    for (int p = lane; p < o.z; p += 32)
#pragma unroll
        for (int n = 0; n < N; ++n) top[n] = fmaxf(top[n], at(p)[ROWS * D + 2 * (m0 + n)]);
    float acc[N][F], l[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
#pragma unroll
        for (int i = 16; i; i >>= 1) top[n] = fmaxf(top[n], __shfl_xor_sync(0xffffffffu, top[n], i));
        l[n] = 0.0f;
#pragma unroll
        for (int i = 0; i < F; ++i) acc[n][i] = 0.0f;
    }
    for (int p = 0; p < o.z; ++p) {
        const float* x = at(p);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const float2 ml = *reinterpret_cast<const float2*>(x + ROWS * D + 2 * (m0 + n));
            // (a piece without a slot of this row has l = 0, and sums that may be 0 x NaN; one that saw only NaN
            // scores has l = NaN, which stays)
            const float f = ml.x == ninf ? 0.0f : ex2(ml.x - top[n]);
            l[n] = fmaf(f, ml.y, l[n]);
#pragma unroll
            for (int i = 0; i < F; ++i) {
                const float y = x[(m0 + n) * D + i * 32 + lane];
                if (ml.x != ninf) acc[n][i] = fmaf(f, y, acc[n][i]);
            }
        }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const uint32_t R = (uint32_t)c.y + m0 + n, token = R / (uint32_t)G;
        if (token >= (uint32_t)t.y) return;
        const int64_t row = ((int64_t)t.x + token) * H + (int64_t)o.y * G + (R - token * G);
        const float inv = l[n] == 0.0f ? 0.0f : kAtSumUnit * __fdiv_rn(1.0f, l[n]);
#pragma unroll
        for (int i = 0; i < F; ++i)
            if (i * 32 + lane < d)
                from_f(reinterpret_cast<T*>(a.out)[row * d + i * 32 + lane], l[n] == 0.0f ? 0.0f : acc[n][i] * inv);
        if (a.lse && lane == 0) a.lse[row] = row_lse(top[n], l[n]);
    }
}

// ------------------------------------------------------------------------------ host side
static size_t pf_round(size_t n) { return (n + 255) & ~(size_t)255; }
static int pf_sms() {
    const int n = device_sm_count();
    return n < kPfMostSms ? n : kPfMostSms;
}
static int64_t pf_chunks(const spin_kv_config& cfg, int64_t n_tokens) {
    const int64_t G = cfg.n_heads / cfg.kv_heads;
    return n_tokens * G / kPfRows + cfg.n_req;
}

static size_t pf_layout(const spin_kv_config& cfg, int64_t n_tokens, void* ws, PfPlan* p) {
    const int64_t n = pf_chunks(cfg, n_tokens);
    const size_t sms = (size_t)pf_sms();
    char* c = reinterpret_cast<char*>(ws);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char* x = c + at;
        at += pf_round(bytes);
        return x;
    };
    PfPlan q;
    q.head = reinterpret_cast<int64_t*>(take(16));
    q.begin = reinterpret_cast<int64_t*>(take((size_t)(n + 1) * 8));
    q.chunk = reinterpret_cast<int4*>(take((size_t)n * sizeof(int4)));
    q.tokens = reinterpret_cast<int2*>(take((size_t)n * sizeof(int2)));
    q.owner = reinterpret_cast<int4*>(take(sms * sizeof(int4)));
    q.base = reinterpret_cast<int*>(take(((size_t)cfg.n_req + 1) * 4));
    q.rec = reinterpret_cast<float*>(take(sms * 2 * 2 * kPfRows * ((size_t)pf_dim(cfg.head_dim) + 2) * sizeof(float)));
    const bool folds = cfg.max_slots > pf_fold(cfg.dtype == SPIN_DTYPE_F32);
    q.fold = reinterpret_cast<float*>(take(folds ? sms * 2 * kPfRows * (size_t)pf_dim(cfg.head_dim) * sizeof(float) : 0));
    q.most = (int)n;
    q.ranks = (int)sms;
    if (p) *p = q;
    return at;
}

size_t kv_prefill_workspace_bytes(const spin_kv_config& cfg, int64_t n_tokens, int) {
    return pf_layout(cfg, n_tokens, nullptr, nullptr);
}

template <typename T, int D, int NQ>
static cudaError_t launch_tiles(const spin_kv_config& cfg, const KvChunkArgs& a, cudaStream_t s) {
    using S = PfShape<T, D, NQ>;
    static std::atomic<uint64_t> allowed;
    auto k = prefill_kernel<T, D, NQ>;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), S::BYTES, allowed);
    if (e != cudaSuccess) return e;
    PfPlan p;
    pf_layout(cfg, a.n_tokens, a.workspace, &p);
    e = launch_pdl(prefill_plan_kernel<NQ * kPfRows, S::BN>, dim3(1), dim3(1024), 0, s, nullptr, 0, cfg, a, p);
    if (e != cudaSuccess || a.max_new == 0) return e;
    e = launch_pdl(k, dim3(p.ranks), dim3(kPfThreads), S::BYTES, s, nullptr, 0, cfg, a, p);
    if (e != cudaSuccess) return e;
    return launch_pdl(prefill_join_kernel<T, D, NQ>, dim3(p.ranks, NQ * kPfRows / (kPfJoinWarps * kPfJoinRows)), dim3(32 * kPfJoinWarps), 0, s,
                      nullptr, 0, cfg, a, p);
}

// Two row tiles a CTA, unless one holds all rows that a request has for a key head (16 requests of 128 rows behind up to
// 32000 slots, 64 heads on 8: 240 us, 312 with two); wide heads and fp32 (two terms of
// queries and weights) leave room for one.
template <typename T, int D>
static cudaError_t launch_rows(const spin_kv_config& cfg, const KvChunkArgs& a, cudaStream_t s) {
    if constexpr (D <= 128 && !std::is_same<T, float>::value)
        if ((int64_t)a.max_new * (cfg.n_heads / cfg.kv_heads) > kPfRows) return launch_tiles<T, D, 2>(cfg, a, s);
    return launch_tiles<T, D, 1>(cfg, a, s);
}

template <typename T>
static cudaError_t launch_typed(const spin_kv_config& cfg, const KvChunkArgs& a, cudaStream_t s) {
    switch (pf_dim(cfg.head_dim)) {
        case 64: return launch_rows<T, 64>(cfg, a, s);
        case 128: return launch_rows<T, 128>(cfg, a, s);
        default: return launch_rows<T, 256>(cfg, a, s);
    }
}

cudaError_t launch_kv_prefill(const spin_kv_config& cfg, const KvChunkArgs& a, cudaStream_t s) {
    switch (cfg.dtype) {
        case SPIN_DTYPE_F32: return launch_typed<float>(cfg, a, s);
        case SPIN_DTYPE_BF16: return launch_typed<__nv_bfloat16>(cfg, a, s);
        default: return launch_typed<__half>(cfg, a, s);
    }
}

}  // namespace spin
