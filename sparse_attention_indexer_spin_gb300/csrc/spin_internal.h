// spin_internal.h -- host-side launchers of the SPIN kernels (called by spin_api.cu only).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/spin.h"
#include "spin_common.cuh"

namespace spin {

struct SelectArgs {
    const float* V;
    const float* D;
    const float* Vmax;
    const int32_t* warm;
    const int32_t* n_slots;
    const int32_t* q_pos;
    int rows;
    const int32_t* rho_override;
    uint64_t step;
    const uint64_t* step_dev;  // non-NULL: the kernels read the step here instead
    int layer;
    int32_t* blocks;
    int32_t* n_blocks;
    int32_t* union_blocks;
    int32_t* n_union;
    float* block_scores;  // workspace: S [R][rows][MB] fp32, then exploration draws [R][rows][MB] u32
    uint32_t* status;
    int n_layers;         // layers stacked along the outermost dimension of every array (0 or 1: one)
    const uint32_t* block_age = nullptr;  // block-age exploration: ages [R][MB] replace the draws
};

struct ScoreArgs {
    const void* q;
    const float* w;
    const void* k_pool;
    const float* k_scale;
    int64_t n_pages;
    const int32_t* block_table;
    int64_t bt_stride;
    const int32_t* list;
    const int32_t* n_list;
    const int32_t* n_slots;
    int rows;
    float* scores;
    uint32_t* status;
    HintArgs hint;  // rec == NULL: no candidate collection for the hinted top-K
};

struct EmaArgs {
    float* V;
    float* D;
    float* Vmax;
    int32_t* warm;
    const float* scores;
    int rows;
    const int32_t* list;
    const int32_t* n_list;
    const int32_t* n_slots;
    const int32_t* q_pos;
    const int32_t* accepted;  // NULL: a = 0
    uint32_t* status;
    int n_layers;             // layers stacked along the outermost dimension (0 or 1: one)
    uint32_t* block_age = nullptr;  // block-age exploration: listed blocks get age_step + 1
    uint64_t age_step = 0;
};

size_t select_workspace_bytes(const spin_config& cfg, int rows);

cudaError_t launch_init_state(const spin_config& cfg, float* V, float* D, float* Vmax,
                              int32_t* warm, int req, cudaStream_t s);
cudaError_t launch_select(const spin_config& cfg, const SelectArgs& a, cudaStream_t s);
cudaError_t launch_score_generic(const spin_config& cfg, const ScoreArgs& a, cudaStream_t s);
// Returns cudaErrorNotSupported when the shape has no streaming kernel instance.
cudaError_t launch_score_stream(const spin_config& cfg, const ScoreArgs& a, cudaStream_t s);
bool score_stream_supported(const spin_config& cfg, int rows);
cudaError_t launch_score_tc(const spin_config& cfg, const ScoreArgs& a, cudaStream_t s);
bool score_tc_supported(const spin_config& cfg, int rows);
bool topk_sample_fits(const spin_config& cfg);
cudaError_t launch_topk_sample(const spin_config& cfg, const float* scores, const int32_t* list,
                               const int32_t* n_list, const int32_t* n_slots, int rows, int32_t* topk_idx,
                               uint32_t* status, cudaStream_t s);
cudaError_t launch_topk(const spin_config& cfg, const float* scores, const int32_t* list,
                        const int32_t* n_list, const int32_t* n_slots, int rows,
                        int32_t* topk_idx, uint32_t* status, cudaStream_t s);
cudaError_t launch_ema(const spin_config& cfg, const EmaArgs& a, cudaStream_t s);

// Temporal top-K (spin_topk_hint.cu).
bool topk_hint_supported(const spin_config& cfg);
int topk_hint_cap(const spin_config& cfg);
size_t topk_hint_bytes(const spin_config& cfg, int rows);
HintArgs topk_hint_args(const spin_config& cfg, int rows, void* hint);
cudaError_t launch_topk_hint(const spin_config& cfg, const float* scores, const float* w, const int32_t* list,
                             const int32_t* n_list, const int32_t* n_slots, int rows, int32_t* topk_idx,
                             const HintArgs& h, uint32_t* status, cudaStream_t s);

int device_sm_count();

// KV cache (spin_kv_append.cu, spin_kv_attend.cu) and its pages (spin_pages.cu).
struct KvAppendArgs {
    const void* x[2];       // new keys, new values [n_tokens][kv_heads][head_dim]
    uint8_t* pool[2];
    float* scale[2];
    int64_t n_tokens;
    const int32_t* new_start;
    int max_new;
    const int32_t* n_before;
    int64_t n_pages;
    const int32_t* block_table;
    int64_t bt_stride;
    uint32_t* status;
};

struct KvAttendArgs {
    const void* q;
    const uint8_t* k_pool;
    const uint8_t* v_pool;
    const float* k_scale;
    const float* v_scale;
    int64_t n_pages;
    const int32_t* block_table;
    int64_t bt_stride;
    const int32_t* n_slots;
    int rows;
    const int32_t* list;    // NULL: every slot
    int top_k;
    void* out;
    float* lse;             // may be NULL
    float* workspace;
    uint32_t* status;
};

// Rotary positions (spin_rope.cu).
constexpr int kRopeMaxRows = 4;
struct RopeArgs {
    spin_rope_rows rows[kRopeMaxRows];
    int n_rows;
    int64_t n_tokens;
    const int32_t* positions;
    const uint64_t* turns;
};
cudaError_t launch_rope(const spin_rope_config& cfg, const RopeArgs& a, cudaStream_t s);

// A ragged chunk of new tokens on the cache (spin_kv_prefill.cu, spin_kv_weigh.cu).
struct KvChunkArgs {
    const void* q;
    int64_t n_tokens;
    const int32_t* new_start;
    int max_new;
    const int32_t* n_before;
    const uint8_t* k_pool;
    const uint8_t* v_pool;   // prefill
    const float* k_scale;
    const float* v_scale;    // prefill
    int64_t n_pages;
    const int32_t* block_table;
    int64_t bt_stride;
    void* out;               // prefill
    float* lse;              // prefill: written, may be NULL; weigh: read
    float decay;             // weigh
    float* weight;           // weigh
    void* workspace;
    uint32_t* status;
};
size_t kv_prefill_workspace_bytes(const spin_kv_config& cfg, int64_t n_tokens, int max_new);
cudaError_t launch_kv_prefill(const spin_kv_config& cfg, const KvChunkArgs& a, cudaStream_t s);
size_t kv_weigh_workspace_bytes(const spin_kv_config& cfg, int64_t n_tokens, int max_new);
size_t kv_weigh_tc_workspace_bytes(const spin_kv_config& cfg, int64_t n_tokens);
cudaError_t launch_kv_weigh_tc(const spin_kv_config& cfg, const KvChunkArgs& a, cudaStream_t s);
cudaError_t launch_kv_weigh(const spin_kv_config& cfg, const KvChunkArgs& a, cudaStream_t s);

constexpr int kMaxPools = 16;

struct PageTable {
    int32_t n_req;
    int64_t n_pages;
    int32_t* table;
    int64_t stride;
    int32_t* ref;
    uint32_t* status;
};

struct PagePoolSet {
    spin_page_pool pool[kMaxPools];
    int n;
};

cudaError_t launch_kv_append(const spin_kv_config& cfg, const KvAppendArgs& a, cudaStream_t s);
size_t kv_attend_workspace_bytes(const spin_kv_config& cfg, int rows, int top_k);
cudaError_t launch_kv_attend(const spin_kv_config& cfg, const KvAttendArgs& a, cudaStream_t s);

size_t pages_workspace_bytes(int32_t n_req, int64_t n_pages);
cudaError_t launch_pages_fork(const PageTable& t, const int32_t* table_in, const int32_t* parent, cudaStream_t s);
cudaError_t launch_pages_free(const PageTable& t, const int32_t* keep, cudaStream_t s);
cudaError_t launch_pages_reserve(const PageTable& t, const int32_t* n_slots, const int32_t* n_new,
                                 const PagePoolSet& pools, int32_t* granted, void* ws, cudaStream_t s);
cudaError_t launch_pages_copy(const PageTable& t, const PagePoolSet& pools, void* ws, cudaStream_t s);
cudaError_t launch_pages_compact(const PageTable& t, const PagePoolSet& pools, int32_t* n_live, void* ws,
                                 cudaStream_t s);

struct PageEvictArgs {
    int32_t* n_slots;
    const float* weight;
    float* weight_out;
    const int32_t* keep;
    int n_first, n_last;
    int32_t* kept;
    void* workspace;
};
size_t pages_evict_workspace_bytes(int32_t n_req, int64_t bt_stride);
cudaError_t launch_pages_evict(const PageTable& t, const PageEvictArgs& a, cudaStream_t s);

// Self-test of the bounded mbarrier wait (spin_selftest.cu).
cudaError_t launch_wait_selftest(int mode, uint64_t limit_ns, uint32_t* status, unsigned long long* elapsed_ns,
                                 cudaStream_t s);
cudaError_t launch_wait_moving_selftest(int steps, int arrives, uint64_t limit_ns, uint32_t* status,
                                        unsigned long long* elapsed_ns, cudaStream_t s);

// Per-layer block budgets (host functions; spin_budget.cu).  Arguments are validated by the
// C-ABI wrappers.
int64_t budget_blocks_host(int64_t nb, int64_t top_k, int32_t rho_bp);
void mean_miss_curve_host(const float* S, int32_t n_req, int64_t s_stride, const int32_t* nb,
                          const int32_t* topk, int32_t top_k, int32_t n_points, float* miss);
void allocate_budgets_host(const float* miss, int32_t n_layers, int32_t n_points, int32_t target_g,
                           int32_t g_min, int32_t* g_out);

}  // namespace spin
