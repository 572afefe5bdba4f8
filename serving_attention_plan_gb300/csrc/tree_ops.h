// Attention over parts of a cache that is chosen on the GPU: trees of drafted tokens, and pages that a score
// selects.  Parameter blocks and launchers (each returns an fi_status).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "cache_ops.h"

namespace fi {

// Runs `f` once for each device that is current when it is asked for: function attributes belong to a device.
class PerDevice {
 public:
  template <typename F>
  cudaError_t run(F&& f) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (done_.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = f();
    if (e == cudaSuccess) done_.fetch_or(bit, std::memory_order_release);
    return e;
  }

 private:
  std::atomic<uint64_t> done_{0};
};

// ---- trees ---------------------------------------------------------------------------------------------
constexpr int kTreeRows = 128;      // query rows (tokens x heads of a group) of a tile
constexpr int kTreeKeys = 128;
constexpr int kTreeLeastTiles = 2;  // tiles of a CTA's piece of the line, as long as there are enough

// Tiles of the requests before each one (Geo::tree0) and of all; false if there are more than 2^31 - 1.
// starts: the request in which the line of each of `ctas` CTAs begins.
bool fill_tree(Geo* geo, int batch, int hkv, int group, int ctas, int32_t* total, int32_t* starts);

struct TreeParams {
  PageView pv;
  const __nv_bfloat16* q;
  const void *k_pages, *v_pages;
  const int32_t* starts;  // of each CTA, the request in which its part of the line begins
  const uint32_t* mask;   // [total_q][mask_words]
  int mask_words;
  __nv_bfloat16* o;
  float* lse;
  float* part_o;    // [2 CTAs][2 row tiles][128 rows][128], normalised
  float* part_lse;  // log2 domain
  int hqo, group, tile_tokens;  // tile_tokens: 128 / group
  uint32_t q_tile_bytes;
  float scale_log2;  // includes k_scale
  float v_scale;
  float cap_log2, inv_cap_log2;  // soft-cap, 0 for none
  int wide_cap;                  // the soft-cap is above kExpTanhMostCap
};
int launch_tree(const TreeParams& p, int total_q, bool fp8, int num_sms, cudaStream_t stream);

struct CommitParams {
  PageView pv;
  const int32_t* path;  // [batch][path_len]
  int path_len;
  void *k_pages, *v_pages;
};
int launch_commit(const CommitParams& p, int most_batch, bool fp8, int num_sms, cudaStream_t stream);

// ---- chosen pages --------------------------------------------------------------------------------------
struct BoundsParams {
  PageView pv;
  const void* k_pages;
  __nv_bfloat16* bounds;  // [num_pages][hkv][2][128]
  int new_keys;           // 1: only the pages that hold a request's last l_q keys
};
int launch_bounds(const BoundsParams& p, int64_t tasks, bool fp8, int num_sms, cudaStream_t stream);

struct ScoreParams {
  PageView pv;
  const __nv_bfloat16* q;
  const __nv_bfloat16* bounds;
  float* scores;  // [total_q][hkv][row_pages]
  int row_pages;
  int most_batch;  // of the workspace
  int most_lq;     // query tokens of a request of the plan at hand
  int parts;       // set by the launcher: a power of two, parts of a block's sets that warps can have apart
  int hqo, group;
  float scale;     // includes k_scale
};
int launch_scores(ScoreParams p, int64_t tasks, int num_sms, cudaStream_t stream);

struct PickParams {
  PageView pv;
  const float* scores;  // [total_q][hkv][row_pages]
  int32_t* selected;    // [total_q][hkv][budget]
  int row_pages, sink, recent, budget;
};
int launch_pick(const PickParams& p, int64_t rows, int most_pages, int num_sms, cudaStream_t stream);

// The work of an attention launch over selected pages, made on the GPU in the form in which the host planner hands work to
// those kernels: cta_indptr, items, split units and the slots' units, for `ctas` persistent CTAs.
struct ListPlanParams {
  PageView pv;
  const int32_t* selected;  // [total_q][hkv][budget]
  int budget;
  int ctas;
  int block_pages;  // pages of a step of the line that the CTAs share out
  int least;        // steps of a CTA's piece, as long as there are enough
  int32_t *header, *cta_indptr, *items, *units, *slot_unit;
};
int launch_list_plan(const ListPlanParams& p, int64_t units, int num_sms, cudaStream_t stream);

}  // namespace fi
