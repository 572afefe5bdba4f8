// Cache operators that run on a workspace's plan: append of new tokens, accumulated attention
// weights, selection of the keys to keep, compaction.  Parameter blocks and launchers (each returns
// an fi_status).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace fi {

// Geometry of one request of the plan (host and device); entry [batch] holds the totals in q0, kv0,
// blk0 and tile0.
struct Geo {
  int32_t q0, lq;    // first query token, query tokens
  int32_t kv0, lkv;  // first entry in the page list, keys
  int32_t blk0;      // 32-key blocks of the requests before this one that take the row form of the weights
  int32_t tile0;     // 256-key tiles of the requests before this one (told by fi_cache_plan_compute, read by no kernel)
  int32_t work0;     // tensor-core weights: Q tiles (over all KV heads) of the requests before this one
  int32_t pad;
};
// The plan as a whole, in the place before the first entry: one load gives a kernel all of it.
struct GeoHead {
  int32_t batch, total_q;
  int32_t blocks;          // 32-key blocks of the row form
  int32_t work;            // Q tiles of the tensor-core weights, 0 if they were not counted
  int32_t causal, window;  // the window that work was counted with (-1: none)
  int32_t pad0, pad1;
};
static_assert(sizeof(Geo) == 32 && sizeof(GeoHead) == sizeof(Geo), "one sector each");
constexpr int kBlkKeys = 32;
constexpr int kTileKeys = 256;
constexpr int kWeightTileRows = 128;  // query rows of a Q tile of the tensor-core weights

// Of key tile kt: the first query token that sees one of its keys, how many tokens from there on do,
// and the Q tiles of `tile_tokens` tokens they take (at least 1: the decay has to reach every key).
__host__ __device__ inline void weight_item(int lq, int lkv, int kt, bool causal, int window, int tile_tokens, int* t0,
                                            int* tokens, int* cost) {
  int first = 0, last = lq;
  if (causal) {
    const int key0 = kt * kTileKeys, key1 = key0 + kTileKeys < lkv ? key0 + kTileKeys : lkv, off = lkv - lq;
    if (key0 - off > 0) first = key0 - off;
    if (window >= 0 && key1 - off + (long long)window < last) last = key1 - off + window;
  }
  const int n = last > first ? last - first : 0;
  *t0 = first;
  *tokens = n;
  const int c = (n + tile_tokens - 1) / tile_tokens;
  *cost = c > 1 ? c : 1;
}

struct GeoTotals {
  bool ok = false;     // the counts below fit the entries' 32-bit fields
  int64_t blocks = 0;  // 32-key blocks (of the row form, once split)
  int64_t work = 0;    // Q tiles of the tensor-core form
  int32_t max_lkv = 0;
};
// The entries [0, batch] of a validated batch (cache_plan.cpp, host only, like the two checks).
GeoTotals fill_geo(const int32_t* qo_indptr, const int32_t* kv_indptr, const int32_t* last_page_len, int batch,
                   int page_size, Geo* out);
// Splits the requests of filled entries between the two forms of the weights: those of more than row_limit query
// rows get Q tiles (work0) and no blocks (blk0), the others blocks and no tiles.
void split_weights(Geo* geo, int batch, int hkv, int group, int row_limit, bool causal, int window, GeoTotals* totals);
// Query rows (tokens x heads of a group) up to which a request takes the row form in a batch that needs the
// tensor cores.  Measured, row form against tensor cores, 128 requests of U[64, 4096] keys, 32/8 heads: bf16 16 rows
// 147 / 359 us, 32 rows 254 / 396, 64 rows 382 / 338, 128 rows 783 / 361; e4m3 32 rows 240 / 695, 64 rows
// 419 / 661, 128 rows 959 / 776; 4 requests of U[64, 16384], bf16 32 rows 36 / 47, 64 rows 33 / 25.
constexpr int kRowFormMostBf16 = 32;
constexpr int kRowFormMostE4m3 = 64;
// FI_OK if no page id (0 .. max_page) occurs twice in the two lists, else FI_ERR_UNSUPPORTED; FI_ERR_CAPACITY without host memory.
int check_pages_once(const int32_t* a, int64_t na, const int32_t* b, int64_t nb, int32_t max_page);
// FI_OK if no page takes new tokens (the last l_q keys of a request) from two places of the list, or while the
// shared list (of a composable plan; n_shared may be 0) holds it too.
int check_tails_once(const Geo* geo, const int32_t* kv_indices, int batch, int page_size, const int32_t* shared,
                     int64_t n_shared);
// Radians per position -> the fraction of a turn per position, in 2^-64 turns.
uint64_t turns_fraction(double inv_freq);

struct PageView {  // the plan and the page pool, as every cache operator sees them
  const Geo* geo;  // a GeoHead lies before the first entry
  const int32_t* kv_indices;
  int32_t* err;
  int num_pages, page_size;
  int page_shift;  // log2(page_size), or -1
  int hkv;
  // element strides of K/V pages
  long long page_stride, head_stride, tok_stride;
};

constexpr int kMaxFreqs = 64;
struct AppendParams {
  PageView pv;
  const void *q, *k, *v;
  long long q_stride, k_stride, v_stride;  // elements between tokens
  const void *q_weight, *k_weight;         // bf16 [128] or null
  const int32_t* positions;                // or null
  void* q_out;
  void *k_pages, *v_pages;
  float eps, k_inv_scale, v_inv_scale;
  int hqo;
  int rotary;       // rotated dims: a multiple of 16, 0 for none
  int interleaved;  // pairs (2j, 2j + 1) instead of (j, j + rotary / 2)
  uint64_t freq[kMaxFreqs];  // revolutions per position, as a 64-bit fraction of a turn
};
// In the launchers below, `most_*` is what the grid is made for: the plan's own number, or, of a captured launch, the
// workspace's capacity, since a later plan may fill it.
int launch_append(const AppendParams& p, int total_q, int most_q, bool fp8, int num_sms, cudaStream_t stream);

// The tanh of a soft-cap by exponentials has an absolute error of 1.5e-7, which the cap multiplies: up to this cap 1e-5 in
// a logit.  Above it the tanh is taken with a relative error (tanh_near below |y| = 1/4, by exponentials from there on, where
// 1.5e-7 is 6e-7 of the value).
constexpr float kExpTanhMostCap = 64.f;

struct WeightsParams {
  PageView pv;
  const void* q;       // bf16 [total_q, hqo, 128]
  const void* k_pages;
  const float* lse;    // [total_q, hqo]
  float* weights;      // [num_pages, hkv, page_size]
  float decay;
  int new_keys;        // 1: a request's last l_q keys start from zero
  int hqo, group;
  float scale_log2;    // logit scale in the log2 domain (includes k_scale)
  float cap_log2, inv_cap_log2;  // soft-cap, 0 for none
  int wide_cap;        // the soft-cap is above kExpTanhMostCap
  int window_left;     // >= 0: sliding window (the tensor-core form reads it from the plan)
  // tensor-core form
  int tile_tokens;      // tokens of a Q tile: 128 / group
  float* part;          // [CTAs][2][256] partial sums of items cut between CTAs
  uint32_t* part_count; // [CTAs], zero between launches
};
constexpr int kRowsMostWarps = 16;  // most warps of a CTA of the row form
int launch_weights_rows(const WeightsParams& p, bool fp8, int64_t most_blk, int num_sms, cudaStream_t stream);

int launch_weights_tc(const WeightsParams& p, int total_q, bool fp8, int num_sms, cudaStream_t stream);

struct SelectParams {
  PageView pv;
  const float* weights;
  int32_t* kept;  // [batch, hkv, budget]
  int sink, recent, budget;
  int by_four;  // weights can be fetched four slots at a time; set by the launcher
};
int launch_select(SelectParams p, int batch, int most_batch, int max_lkv, int num_sms, cudaStream_t stream);

struct CompactParams {
  PageView pv;
  const int32_t* kept;  // [batch, hkv, budget]
  void *k_pages, *v_pages;
  float* weights;  // or null
  int budget;
};
int launch_compact(const CompactParams& p, int batch, int most_batch, bool fp8, int num_sms, cudaStream_t stream);

}  // namespace fi
