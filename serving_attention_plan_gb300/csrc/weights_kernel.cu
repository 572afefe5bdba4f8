// Accumulated attention weights, row form: w_j = sum over the query rows (tokens x heads of the KV
// head's group) that see key j of exp(logit_j - lse_row), added to the decayed running sum of the
// key's page slot.
//
// For a decode step the bound is one read of the K cache, so everything serves to keep reads in flight.
// A warp owns 32 keys of one KV head at a time as two 16-row A operands of warp-level MMAs.  The
// contraction index may be permuted freely as long as K and Q agree, so lane (row, t) takes the
// 16 bytes at dims 32 c + 8 t of its rows as two k-steps' fragments: reads are full 32-byte sectors, and
// every lane consumes exactly the bytes it fetched.  They go through a ring in shared memory that is private to
// the lane (asynchronous copies, no registers, no barrier), several units ahead; page ids are fetched one
// unit earlier still.  (With the fragments loaded straight into registers a warp had one unit in flight
// behind its look-ups: 115 us for 128 requests of U[1, 4096] keys and 88 us for 2 x 115 K keys of e4m3 at page size
// 1, now 95 (0.90 of the copy rate) and 56.)
// The keys sit on the 16-row side and 8 query rows on the other; K stays in registers while the warp walks
// over the query rows in groups of 8, so the form is right for any number of rows.  Query fragments
// of at most 8 rows are kept from unit to unit while the request and head stay the same, which the unit order makes
// the rule (heads fastest, eight warps).  Each key is summed by one warp in one order: results do
// not depend on scheduling.
#include <cuda_fp8.h>

#include <algorithm>
#include <mutex>

#include "cache_common.cuh"
#include "prefill_launch.h"

namespace fi {
namespace {

// Warps of a CTA (one CTA per SM), multiples of eight so that a warp mostly keeps its head, and units in flight of
// each: 8 x 3 x 8 KB of bf16, 16 x 3 x 4 KB of e4m3, whose conversions need more warps (2 x 115 K
// keys: 56 us, with 8 x 6 units 69).
template <bool kFp8>
constexpr int kRowsWarps = kFp8 ? kRowsMostWarps : 8;
template <bool kFp8>
constexpr int kAhead = 3;
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ void mma_16816_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
               "{%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two e4m3 codes (low 16 bits) -> two f16 (exact).
__device__ __forceinline__ uint32_t widen2(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes & 0xffffu), __NV_E4M3);
  return uint32_t(h.x) | (uint32_t(h.y) << 16);
}

__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w) {
  const float2 f = bf16x2_to_f2(w);
  const __half2 h = __floats2half2_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A lane's share of one 128-dim row: 32 elements as 16 pairs, in k-step order (pair 2 s and 2 s + 1
// are k-step s's).  bf16: 16 bytes at dims 32 c + 8 t, c = 0..3; e4m3: 16 codes at dims 64 c + 16 t.
template <bool kFp8>
constexpr int kPieces = kFp8 ? 2 : 4;

template <bool kFp8>
struct RowsSmem {
  static constexpr int kWarps = kRowsWarps<kFp8>, kStages = kAhead<kFp8>;
  uint4 k[kWarps][kStages][4 * kPieces<kFp8>][32];  // [..][row i, piece c][lane]
  float old[kWarps][kStages][32];  // the key's running sum
  int at[kWarps][kStages][32];     // its place in the weights, -1: none
  int4 unit[kWarps][kStages][2];   // {first key, head, q0, lq}, {lkv, request, 0, 0}
};

template <bool kFp8>
__device__ __forceinline__ uint32_t pair_of(const uint4 (&v)[kPieces<kFp8>], int i) {  // i a constant after unrolling
  const uint32_t* w = reinterpret_cast<const uint32_t*>(v);
  if constexpr (kFp8) return widen2(w[i >> 1] >> (16 * (i & 1)));
  return w[i];
}

// The matching share of a query row.
template <bool kFp8>
__device__ __forceinline__ void load_q(const __nv_bfloat16* row, int t, uint32_t (&b)[16]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int dim = kFp8 ? 64 * (c >> 1) + 16 * t + 8 * (c & 1) : 32 * c + 8 * t;
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(row + dim));
    b[4 * c] = kFp8 ? bf16x2_to_f16x2(v.x) : v.x;
    b[4 * c + 1] = kFp8 ? bf16x2_to_f16x2(v.y) : v.y;
    b[4 * c + 2] = kFp8 ? bf16x2_to_f16x2(v.z) : v.z;
    b[4 * c + 3] = kFp8 ? bf16x2_to_f16x2(v.w) : v.w;
  }
}

// Variant of a kernel: none, a window or soft-cap, or a soft-cap above kExpTanhMostCap (with or without a window).
enum Var { kVarNone = 0, kVarOn, kVarWideCap };

template <bool kFp8, int kVar>
__global__ void __launch_bounds__(32 * kRowsWarps<kFp8>, 1) weights_rows_kernel(const __grid_constant__ WeightsParams p) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  RowsSmem<kFp8>& sm = *reinterpret_cast<RowsSmem<kFp8>*>(smem_raw);
  constexpr int kS = kAhead<kFp8>, kP = kPieces<kFp8>, kW = kRowsWarps<kFp8>;
  wait_prior_grid();
  const PageView& pv = p.pv;
  const GeoHead plan = load_head(pv.geo);
  const int batch = plan.batch;
  if (batch == 0) return;
  const bool causal = plan.causal != 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, t = lane & 3;
  // this CTA's run of (block, KV head) units, heads fastest; its warps take them in turn
  const long long units = (long long)plan.blocks * pv.hkv;
  const long long begin = units * blockIdx.x / gridDim.x, end = units * (blockIdx.x + 1) / gridDim.x;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q);
  const uint8_t* pages = static_cast<const uint8_t*>(p.k_pages);
  const int page_rows = int(pv.page_stride / kHeadDim), slot_rows = int(pv.tok_stride / kHeadDim),
            head_rows = int(pv.head_stride / kHeadDim);

  // look-up: the request and page id of the unit that is fetched next, blk and head stepping along
  const long long first = begin + warp;
  int blk = int(first / pv.hkv), next_head = int(first - (long long)blk * pv.hkv);
  const int step_blk = kW / pv.hkv, step_head = kW - step_blk * pv.hkv;
  int r = -1, next_blk = 0, key0 = 0, head = 0, page = 0, slot = 0;
  Geo g{};
  auto look_up = [&](long long u) {
    page = -1;
    if (u >= end) return;
    if (r < 0 || blk >= next_blk) {
      r = find_request(pv.geo, batch, &Geo::blk0, blk);
      g = load_geo(pv.geo, r);
      next_blk = __ldg(&pv.geo[r + 1].blk0);
    }
    head = next_head;
    key0 = (blk - g.blk0) * kBlkKeys;
    // the lane looks up key gid + 8 t; row i of its K rows is key gid + 8 i
    const int key = key0 + gid + 8 * t;
    const int e = pv.page_shift >= 0 ? key >> pv.page_shift : key / pv.page_size;
    slot = key - e * pv.page_size;
    if (key < g.lkv) page = __ldg(pv.kv_indices + g.kv0 + e);
    blk += step_blk;
    next_head += step_head;
    if (next_head >= pv.hkv) {
      next_head -= pv.hkv;
      ++blk;
    }
  };
  // fetch of the unit just looked up into stage s of the ring
  auto fetch = [&](long long u, int s) {
    if (u < end) {
      int row = -1, at = -1;
      if (page >= 0) {
        if (page < pv.num_pages) {
          row = page * page_rows + slot * slot_rows + head * head_rows;
          at = int(weight_offset(pv, page, slot, head));
        } else {
          atomicOr(pv.err, FI_DEVERR_PAGE_OOB);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int src = __shfl_sync(kAll, row, gid * 4 + i);
        const uint8_t* from = pages + (long long)max(src, 0) * (kHeadDim * (kFp8 ? 1 : 2)) + 16 * t;
#pragma unroll
        for (int c = 0; c < kP; ++c) cp_async_16_or_none(&sm.k[warp][s][i * kP + c][lane], from + 64 * c, src >= 0);
      }
      const bool keeps = at >= 0 && p.decay != 0.f && !(p.new_keys && key0 + gid + 8 * t >= g.lkv - g.lq);
      if (keeps)
        cp_async_4(&sm.old[warp][s][lane], p.weights + at);
      else
        sm.old[warp][s][lane] = 0.f;
      sm.at[warp][s][lane] = at;
      if (lane == 0) {
        sm.unit[warp][s][0] = make_int4(key0, head, g.q0, g.lq);
        sm.unit[warp][s][1] = make_int4(g.lkv, r, 0, 0);
      }
    }
    cp_async_commit();
  };

  look_up(first);
#pragma unroll 1
  for (int s = 0; s < kS - 1; ++s) {
    fetch(first + s * kW, s);
    look_up(first + (s + 1) * kW);
  }
  // the query rows at hand: fragments, and of the two columns whose scores this lane gets -lse and the
  // bounds of the keys [low, lim) that the column's token sees
  uint32_t b[16];
  float nl[2];
  int lim[2], low[2];
  int last_r = -1, last_head = -1;
  int s = 0, s_in = kS - 1;
#pragma unroll 1
  for (long long u = first; u < end; u += kW) {
    fetch(u + (kS - 1) * kW, s_in);
    look_up(u + kS * kW);
    __syncwarp();
    const int4 ua = sm.unit[warp][s][0], ub = sm.unit[warp][s][1];
    const int k0 = ua.x, h = ua.y, q0 = ua.z, lkv = ub.x, diag = lkv - ua.w, rows = ua.w * p.group;
    const bool same = ub.y == last_r && h == last_head && rows <= 8;
    last_r = ub.y;
    last_head = h;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    uint4 k[4][kP];
    for (int n0 = 0; n0 < rows; n0 += 8) {
      if (!same) {
        {
          const int n = n0 + gid;
          const int tok = n / p.group, hh = n - tok * p.group;
          if (n < rows) {
            load_q<kFp8>(q + ((long long)(q0 + tok) * p.hqo + h * p.group + hh) * kHeadDim, t, b);
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) b[i] = 0;
          }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int n = n0 + 2 * t + c;
          const int tok = n / p.group, hh = n - tok * p.group;
          lim[c] = low[c] = 0;
          nl[c] = 0.f;
          if (n < rows) {
            nl[c] = -kLog2e * __ldg(p.lse + (long long)(q0 + tok) * p.hqo + h * p.group + hh);
            lim[c] = causal ? min(lkv, diag + tok + 1) : lkv;
            if (nl[c] == INFINITY) lim[c] = 0;  // lse = -inf: the row saw no key
            if (kVar && p.window_left >= 0) low[c] = diag + tok - p.window_left;
          }
        }
      }
      if (n0 == 0) {
        cp_async_wait<kS - 1>();  // this lane's share of the unit has landed
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int c = 0; c < kP; ++c) k[i][c] = sm.k[warp][s][i * kP + c][lane];
      }
      float acc[2][4];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[m][e] = 0.f;
      }
#pragma unroll
      for (int st = 0; st < 8; ++st) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const uint32_t a[4] = {pair_of<kFp8>(k[2 * m], 2 * st), pair_of<kFp8>(k[2 * m + 1], 2 * st),
                                 pair_of<kFp8>(k[2 * m], 2 * st + 1), pair_of<kFp8>(k[2 * m + 1], 2 * st + 1)};
          if constexpr (kFp8)
            mma_16816_f16(acc[m], a, b[2 * st], b[2 * st + 1]);
          else
            mma_16816(acc[m], a, b[2 * st], b[2 * st + 1]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = k0 + gid + 8 * i;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float x = acc[i >> 1][2 * (i & 1) + c] * p.scale_log2;
          if constexpr (kVar == kVarWideCap) {
            const float y = x * p.inv_cap_log2, u = y * y;
            x = p.cap_log2 * (u <= kNearReach ? y * tanh_near_factor(make_float2(u, u)).x : tanh_exp2(y));
          } else if (kVar != kVarNone && p.cap_log2 > 0.f) {
            x = p.cap_log2 * tanh_exp2(x * p.inv_cap_log2);
          }
          // the select drops what hidden keys and missing rows computed, NaN included
          const bool seen = key < lim[c] && (!kVar || key >= low[c]);
          sum[i] += seen ? fast_exp2(x + nl[c]) : 0.f;
        }
      }
    }
    if (rows == 0) cp_async_wait<kS - 1>();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sum[i] += __shfl_xor_sync(kAll, sum[i], 1);
      sum[i] += __shfl_xor_sync(kAll, sum[i], 2);
    }
    const float w = t == 0 ? sum[0] : t == 1 ? sum[1] : t == 2 ? sum[2] : sum[3];
    const int at = sm.at[warp][s][lane];
    if (at >= 0) p.weights[at] = p.decay * sm.old[warp][s][lane] + w;
    __syncwarp();  // the stage is read out before it is filled again
    s = s + 1 == kS ? 0 : s + 1;
    s_in = s_in + 1 == kS ? 0 : s_in + 1;
  }
  cp_async_wait<0>();
}

}  // namespace

int launch_weights_rows(const WeightsParams& p, bool fp8, int64_t most_blk, int num_sms, cudaStream_t stream) {
  const int64_t units = most_blk * p.pv.hkv;
  const int warps = fp8 ? kRowsWarps<true> : kRowsWarps<false>;
  const unsigned grid = unsigned(std::max<int64_t>(1, std::min<int64_t>((units + warps - 1) / warps, num_sms)));
  const int var = p.wide_cap ? kVarWideCap : p.window_left >= 0 || p.cap_log2 > 0.f ? kVarOn : kVarNone;
  using Kernel = void (*)(const WeightsParams);
  static const Kernel kernels[6] = {weights_rows_kernel<false, kVarNone>, weights_rows_kernel<false, kVarOn>, weights_rows_kernel<false, kVarWideCap>,
                                    weights_rows_kernel<true, kVarNone>, weights_rows_kernel<true, kVarOn>, weights_rows_kernel<true, kVarWideCap>};
  static std::once_flag once;
  static cudaError_t attr = cudaSuccess;
  const size_t smem[2] = {sizeof(RowsSmem<false>), sizeof(RowsSmem<true>)};
  static_assert(sizeof(RowsSmem<false>) <= 227 * 1024 && sizeof(RowsSmem<true>) <= 227 * 1024, "shared memory per CTA");
  std::call_once(once, [&] {
    for (int i = 0; i < 6 && attr == cudaSuccess; ++i)
      attr = cudaFuncSetAttribute(kernels[i], cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem[i / 3]));
  });
  if (attr != cudaSuccess) return record_cuda_error(attr, "cudaFuncSetAttribute(weights_rows_kernel)");
  const cudaError_t e =
      launch_dependent(kernels[(fp8 ? 3 : 0) + var], grid, unsigned(32 * warps), smem[fp8 ? 1 : 0], 1, stream, p);
  return e == cudaSuccess ? 0 : record_cuda_error(e, "weights_rows_kernel launch");
}

}  // namespace fi
