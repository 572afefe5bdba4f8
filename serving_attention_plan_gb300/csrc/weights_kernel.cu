// Accumulated attention weights, row form: w_j = sum over the query rows (tokens x heads of the KV
// head's group) that see key j of exp(logit_j - lse_row), added to the decayed running sum of the
// key's page slot.
//
// For a decode step the bound is one read of the K cache, so K goes straight from memory into the
// operand registers of warp-level MMAs and nothing else moves: a warp owns 32 keys of one KV head
// as two 16-row A operands.  The contraction index may be permuted freely as long as K and Q agree,
// so lane (row, t) takes the 16 bytes at dims 32 c + 8 t of its rows as two k-steps' fragments:
// loads are full 32-byte sectors, and there is no shared memory, no barrier and no cross-warp sum.
// The keys sit on the 16-row side and 8 query rows on the other; K stays in registers while the
// warp walks over the query rows in groups of 8, so the form is right for any number of rows.
// Each key is summed by one warp in one order: results do not depend on scheduling.
#include <cuda_fp8.h>

#include <algorithm>

#include "cache_common.cuh"
#include "prefill_launch.h"

namespace fi {
namespace {

constexpr int kRowsThreads = 256;
constexpr int kRowsWarps = kRowsThreads / 32;
constexpr int kRowsCtasPerSm = 2;
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

// Plain loads past L1: each K byte is used once.
__device__ __forceinline__ uint4 load_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// A lane's share of one 128-dim row: 32 elements as 16 pairs, in k-step order (pair 2 s and 2 s + 1
// are k-step s's).  bf16: 16 bytes at dims 32 c + 8 t, c = 0..3; e4m3: 16 codes at dims 64 c + 16 t.
template <bool kFp8>
struct KRow {
  uint4 v[kFp8 ? 2 : 4];
  __device__ __forceinline__ void load(const void* row, int t) {
#pragma unroll
    for (int c = 0; c < (kFp8 ? 2 : 4); ++c) v[c] = load_stream(static_cast<const uint8_t*>(row) + 64 * c + 16 * t);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int c = 0; c < (kFp8 ? 2 : 4); ++c) v[c] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ uint32_t pair(int i) const {  // i in 0..15, a constant after unrolling
    const uint32_t* w = reinterpret_cast<const uint32_t*>(v);
    if constexpr (kFp8) return widen2(w[i >> 1] >> (16 * (i & 1)));
    return w[i];
  }
};

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

template <bool kFp8, bool kVar>
__global__ void __launch_bounds__(kRowsThreads, kRowsCtasPerSm) weights_rows_kernel(const __grid_constant__ WeightsParams p) {
  wait_prior_grid();
  const PageView& pv = p.pv;
  const int batch = __ldg(pv.header + H_BATCH);
  if (batch == 0) return;
  const bool causal = __ldg(pv.header + H_CAUSAL) != 0;
  const int lane = threadIdx.x & 31, gid = lane >> 2, t = lane & 3;
  // this CTA's run of (block, KV head) units, heads fastest; its warps take them in turn
  const long long units = (long long)__ldg(&pv.geo[batch].blk0) * pv.hkv;
  const long long begin = units * blockIdx.x / gridDim.x, end = units * (blockIdx.x + 1) / gridDim.x;
  int r = -1;
  Geo g{};
  int next_blk = 0;
  for (long long u = begin + (threadIdx.x >> 5); u < end; u += kRowsWarps) {
    const int blk = int(u / pv.hkv), head = int(u - (long long)blk * pv.hkv);
    if (r < 0 || blk >= next_blk) {
      r = find_request(pv.geo, batch, &Geo::blk0, blk);
      g = load_geo(pv.geo, r);
      next_blk = __ldg(&pv.geo[r + 1].blk0);
    }
    const int key0 = (blk - g.blk0) * kBlkKeys;
    // the lane looks up key gid + 8 t; row i of its K rows is key gid + 8 i
    const int my_key = key0 + gid + 8 * t;
    long long off = -1;
    float* out = nullptr;
    float old = 0.f;
    {
      int page, slot;
      if (my_key < g.lkv && locate(pv, g.kv0, my_key, page, slot)) {
        off = kv_offset(pv, page, slot, head);
        out = p.weights + weight_offset(pv, page, slot, head);
      }
    }
    KRow<kFp8> k[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long o = __shfl_sync(kAll, off, gid * 4 + i);
      if (o >= 0)
        k[i].load(static_cast<const uint8_t*>(p.k_pages) + o * (kFp8 ? 1 : 2), t);
      else
        k[i].clear();
    }
    const int diag = g.lkv - g.lq;  // position of the request's first query token
    const bool fresh = p.new_keys && my_key >= diag;
    if (out != nullptr && !fresh && p.decay != 0.f) old = p.decay * *out;

    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    const int rows = g.lq * p.group;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q);
    for (int n0 = 0; n0 < rows; n0 += 8) {
      uint32_t b[16];
      {
        const int n = n0 + gid;
        const int tok = n / p.group, hh = n - tok * p.group;
        if (n < rows) {
          load_q<kFp8>(q + ((long long)(g.q0 + tok) * p.hqo + head * p.group + hh) * kHeadDim, t, b);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) b[i] = 0;
        }
      }
      // the two columns whose scores this lane gets
      float nl[2];
      int lim[2], low[2];  // keys [low, lim) are visible to the column's token
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int n = n0 + 2 * t + c;
        const int tok = n / p.group, hh = n - tok * p.group;
        lim[c] = low[c] = 0;
        nl[c] = 0.f;
        if (n < rows) {
          nl[c] = -kLog2e * __ldg(p.lse + (long long)(g.q0 + tok) * p.hqo + head * p.group + hh);
          lim[c] = causal ? min(g.lkv, diag + tok + 1) : g.lkv;
          if (nl[c] == INFINITY) lim[c] = 0;  // lse = -inf: the row saw no key
          if (kVar && p.window_left >= 0) low[c] = diag + tok - p.window_left;
        }
      }
      float acc[2][4];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[m][e] = 0.f;
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          const uint32_t a[4] = {k[2 * m].pair(2 * s), k[2 * m + 1].pair(2 * s), k[2 * m].pair(2 * s + 1),
                                 k[2 * m + 1].pair(2 * s + 1)};
          if constexpr (kFp8)
            mma_16816_f16(acc[m], a, b[2 * s], b[2 * s + 1]);
          else
            mma_16816(acc[m], a, b[2 * s], b[2 * s + 1]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = key0 + gid + 8 * i;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float s = acc[i >> 1][2 * (i & 1) + c] * p.scale_log2;
          if (kVar && p.cap_log2 > 0.f) s = p.cap_log2 * tanh_exp2(s * p.inv_cap_log2);
          // the select drops what hidden keys and missing rows computed, NaN included
          const bool seen = key < lim[c] && (!kVar || key >= low[c]);
          sum[i] += seen ? fast_exp2(s + nl[c]) : 0.f;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sum[i] += __shfl_xor_sync(kAll, sum[i], 1);
      sum[i] += __shfl_xor_sync(kAll, sum[i], 2);
    }
    const float w = t == 0 ? sum[0] : t == 1 ? sum[1] : t == 2 ? sum[2] : sum[3];
    if (out != nullptr) *out = old + w;
  }
}

}  // namespace

int launch_weights_rows(const WeightsParams& p, bool fp8, int64_t n_blk, int num_sms, cudaStream_t stream) {
  const int64_t units = n_blk * p.pv.hkv;
  const unsigned grid =
      unsigned(std::max<int64_t>(1, std::min<int64_t>((units + kRowsWarps - 1) / kRowsWarps, kRowsCtasPerSm * num_sms)));
  const bool var = p.window_left >= 0 || p.cap_log2 > 0.f;
  cudaError_t e;
  if (fp8)
    e = var ? launch_dependent(weights_rows_kernel<true, true>, grid, kRowsThreads, 0, 1, stream, p)
            : launch_dependent(weights_rows_kernel<true, false>, grid, kRowsThreads, 0, 1, stream, p);
  else
    e = var ? launch_dependent(weights_rows_kernel<false, true>, grid, kRowsThreads, 0, 1, stream, p)
            : launch_dependent(weights_rows_kernel<false, false>, grid, kRowsThreads, 0, 1, stream, p);
  return e == cudaSuccess ? 0 : record_cuda_error(e, "weights_rows_kernel launch");
}

}  // namespace fi
