// Accumulated attention weights, tensor-core form: the same sums as the row form, for plans with more
// than 8 query rows a request (prompts and chunks).
//
//   w_j = sum over query rows r (tokens x heads of the group) that see key j of exp2(scale2 q_r.k_j - lse2_r)
//
// The scores are computed as S^T = K Q^T: keys are the 128 lanes of the tcgen05 accumulator, query
// rows its columns.  A thread then owns one key and sums over columns in its own registers: no
// maximum, no cross-lane step, no second product, and one write per key at the end.  A work item is
// 256 keys of one KV head (two 128-lane MMA tiles that share every Q tile, which halves the L2
// traffic of Q) against all query rows that see one of them, in tiles of 128 rows (128 / g tokens x
// g heads, one TMA box a 64-dim half).
//
// What bounds it: per Q tile and item the tensor cores take 2 x 128x128x128 products (1024 clocks at
// the nominal rate) and the exponentials 32768 results (1024 clocks at 32 a clock and SM): the two
// run at the same time, with two score buffers per half.
//
// Work split: the Q tiles of all items lie on one line, request by request, KV head by KV head, key
// tile by key tile (the causal mask gives later key tiles fewer Q tiles); CTA c takes the c-th
// equal piece, so CTAs differ by one Q tile however ragged the batch is.  An item cut by a piece's
// border leaves its partial sums in a slot per CTA, and the last of its CTAs to finish adds them in
// line order: the result does not depend on who is last.  Each CTA has at most two cut items, so the
// slots are bounded by the grid, not by the batch.
//
// One CTA per SM, 14 warps:
//   warps 0-7    exponentials and sums: warps 0-3 the first 128 keys, 4-7 the others
//   warp 8       TMA producer of Q tiles (three stages) and their lse rows
//   warp 9       tensor memory, MMA issue
//   warps 10-13  K tile loader (two stages): 16-byte loads into the 128-byte swizzle, any page size and
//                layout; e4m3 codes are widened to bf16 (exact) on the way, so Q stays bf16
#include <cuda.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <mutex>

#include "cache_common.cuh"
#include "prefill_launch.h"
#include "tcgen05.cuh"

namespace fi {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kTcThreads = 448;
constexpr int kKeys = kTileKeys;                // keys of an item
constexpr int kCols = kWeightTileRows;          // query rows of a Q tile
constexpr int kKHalfBytes = kKeys * 128;        // one 64-dim half of the K tile
constexpr int kQHalfBytes = kCols * 128;
constexpr int kQStages = 3;
constexpr int kKStages = 2;
constexpr uint32_t kTmemCols = 512;             // S[half][buffer]: 128 columns each

struct TcSmem {
  uint8_t k[kKStages][2 * kKHalfBytes];
  uint8_t q[kQStages][2 * kQHalfBytes];
  float nl[kQStages][kCols];  // -lse in the log2 domain, -inf for columns that count for nothing
  int special[kQStages];      // 1: some column of the tile counts for nothing (its score may be anything)
  uint64_t k_full[kKStages], k_empty[kKStages], q_full[kQStages], q_empty[kQStages], l_full[kQStages], l_empty[kQStages];
  uint64_t s_full[2][2], s_empty[2][2];
  uint32_t tmem_base;
  int abort;
  int last;
};

// The CTA's walk over its piece of the line, one segment (run of Q tiles of one item) at a time.
// Every member is uniform over the warp; whole warps call init and next.
struct Walk {
  int pos, end;          // remaining piece of the line
  int r, head, kt;       // request, KV head, key tile
  Geo g;
  int work1;             // line position behind this request
  int t0, cost;          // first query token that sees the item, its Q tiles (at least 1)
  int tokens;            // query tokens that see the item
  int q0, q1;            // Q tiles of this segment

  __device__ __forceinline__ static void item(const WeightsParams& p, bool causal, const Geo& g, int kt, int& t0,
                                              int& tokens, int& cost) {
    weight_item(g.lq, g.lkv, kt, causal, p.window_left, p.tile_tokens, &t0, &tokens, &cost);
  }
  __device__ __forceinline__ void load(const WeightsParams& p) {
    g = load_geo(p.pv.geo, r);
    work1 = __ldg(&p.pv.geo[r + 1].work0);
  }
  __device__ __forceinline__ void segment(const WeightsParams& p, bool causal) {
    item(p, causal, g, kt, t0, tokens, cost);
    q1 = min(cost, q0 + end - pos);
  }
  __device__ void init(const WeightsParams& p, bool causal, int batch, int begin, int finish) {
    const int lane = threadIdx.x & 31;
    pos = begin;
    end = finish;
    if (pos >= end) return;
    r = find_request(p.pv.geo, batch, &Geo::work0, pos);
    load(p);
    const int per_head = (work1 - g.work0) / p.pv.hkv;
    int rem = pos - g.work0;
    head = rem / per_head;
    rem -= head * per_head;
    // the key tile that holds position `rem` of the head's line: a scan over 32 tiles at a time
    int before = 0;
    for (kt = 0;; kt += 32) {
      int a, b, c = 0;
      if ((kt + lane) * kKeys < g.lkv) item(p, causal, g, kt + lane, a, b, c);
      int incl = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kAll, incl, o);
        if (lane >= o) incl += v;
      }
      const int all = __shfl_sync(kAll, incl, 31);
      if (rem < before + all) {
        const int at = __ffs(__ballot_sync(kAll, rem < before + incl)) - 1;
        before += __shfl_sync(kAll, incl - c, at);
        kt += at;
        break;
      }
      before += all;
    }
    q0 = rem - before;
    segment(p, causal);
  }
  __device__ __forceinline__ bool more() const { return pos < end; }
  __device__ void next(const WeightsParams& p, bool causal) {
    pos += q1 - q0;
    if (pos >= end) return;
    q0 = 0;
    ++kt;
    if (kt * kKeys >= g.lkv) {
      kt = 0;
      if (++head == p.pv.hkv) {
        head = 0;
        do {
          ++r;
          load(p);
        } while (work1 == g.work0);
      }
    }
    segment(p, causal);
  }
};

// Four e4m3 codes -> four bf16 (exact: e4m3 values have 4 significant bits and small exponents).
__device__ __forceinline__ uint2 widen4(uint32_t codes) {
  const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes & 0xffffu), __NV_E4M3);
  const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes >> 16), __NV_E4M3);
  const float2 a = __half22float2(__half2(lo)), b = __half22float2(__half2(hi));
  return make_uint2(f2_to_bf16x2(a.x, a.y), f2_to_bf16x2(b.x, b.y));
}

template <bool kFp8>
__device__ void load_keys(const WeightsParams& p, TcSmem& sm, Walk w, bool causal) {
  const PageView& pv = p.pv;
  const int tid = threadIdx.x - 320;             // 0..127
  constexpr int kLanes = kFp8 ? 8 : 16;          // threads of a row, 16 bytes each
  constexpr int kRowsPass = 128 / kLanes;
  constexpr int kBatch = 8;
  const int ch = tid % kLanes, row0 = tid / kLanes;
  const uint8_t* pages = static_cast<const uint8_t*>(p.k_pages);
  for (int n = 0; w.more(); w.next(p, causal), ++n) {
    const int ks = n % kKStages;
    bool ok = true;
    if (n >= kKStages) ok = mbar_wait(&sm.k_empty[ks], (n / kKStages - 1) & 1, pv.err, &sm.abort);
    if (!__all_sync(kAll, ok)) return;
    for (int i0 = 0; i0 < kKeys; i0 += kBatch * kRowsPass) {
      uint4 v[kBatch];
      long long off[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int key = w.kt * kKeys + i0 + i * kRowsPass + row0;
        int page, slot;
        off[i] = -1;
        if (key < w.g.lkv && locate(pv, w.g.kv0, key, page, slot)) off[i] = kv_offset(pv, page, slot, w.head);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        v[i] = off[i] >= 0 ? __ldg(reinterpret_cast<const uint4*>(pages + off[i] * (kFp8 ? 1 : 2) + 16 * ch))
                           : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int row = i0 + i * kRowsPass + row0;
        auto put = [&](int c16, uint4 x) {  // 16-byte piece c16 (0..15) of a bf16 row
          uint8_t* at = sm.k[ks] + (c16 >> 3) * kKHalfBytes + row * 128 + (((c16 & 7) ^ (row & 7)) << 4);
          *reinterpret_cast<uint4*>(at) = x;
        };
        if constexpr (kFp8) {
          const uint2 a = widen4(v[i].x), b = widen4(v[i].y), c = widen4(v[i].z), d = widen4(v[i].w);
          put(2 * ch, make_uint4(a.x, a.y, b.x, b.y));
          put(2 * ch + 1, make_uint4(c.x, c.y, d.x, d.y));
        } else {
          put(ch, v[i]);
        }
      }
    }
    fence_proxy_async_smem();
    mbar_arrive(&sm.k_full[ks]);
  }
}

__device__ void load_queries(const WeightsParams& p, TcSmem& sm, Walk w, bool causal, const CUtensorMap* tm_q) {
  const int lane = threadIdx.x & 31;
  const int cols = p.tile_tokens * p.group;
  int n = 0;
  bool ok = true;
  for (; ok && w.more(); w.next(p, causal)) {
    // this lane's columns are lane + 32 i: their place in the tile does not change
    int tok[4], hh[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      tok[i] = (lane + 32 * i) / p.group;
      hh[i] = (lane + 32 * i) - tok[i] * p.group;
    }
    auto fetch = [&](int qt, float (&nl)[4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = qt * p.tile_tokens + tok[i];
        nl[i] = -INFINITY;
        if (lane + 32 * i < cols && t < w.tokens) {
          const float l = __ldg(p.lse + (long long)(w.g.q0 + w.t0 + t) * p.hqo + w.head * p.group + hh[i]);
          if (l != -INFINITY) nl[i] = -kLog2e * l;
        }
      }
    };
    float cur[4], nxt[4];
    fetch(w.q0, cur);
    for (int qt = w.q0; ok && qt < w.q1; ++qt, ++n) {
      const int qs = n % kQStages;
      if (n >= kQStages) {
        ok = mbar_wait(&sm.q_empty[qs], (n / kQStages - 1) & 1, p.pv.err, &sm.abort) &&
             mbar_wait(&sm.l_empty[qs], (n / kQStages - 1) & 1, p.pv.err, &sm.abort);
        ok = __all_sync(kAll, ok);
        if (!ok) break;
      }
      if (lane == 0) {
        mbar_arrive_expect_tx(&sm.q_full[qs], uint32_t(2 * 128 * cols));
        const int tok0 = w.g.q0 + w.t0 + qt * p.tile_tokens;
        tc::tma_load_3d(sm.q[qs], tm_q, 0, w.head * p.group, tok0, &sm.q_full[qs]);
        tc::tma_load_3d(sm.q[qs] + kQHalfBytes, tm_q, 64, w.head * p.group, tok0, &sm.q_full[qs]);
      }
      if (qt + 1 < w.q1) fetch(qt + 1, nxt);
      bool dead = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sm.nl[qs][lane + 32 * i] = cur[i];
        dead |= lane + 32 * i < cols && cur[i] == -INFINITY;
        cur[i] = nxt[i];
      }
      const bool any = __any_sync(kAll, dead);
      if (lane == 0) sm.special[qs] = any;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.l_full[qs]);
    }
  }
  // never leave with tensor copies still landing in this CTA's shared memory
  for (int k = max(0, n - kQStages); k < n; ++k) mbar_wait_bounded(&sm.q_full[k % kQStages], (k / kQStages) & 1);
}

__device__ void issue(const WeightsParams& p, TcSmem& sm, Walk w, bool causal, uint32_t tmem) {
  constexpr uint32_t idesc = tc::idesc_bf16_f32(128, kCols, 0, 0);  // A = keys, B = query rows, both K-major
  const bool lead = (threadIdx.x & 31) == 0;
  const uint32_t k_addr = smem_u32(sm.k[0]), q_addr = smem_u32(sm.q[0]);
  int n = 0;
  for (int seg = 0; w.more(); w.next(p, causal), ++seg) {
    const int ks = seg % kKStages;
    if (!__all_sync(kAll, mbar_wait(&sm.k_full[ks], (seg / kKStages) & 1, p.pv.err, &sm.abort))) return;
    for (int qt = w.q0; qt < w.q1; ++qt, ++n) {
      const int qs = n % kQStages, b = n & 1;
      if (!__all_sync(kAll, mbar_wait(&sm.q_full[qs], (n / kQStages) & 1, p.pv.err, &sm.abort))) return;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (n >= 2 && !__all_sync(kAll, mbar_wait(&sm.s_empty[h][b], ((n >> 1) - 1) & 1, p.pv.err, &sm.abort))) return;
        tc::fence_after_sync();
        if (lead) {
#pragma unroll
          for (int kh = 0; kh < 2; ++kh) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const uint64_t a = tc::smem_desc(k_addr + ks * 2 * kKHalfBytes + kh * kKHalfBytes + h * (128 * 128) + kk * 32,
                                               16, 1024, tc::kLayoutSw128);
              const uint64_t bd = tc::smem_desc(q_addr + qs * 2 * kQHalfBytes + kh * kQHalfBytes + kk * 32, 16, 1024,
                                                tc::kLayoutSw128);
              tc::mma_ss(tmem + uint32_t((2 * h + b) * kCols), a, bd, idesc, (kh | kk) != 0 ? 1u : 0u);
            }
          }
          tc::commit(&sm.s_full[h][b]);
        }
        __syncwarp();
      }
      if (lead) tc::commit(&sm.q_empty[qs]);
    }
    if (lead) tc::commit(&sm.k_empty[ks]);
    __syncwarp();
  }
}

// Waits for the tensor-memory loads in flight.  The registers pass through, so that nothing that uses
// them can be scheduled before the wait.
__device__ __forceinline__ void wait_scores(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])::"memory");
}

// 32 scores of the thread's key -> added to acc.  Columns outside [lo, hi) and those with nl = -inf
// count for nothing when kMasked; without it none is outside and all scores are finite or their own
// row's business.
template <bool kMasked, bool kCap>
__device__ __forceinline__ void add32(const uint32_t (&s)[32], const float* nl, int lo, int hi, const WeightsParams& p,
                                      float2 (&acc)[4]) {
  const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float4 n4 = *reinterpret_cast<const float4*>(nl + 4 * j);
    const float nn[4] = {n4.x, n4.y, n4.z, n4.w};
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      const int c = 4 * j + e;
      float2 x = make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1]));
      const float2 n2 = make_float2(nn[e], nn[e + 1]);
      if constexpr (kCap) {
        x = make_float2(p.cap_log2 * tanh_exp2(x.x * p.scale_log2 * p.inv_cap_log2),
                        p.cap_log2 * tanh_exp2(x.y * p.scale_log2 * p.inv_cap_log2));
        x = __fadd2_rn(x, n2);
      } else {
        x = __ffma2_rn(x, sc2, n2);
      }
      float2 w = make_float2(fast_exp2(x.x), fast_exp2(x.y));
      if constexpr (kMasked) {
        w.x = c >= lo && c < hi && nn[e] != -INFINITY ? w.x : 0.f;
        w.y = c + 1 >= lo && c + 1 < hi && nn[e + 1] != -INFINITY ? w.y : 0.f;
      }
      acc[(c >> 1) & 3] = __fadd2_rn(acc[(c >> 1) & 3], w);
    }
  }
}

template <bool kWin, bool kCap>
__device__ void sum_weights(const WeightsParams& p, TcSmem& sm, Walk w, bool causal, uint32_t tmem, int line, int ctas) {
  const PageView& pv = p.pv;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, h = warp >> 2;
  const int row = threadIdx.x;  // key of the item: 128 h + TMEM lane
  const uint32_t lane_base = tmem + (uint32_t((warp & 3) * 32) << 16);
  int n = 0;
  bool alive = true;
  for (; w.more(); w.next(p, causal)) {
    const int key = w.kt * kKeys + row;
    const int diag = w.g.lkv - w.g.lq;  // position of the request's first query token
    float* out = nullptr;
    float old = 0.f;
    {
      int page, slot;
      if (key < w.g.lkv && locate(pv, w.g.kv0, key, page, slot)) out = p.weights + weight_offset(pv, page, slot, w.head);
      if (out != nullptr && p.decay != 0.f && !(p.new_keys && key >= diag)) old = p.decay * __ldcg(out);
    }
    float sum = 0.f;
    for (int qt = w.q0; qt < w.q1; ++qt, ++n) {
      const int qs = n % kQStages, b = n & 1;
      alive = alive && __all_sync(kAll, mbar_wait(&sm.l_full[qs], (n / kQStages) & 1, pv.err, &sm.abort) &&
                                            mbar_wait(&sm.s_full[h][b], (n >> 1) & 1, pv.err, &sm.abort));
      if (alive) {
        tc::fence_after_sync();
        const uint32_t t_s = lane_base + uint32_t((2 * h + b) * kCols);
        const int tok = w.t0 + qt * p.tile_tokens;  // first token of the tile
        // column c belongs to token tok + c / g; key sees tokens from key - diag to key - diag + window
        int lo = 0, hi = kCols;
        if (causal) {
          lo = min(kCols, max(0, (key - diag - tok)) * p.group);
          if (kWin) hi = int(max(0ll, min((long long)p.tile_tokens, (long long)key - diag - tok + p.window_left + 1))) * p.group;
          if (kWin && hi == p.tile_tokens * p.group) hi = kCols;
        }
        const bool masked = __any_sync(kAll, lo > 0 || hi < kCols) || sm.special[qs];
        float2 acc[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = make_float2(0.f, 0.f);
        uint32_t s[2][32];
        tc::tmem_ld32(t_s, s[0]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          wait_scores(s[c & 1]);
          if (c < 3) tc::tmem_ld32(t_s + 32 * (c + 1), s[(c + 1) & 1]);
          if (c == 3) {
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.s_empty[h][b]);
          }
          if (masked)
            add32<true, kCap>(s[c & 1], sm.nl[qs] + 32 * c, lo - 32 * c, hi - 32 * c, p, acc);
          else
            add32<false, kCap>(s[c & 1], sm.nl[qs] + 32 * c, 0, 32, p, acc);
        }
        const float2 a = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
        sum += a.x + a.y;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.l_empty[qs]);
    }
    if (!alive) out = nullptr;  // the error is recorded; the barriers and counts below still go their way
    if (w.q0 == 0 && w.q1 == w.cost) {
      if (out != nullptr) *out = old + sum;
      continue;
    }
    // a cut item: leave this piece, the last of its CTAs adds all of them in line order
    const int start = w.pos - w.q0;
    const int c1 = int(((long long)(start + 1) * ctas - 1) / line), c2 = int(((long long)(start + w.cost) * ctas - 1) / line);
    p.part[(size_t(blockIdx.x) * 2 + (w.q0 == 0 ? 1 : 0)) * kKeys + row] = sum;
    __threadfence();
    named_bar_sync(1, 256);
    if (threadIdx.x == 0) sm.last = atomicAdd(p.part_count + c1, 1u) == unsigned(c2 - c1);
    named_bar_sync(1, 256);
    if (sm.last) {
      __threadfence();
      float total = 0.f;
      for (int c = c1; c <= c2; ++c) total += __ldcg(p.part + (size_t(c) * 2 + (c == c1 ? 1 : 0)) * kKeys + row);
      if (out != nullptr) *out = old + total;
      if (threadIdx.x == 0) p.part_count[c1] = 0;
    }
  }
}

template <bool kFp8, bool kWin, bool kCap>
__global__ void __launch_bounds__(kTcThreads, 1)
    weights_tc_kernel(const __grid_constant__ WeightsParams p, const __grid_constant__ CUtensorMap tm_q) {
  extern __shared__ unsigned char smem_raw[];
  TcSmem& sm = *reinterpret_cast<TcSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(&sm.k_full[i], 128);
      mbar_init(&sm.k_empty[i], 1);
    }
    for (int i = 0; i < kQStages; ++i) {
      mbar_init(&sm.q_full[i], 1);
      mbar_init(&sm.q_empty[i], 1);
      mbar_init(&sm.l_full[i], 1);
      mbar_init(&sm.l_empty[i], 8);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sm.s_full[i >> 1][i & 1], 1);
      mbar_init(&sm.s_empty[i >> 1][i & 1], 4);
    }
    sm.abort = 0;
    fence_mbar_init();
  }
  if (p.tile_tokens * p.group < kCols) {  // rows of the Q stages that no copy fills: zero scores
    for (int i = threadIdx.x; i < int(sizeof(sm.q) / 16); i += kTcThreads)
      reinterpret_cast<uint4*>(sm.q[0])[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  if (warp == 8 && lane == 0) tc::tma_prefetch_desc(&tm_q);
  if (warp == 9) {
    tc::tmem_alloc(&sm.tmem_base, kTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  wait_prior_grid();
  const uint32_t tmem = sm.tmem_base;
  const int batch = __ldg(p.pv.header + H_BATCH);
  const bool causal = __ldg(p.pv.header + H_CAUSAL) != 0;
  const int line = __ldg(&p.pv.geo[batch].work0);
  const int ctas = min(int(gridDim.x), line);
  if ((tmem & 0xFFFFu) + kTmemCols > 512u) {
    if (threadIdx.x == 0) atomicOr(p.pv.err, FI_DEVERR_TMEM);
  } else if (int(blockIdx.x) < ctas) {
    Walk w;
    w.init(p, causal, batch, int((long long)line * blockIdx.x / ctas), int((long long)line * (blockIdx.x + 1) / ctas));
    if (warp < 8)
      sum_weights<kWin, kCap>(p, sm, w, causal, tmem, line, ctas);
    else if (warp == 8)
      load_queries(p, sm, w, causal, &tm_q);
    else if (warp == 9)
      issue(p, sm, w, causal, tmem);
    else
      load_keys<kFp8>(p, sm, w, causal);
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 9) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace

int launch_weights_tc(const WeightsParams& p, int total_q, bool fp8, int num_sms, cudaStream_t stream) {
  CUtensorMap tq;
  if (!make_query_map(&tq, p.q, p.hqo, total_q, p.group, p.tile_tokens)) return FI_ERR_INVALID_ARG;
  constexpr size_t smem = sizeof(TcSmem) + 1024;
  static_assert(smem <= 227 * 1024, "shared memory exceeds the per-CTA limit");
  using Kernel = void (*)(const WeightsParams, const CUtensorMap);
  static const Kernel kernels[8] = {
      weights_tc_kernel<false, false, false>, weights_tc_kernel<false, false, true>, weights_tc_kernel<false, true, false>,
      weights_tc_kernel<false, true, true>,   weights_tc_kernel<true, false, false>, weights_tc_kernel<true, false, true>,
      weights_tc_kernel<true, true, false>,   weights_tc_kernel<true, true, true>};
  static std::once_flag once;
  static cudaError_t attr = cudaSuccess;
  std::call_once(once, [] {
    for (int i = 0; i < 8 && attr == cudaSuccess; ++i)
      attr = cudaFuncSetAttribute(kernels[i], cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  });
  if (attr != cudaSuccess) return record_cuda_error(attr, "cudaFuncSetAttribute(weights_tc_kernel)");
  const Kernel k = kernels[(fp8 ? 4 : 0) + (p.window_left >= 0 ? 2 : 0) + (p.cap_log2 > 0.f ? 1 : 0)];
  const cudaError_t e = launch_dependent(k, unsigned(num_sms), kTcThreads, smem, 1, stream, p, tq);
  return e == cudaSuccess ? 0 : record_cuda_error(e, "weights_tc_kernel launch");
}

}  // namespace fi
