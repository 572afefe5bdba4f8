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
// The item's keys stay in tensor memory as the A operand (128 columns), so the products read only Q
// from shared memory; from shared memory both operands of a 128-column product take its whole
// bandwidth.  The -lse of a column is the same for all keys: it is added by one more 16-wide k-step
// with ones on the key side and -lse / scale, split into three bf16 parts (24 bits), on the query
// side.  (Read from shared memory by the threads, 128 values a thread and tile, it took as long as
// the exponentials: a broadcast still moves 16 bytes a lane.)  The exponential's argument is then one
// multiplication.  With a soft-cap the -lse cannot go inside the tanh and is read that way.
//
// What bounds it: per Q tile and item the tensor cores take 2 x 128x128x144 products (1152 clocks at
// the nominal rate) and the exponentials 32768 results (1024 clocks at 32 a clock and SM): the two
// run at the same time, over three score buffers of 128 columns.
//
// Work split: the Q tiles of all items lie on one line, request by request, KV head by KV head, key
// tile by key tile (the causal mask gives later key tiles fewer Q tiles); CTA c takes the c-th
// equal piece, so CTAs differ by one Q tile however ragged the batch is.  An item cut by a piece's
// border leaves its partial sums in a slot per CTA, and the last of its CTAs to finish adds them in
// line order: the result does not depend on who is last.  Each CTA has at most two cut items, so the
// slots are bounded by the grid, not by the batch.
//
// One CTA per SM, 18 warps:
//   warps 0-7    exponentials and sums: warps 0-3 the first 128 keys, 4-7 the others
//   warps 8-15   key loader: a thread holds one key's 128 dims in registers until the previous item's
//                last product is done, then stores them to tensor memory; any page size and layout;
//                e4m3 codes are widened to bf16 (exact) on the way, so Q stays bf16
//   warp 16      TMA producer of Q tiles (four stages) and writer of their -lse rows
//   warp 17      tensor memory, MMA issue
#include <cuda.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <cstddef>
#include <mutex>

#include "cache_common.cuh"
#include "prefill_launch.h"
#include "tcgen05.cuh"

namespace fi {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kTcThreads = 640;  // five warpgroups; the last one's second half is idle
// Registers after launch (640 threads x 96): 256 x 88 + 256 x 112 + 128 x 80 = 640 x 96.
constexpr uint32_t kSumRegs = 88;
constexpr uint32_t kLoadRegs = 112;
constexpr uint32_t kControlRegs = 80;
constexpr int kKeys = kTileKeys;                // keys of an item
constexpr int kCols = kWeightTileRows;          // query rows of a Q tile
constexpr int kQHalfBytes = kCols * 128;        // 64 dims of a Q tile, or its -lse rows
constexpr int kQStages = 4;
constexpr int kSBufs = 3;
constexpr int kRing = 8;                        // tiles whose column notes are kept
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColK = 0;                   // 64 columns per half of the item's keys
constexpr uint32_t kColS = 128;                 // kSBufs score buffers of 128 columns
constexpr float kDead = -1e30f;                 // -lse / scale of a column that counts for nothing

struct TcSmem {
  uint8_t q[kQStages][2 * kQHalfBytes];
  uint8_t l[kQStages][kQHalfBytes];  // per column 128 bytes: {hi, mid, lo, 0...} of -lse / scale, rest zero
  uint8_t ones[kQHalfBytes];         // the key side of the -lse step: {1, 1, 1, 0...}
  float nl[kRing][kCols];            // soft-cap: -lse in the log2 domain
  uint32_t dead[kRing][4];           // columns that count for nothing, whatever their score is
  uint64_t k_full, k_empty, q_full[kQStages], q_empty[kQStages], l_full[kRing];
  uint64_t s_full[kSBufs], s_empty[kSBufs];
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

// One key row a thread: 128 dims as 64 bf16 pairs, in tensor-memory columns 0..63 of the half.
template <bool kFp8>
__device__ void load_keys(const WeightsParams& p, TcSmem& sm, Walk w, bool causal, uint32_t tmem) {
  const PageView& pv = p.pv;
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) - 8;
  const int row = warp * 32 + lane;
  const uint32_t t_k = tmem + (uint32_t((warp & 3) * 32) << 16) + kColK + uint32_t((warp >> 2) * 64);
  for (int n = 0; w.more(); w.next(p, causal), ++n) {
    const int key = w.kt * kKeys + row;
    uint32_t v[2][32];
    int page, slot;
    const bool on = key < w.g.lkv && locate(pv, w.g.kv0, key, page, slot);
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.k_pages) +
                                                      (on ? kv_offset(pv, page, slot, w.head) * (kFp8 ? 1 : 2) : 0));
    if constexpr (kFp8) {
      uint4 x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = on ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint2 y = widen4(u[e]);
          v[i >> 2][(8 * i + 2 * e) & 31] = y.x;
          v[i >> 2][(8 * i + 2 * e + 1) & 31] = y.y;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint4 x = on ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
        v[i >> 3][(4 * i) & 31] = x.x;
        v[i >> 3][(4 * i + 1) & 31] = x.y;
        v[i >> 3][(4 * i + 2) & 31] = x.z;
        v[i >> 3][(4 * i + 3) & 31] = x.w;
      }
    }
    __syncwarp();
    if (n > 0 && !__all_sync(kAll, mbar_wait(&sm.k_empty, (n - 1) & 1, pv.err, &sm.abort))) return;
    tc::fence_after_sync();
    tc::tmem_st32(t_k, v[0]);
    tc::tmem_st32(t_k + 32, v[1]);
    tc::tmem_wait_st();
    tc::fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.k_full);
  }
}

template <bool kCap>
__device__ void load_queries(const WeightsParams& p, TcSmem& sm, Walk w, bool causal, const CUtensorMap* tm_q) {
  const int lane = threadIdx.x & 31;
  const int cols = p.tile_tokens * p.group;
  const float unit = kCap ? -kLog2e : -kLog2e / p.scale_log2;  // soft-cap: log2 domain; else in units of the raw score
  // this lane's columns are lane + 32 i: their place in the tile does not change
  int tok[4], hh[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    tok[i] = (lane + 32 * i) / p.group;
    hh[i] = (lane + 32 * i) - tok[i] * p.group;
  }
  int n = 0;
  bool ok = true;
  for (; ok && w.more(); w.next(p, causal)) {
    auto fetch = [&](int qt, float (&nl)[4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = qt * p.tile_tokens + tok[i];
        nl[i] = -INFINITY;
        if (lane + 32 * i < cols && t < w.tokens)
          nl[i] = __ldg(p.lse + (long long)(w.g.q0 + w.t0 + t) * p.hqo + w.head * p.group + hh[i]);
      }
    };
    float cur[4], nxt[4];
    fetch(w.q0, cur);
    for (int qt = w.q0; ok && qt < w.q1; ++qt, ++n) {
      const int qs = n % kQStages, ring = n % kRing;
      if (n >= kQStages) {
        ok = __all_sync(kAll, mbar_wait(&sm.q_empty[qs], (n / kQStages - 1) & 1, p.pv.err, &sm.abort));
        if (!ok) break;
      }
      if (lane == 0) {
        mbar_arrive_expect_tx(&sm.q_full[qs], uint32_t(2 * 128 * cols));
        const int tok0 = w.g.q0 + w.t0 + qt * p.tile_tokens;
        tc::tma_load_3d(sm.q[qs], tm_q, 0, w.head * p.group, tok0, &sm.q_full[qs]);
        tc::tma_load_3d(sm.q[qs] + kQHalfBytes, tm_q, 64, w.head * p.group, tok0, &sm.q_full[qs]);
      }
      if (qt + 1 < w.q1) fetch(qt + 1, nxt);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = lane + 32 * i;
        const bool dead = cur[i] == -INFINITY;
        const float v = dead ? kDead : cur[i] * unit;
        if constexpr (kCap) {
          sm.nl[ring][c] = v;
        } else {
          const float hi = __bfloat162float(__float2bfloat16_rn(v));
          const float mid = __bfloat162float(__float2bfloat16_rn(v - hi));
          // 16-byte piece 0 of the 128-byte swizzled row
          *reinterpret_cast<uint2*>(sm.l[qs] + c * 128 + ((c & 7) << 4)) =
              make_uint2(f2_to_bf16x2(hi, mid), f2_to_bf16x2(v - hi - mid, 0.f));
        }
        const uint32_t bits = __ballot_sync(kAll, dead);
        if (lane == 0) sm.dead[ring][i] = bits;
        cur[i] = nxt[i];
      }
      if constexpr (!kCap) fence_proxy_async_smem();  // the MMA reads the -lse rows
      mbar_arrive(&sm.q_full[qs]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.l_full[ring]);
    }
  }
  // never leave with tensor copies still landing in this CTA's shared memory
  for (int k = max(0, n - kQStages); k < n; ++k) mbar_wait_bounded(&sm.q_full[k % kQStages], (k / kQStages) & 1);
}

template <bool kCap>
__device__ void issue(const WeightsParams& p, TcSmem& sm, Walk w, bool causal, uint32_t tmem) {
  constexpr uint32_t idesc = tc::idesc_bf16_f32(128, kCols, 0, 0);  // A = keys, B = query rows, both K-major
  const bool lead = (threadIdx.x & 31) == 0;
  const uint32_t q_addr = smem_u32(sm.q[0]), l_addr = smem_u32(sm.l[0]), ones_addr = smem_u32(sm.ones);
  int n = 0, u = 0;
  for (int seg = 0; w.more(); w.next(p, causal), ++seg) {
    if (!__all_sync(kAll, mbar_wait(&sm.k_full, seg & 1, p.pv.err, &sm.abort))) return;
    for (int qt = w.q0; qt < w.q1; ++qt, ++n) {
      const int qs = n % kQStages;
      if (!__all_sync(kAll, mbar_wait(&sm.q_full[qs], (n / kQStages) & 1, p.pv.err, &sm.abort))) return;
#pragma unroll
      for (int h = 0; h < 2; ++h, ++u) {
        const int b = u % kSBufs;
        if (u >= kSBufs && !__all_sync(kAll, mbar_wait(&sm.s_empty[b], (u / kSBufs - 1) & 1, p.pv.err, &sm.abort)))
          return;
        tc::fence_after_sync();
        if (lead) {
          const uint32_t d = tmem + kColS + uint32_t(b * kCols);
#pragma unroll
          for (int k = 0; k < 8; ++k) {  // 16 dims: 8 columns of the keys, 32 bytes of the Q rows
            const uint64_t bd = tc::smem_desc(q_addr + qs * 2 * kQHalfBytes + (k >> 2) * kQHalfBytes + (k & 3) * 32, 16,
                                              1024, tc::kLayoutSw128);
            tc::mma_ts(d, tmem + kColK + uint32_t(h * 64 + k * 8), bd, idesc, k != 0 ? 1u : 0u);
          }
          if constexpr (!kCap)
            tc::mma_ss(d, tc::smem_desc(ones_addr, 16, 1024, tc::kLayoutSw128),
                       tc::smem_desc(l_addr + qs * kQHalfBytes, 16, 1024, tc::kLayoutSw128), idesc, 1u);
          tc::commit(&sm.s_full[b]);
        }
        __syncwarp();
      }
      if (lead) tc::commit(&sm.q_empty[qs]);
    }
    if (lead) tc::commit(&sm.k_empty);
    __syncwarp();
  }
}

constexpr int kChunk = 16;  // score columns a thread holds at a time (two chunks in flight)
__device__ __forceinline__ void load_scores(uint32_t taddr, uint32_t (&r)[kChunk]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
               "%15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                 "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(taddr));
}
// Waits for the tensor-memory loads in flight.  The registers pass through, so that nothing that uses
// them can be scheduled before the wait.
__device__ __forceinline__ void wait_scores(uint32_t (&r)[kChunk]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}

// A chunk of scores of the thread's key -> added to acc.  With kMasked, columns outside [lo, hi) and dead
// ones count for nothing whatever their score is; without it none is outside, and a dead column's score
// is so low that its power is 0.
template <bool kMasked, bool kCap>
__device__ __forceinline__ void add_chunk(const uint32_t (&s)[kChunk], const float* nl, int lo, int hi, uint32_t dead,
                                          const WeightsParams& p, float2 (&acc)[4]) {
  float2 x[kChunk / 2];
#pragma unroll
  for (int i = 0; i < kChunk / 2; ++i) {
    const float2 v = make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1]));
    if constexpr (kCap) {
      const float in = p.scale_log2 * p.inv_cap_log2;
      const float2 n2 = *reinterpret_cast<const float2*>(nl + 2 * i);
      x[i] = __fadd2_rn(make_float2(p.cap_log2 * tanh_exp2(v.x * in), p.cap_log2 * tanh_exp2(v.y * in)), n2);
    } else {
      x[i] = __fmul2_rn(v, make_float2(p.scale_log2, p.scale_log2));
    }
    if constexpr (kMasked) {
      if (2 * i < lo || 2 * i >= hi || ((dead >> (2 * i)) & 1u)) x[i].x = -INFINITY;
      if (2 * i + 1 < lo || 2 * i + 1 >= hi || ((dead >> (2 * i + 1)) & 1u)) x[i].y = -INFINITY;
    }
  }
#pragma unroll
  for (int i = 0; i < kChunk / 2; ++i) acc[i & 3] = __fadd2_rn(acc[i & 3], make_float2(fast_exp2(x[i].x), fast_exp2(x[i].y)));
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
      const int ring = n % kRing, u = 2 * n + h, b = u % kSBufs;
      alive = alive && __all_sync(kAll, mbar_wait(&sm.l_full[ring], (n / kRing) & 1, pv.err, &sm.abort) &&
                                            mbar_wait(&sm.s_full[b], (u / kSBufs) & 1, pv.err, &sm.abort));
      if (alive) {
        tc::fence_after_sync();
        const uint32_t t_s = lane_base + kColS + uint32_t(b * kCols);
        const int tok = w.t0 + qt * p.tile_tokens;  // first token of the tile
        // column c belongs to token tok + c / g; key sees tokens from key - diag to key - diag + window
        int lo = 0, hi = kCols;
        if (causal) {
          lo = min(kCols, max(0, (key - diag - tok)) * p.group);
          if (kWin) hi = int(max(0ll, min((long long)p.tile_tokens, (long long)key - diag - tok + p.window_left + 1))) * p.group;
          if (kWin && hi == p.tile_tokens * p.group) hi = kCols;
        }
        const uint4 dead = *reinterpret_cast<const uint4*>(sm.dead[ring]);
        const bool masked = __any_sync(kAll, lo > 0 || hi < kCols) || (dead.x | dead.y | dead.z | dead.w) != 0u;
        float2 acc[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = make_float2(0.f, 0.f);
        uint32_t s[2][kChunk];
        load_scores(t_s, s[0]);
#pragma unroll
        for (int c = 0; c < kCols / kChunk; ++c) {
          wait_scores(s[c & 1]);
          if (c + 1 < kCols / kChunk) {
            load_scores(t_s + kChunk * (c + 1), s[(c + 1) & 1]);
          } else {
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.s_empty[b]);
          }
          const float* nl = sm.nl[ring] + kChunk * c;
          const uint32_t word = c < 2 ? dead.x : c < 4 ? dead.y : c < 6 ? dead.z : dead.w;
          if (masked)
            add_chunk<true, kCap>(s[c & 1], nl, lo - kChunk * c, hi - kChunk * c, word >> (kChunk * (c & 1)), p, acc);
          else
            add_chunk<false, kCap>(s[c & 1], nl, 0, 0, 0u, p, acc);
        }
        const float2 a = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
        sum += a.x + a.y;
      }
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
    mbar_init(&sm.k_full, 8);
    mbar_init(&sm.k_empty, 1);
    for (int i = 0; i < kQStages; ++i) {
      mbar_init(&sm.q_full[i], 33);  // the copy's issuer and the 32 writers of the -lse rows
      mbar_init(&sm.q_empty[i], 1);
    }
    for (int i = 0; i < kRing; ++i) mbar_init(&sm.l_full[i], 1);
    for (int i = 0; i < kSBufs; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.s_empty[i], 4);
    }
    sm.abort = 0;
    fence_mbar_init();
  }
  // rows of the Q stages that no copy fills, the -lse rows' zeros, the ones
  const int first = p.tile_tokens * p.group < kCols ? 0 : int(offsetof(TcSmem, l) / 16);
  for (int i = first + threadIdx.x; i < int(offsetof(TcSmem, ones) / 16); i += kTcThreads)
    reinterpret_cast<uint4*>(&sm)[i] = make_uint4(0, 0, 0, 0);
  for (int i = threadIdx.x; i < kQHalfBytes / 16; i += kTcThreads) {
    const int r = i >> 3, piece = (i & 7) ^ (r & 7);
    reinterpret_cast<uint4*>(sm.ones)[i] = piece == 0 ? make_uint4(0x3f803f80u, 0x00003f80u, 0, 0) : make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  if (warp == 16 && lane == 0) tc::tma_prefetch_desc(&tm_q);
  if (warp == 17) {
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
    if (warp < 8) {
      tc::regs_decrease<kSumRegs>();
      sum_weights<kWin, kCap>(p, sm, w, causal, tmem, line, ctas);
    } else if (warp < 16) {
      tc::regs_increase<kLoadRegs>();
      load_keys<kFp8>(p, sm, w, causal, tmem);
    } else {
      tc::regs_decrease<kControlRegs>();
      if (warp == 16)
        load_queries<kCap>(p, sm, w, causal, &tm_q);
      else if (warp == 17)
        issue<kCap>(p, sm, w, causal, tmem);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 17) {
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
