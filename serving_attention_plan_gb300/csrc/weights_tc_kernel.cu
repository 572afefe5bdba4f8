// Accumulated attention weights, tensor-core form: the same sums as the row form, for requests with many query
// rows (prompts and chunks; the limits and their measurements stand in cache_ops.h).
//
//   w_j = sum over query rows r (tokens x heads of the group) that see key j of exp2(scale2 q_r.k_j - lse2_r)
//
// A work item is 256 keys of one KV head against all query rows that see one of them, in Q tiles of 128
// rows (128 / g tokens x g heads, one TMA box a 64-dim half).  The item's keys stay in shared memory as
// the 256-column B operand; every Q tile is one 128 x 256 product.  Query rows are the accumulator's
// lanes: a thread's scores all belong to one row, whose -lse and mask bounds sit in registers, so a
// score costs one multiply-add, one exponential and one addition, into 64 running column sums a thread.
// There is no maximum, no second product, and lanes are added up once per item.
//   The other way round (keys on the lanes, one running sum a thread) needs the -lse of each column in
// every thread: read from shared memory it took as long as the exponentials, and as a further k-step of
// the product an eighth more tensor time.  Products of 128 columns measured 75 clocks a 16-dim step with the
// keys in tensor memory and 108 from shared memory (96 columns: 59 and 92), those of 256 columns 172:
// a 128 x 256 tile takes 1376 clocks this way, 1200 + the -lse step the other way.
//
// What bounds it: the products (1376 clocks a tile, above) beside 32768 exponentials (1024 clocks at 32 a
// clock and SM); both run at the same time, over two score buffers.  Measured: 1490-1640 clocks a tile, on four
// prompts of 1024 to 4096 tokens 123 us: 1.12 PFLOP/s of visible pairs (0.59 of the bf16 burst rate; tiles cut by the
// diagonal are computed whole).  A share of the exponentials by a polynomial on the multiply-add pipe made it slower
// (an eighth 145 us, a quarter 152, where none took 138).
//   e4m3: the key loader's widening does not fit its 64 registers (174 to 234 bytes spilled, in all e4m3 variants), and its
// loads come in eight rounds of four a lane and item; 128 requests of 128 rows take 776 us, 361 with bf16 pages.
//
// Work split: the Q tiles of all items lie on one line, request by request, KV head by KV head, key
// tile by key tile (the causal mask gives later key tiles fewer Q tiles); CTA c takes the c-th
// equal piece, so CTAs differ by one Q tile however ragged the batch is.  An item cut by a piece's
// border leaves its partial sums in a slot per CTA, and the last of its CTAs to finish adds them in
// line order: the result does not depend on who is last.  Each CTA has at most two cut items, so the
// slots are bounded by the grid, not by the batch.
//
// One CTA per SM, 20 warps:
//   warps 0-15   exponentials and sums: 4 warps (128 rows) for each 64 of the 256 keys
//   warps 16-17  key loader (two stages), any page size and layout: 16-byte asynchronous copies into the
//                128-byte swizzle; e4m3 codes are widened to bf16 (exact) on the way, so Q stays bf16
//   warp 18      TMA producer of Q tiles (three stages)
//   warp 19      tensor memory, MMA issue
#include <cuda.h>
#include <cudaTypedefs.h>
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
constexpr int kTcThreads = 640;
constexpr int kSumThreads = 512;
// Registers after launch (640 threads x 96): 512 x 104 + 128 x 64 = 640 x 96.
constexpr uint32_t kSumRegs = 104;
constexpr uint32_t kControlRegs = 64;
constexpr int kKeys = kTileKeys;                // keys of an item
constexpr int kRows = kWeightTileRows;          // query rows of a Q tile
constexpr int kCols = 64;                       // keys of a summing warp
constexpr int kLoadThreads = 64;
constexpr int kKHalfBytes = kKeys * 128;        // 64 dims of the item's keys
constexpr int kQHalfBytes = kRows * 128;        // 64 dims of a Q tile
constexpr int kQStages = 3;
constexpr int kKStages = 2;
constexpr int kSBufs = 2;                       // score buffers of 256 columns
constexpr uint32_t kTmemCols = 512;

// The CTA's walk over its piece of the line, one segment (run of Q tiles of one item) at a time.
// Every member is uniform over the warp; whole warps call init and next.
struct Walk {
  int win;               // the plan's sliding window: the line was cut with it
  int pos, end;          // remaining piece of the line
  int r, head, kt;       // request, KV head, key tile
  Geo g;
  int work1;             // line position behind this request
  int t0, cost;          // first query token that sees the item, its Q tiles (at least 1)
  int tokens;            // query tokens that see the item
  int q0, q1;            // Q tiles of this segment

  __device__ __forceinline__ void item(const WeightsParams& p, bool causal, const Geo& g, int kt, int& t0, int& tokens,
                                       int& cost) const {
    weight_item(g.lq, g.lkv, kt, causal, win, p.tile_tokens, &t0, &tokens, &cost);
  }
  __device__ __forceinline__ void load(const WeightsParams& p) {
    g = load_geo(p.pv.geo, r);
    work1 = __ldg(&p.pv.geo[r + 1].work0);
  }
  __device__ __forceinline__ void segment(const WeightsParams& p, bool causal) {
    item(p, causal, g, kt, t0, tokens, cost);
    q1 = min(cost, q0 + end - pos);
  }
  __device__ void init(const WeightsParams& p, const GeoHead& plan, int begin, int finish) {
    const bool causal = plan.causal != 0;
    const int lane = threadIdx.x & 31;
    win = plan.window;
    pos = begin;
    end = finish;
    if (pos >= end) return;
    r = find_request(p.pv.geo, plan.batch, &Geo::work0, pos);
    load(p);
    const int per_head = (work1 - g.work0) / p.pv.hkv;
    int rem = pos - g.work0;
    head = rem / per_head;
    rem -= head * per_head;
    // the key tile that holds position `rem` of the head's line: a scan over 32 tiles at a time
    int before = 0;
    for (kt = 0; kt * kKeys < g.lkv; kt += 32) {
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
  // Thread 0 of the summing warps: the segment at hand, written down.
  template <typename S>
  __device__ void publish(const WeightsParams& p, S& s) const {
    s.tiles = more() ? q1 - q0 : 0;
    if (!more()) return;
    const int tok = t0 + q0 * p.tile_tokens;
    s.pos = g.lkv - g.lq + tok - kt * kKeys;
    s.tokens = tokens - q0 * p.tile_tokens;
    s.lse = (long long)(g.q0 + tok) * p.hqo + head * p.group;
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

// What the summing warps keep of a segment, in shared memory: their registers hold the column sums.
struct Segment {
  int tiles;       // 0: no more
  int pos;         // key position of the first tile's first token, relative to the item's first key
  int tokens;      // query tokens from that one on
  long long lse;   // offset of the first token's first head
};

struct TcSmem {
  uint8_t k[kKStages][2 * kKHalfBytes];
  uint8_t q[kQStages][2 * kQHalfBytes];
  Walk walk;         // of the summing warps, one ahead of them
  Segment seg[2];    // what they know of a segment: the one at work and the next
  float red[2][kKeys];  // a segment's sums, added up over the four groups of 32 rows
  uint64_t k_full[kKStages], k_empty[kKStages], q_full[kQStages], q_empty[kQStages], s_full[kSBufs], s_empty[kSBufs];
  uint64_t red_full[2], red_empty[2];
  uint32_t tmem_base;
  int abort;
  int last;
};

// Four e4m3 codes -> four bf16 (exact: e4m3 values have 4 significant bits and small exponents).
__device__ __forceinline__ uint2 widen4(uint32_t codes) {
  const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes & 0xffffu), __NV_E4M3);
  const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes >> 16), __NV_E4M3);
  const float2 a = __half22float2(__half2(lo)), b = __half22float2(__half2(hi));
  return make_uint2(f2_to_bf16x2(a.x, a.y), f2_to_bf16x2(b.x, b.y));
}

// Writes a finished segment's sums out (the key loader's threads, four keys each).  Of a cut item each
// piece goes to its slot, and the last of its CTAs to come adds all of them in line order.  After a wait
// that gave up (the error is recorded) nothing is written, but the barriers and counts go their way.
__device__ void write_sums(const WeightsParams& p, TcSmem& sm, const Walk& w, int n, int line, int ctas, bool& alive) {
  const PageView& pv = p.pv;
  const int tid = threadIdx.x - kSumThreads;
  constexpr int kMine = kKeys / kLoadThreads;
  float sum[kMine], old[kMine];
  float* out[kMine];
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int key = w.kt * kKeys + tid + i * kLoadThreads;
    int page, slot;
    out[i] = nullptr;
    old[i] = 0.f;
    if (key < w.g.lkv && locate(pv, w.g.kv0, key, page, slot)) {
      out[i] = p.weights + weight_offset(pv, page, slot, w.head);
      if (!(p.new_keys && key >= w.g.lkv - w.g.lq) && p.decay != 0.f) old[i] = p.decay * __ldcg(out[i]);
    }
  }
  alive = alive && __all_sync(kAll, mbar_wait(&sm.red_full[n & 1], (n >> 1) & 1, pv.err, &sm.abort));
#pragma unroll
  for (int i = 0; i < kMine; ++i) sum[i] = sm.red[n & 1][tid + i * kLoadThreads];
  mbar_arrive(&sm.red_empty[n & 1]);
  if (w.q0 != 0 || w.q1 != w.cost) {
    const int start = w.pos - w.q0;
    const int c1 = int(((long long)(start + 1) * ctas - 1) / line), c2 = int(((long long)(start + w.cost) * ctas - 1) / line);
    float* piece = p.part + (size_t(blockIdx.x) * 2 + (w.q0 == 0 ? 1 : 0)) * kKeys + tid;
#pragma unroll
    for (int i = 0; i < kMine; ++i) piece[i * kLoadThreads] = sum[i];
    __threadfence();
    named_bar_sync(2, kLoadThreads);
    if (tid == 0) sm.last = atomicAdd(p.part_count + c1, 1u) == unsigned(c2 - c1);
    named_bar_sync(2, kLoadThreads);
    if (!sm.last) return;
    __threadfence();
#pragma unroll
    for (int i = 0; i < kMine; ++i) sum[i] = 0.f;
    for (int c = c1; c <= c2; ++c) {
      const float* at = p.part + (size_t(c) * 2 + (c == c1 ? 1 : 0)) * kKeys + tid;
#pragma unroll
      for (int i = 0; i < kMine; ++i) sum[i] += __ldcg(at + i * kLoadThreads);
    }
    if (tid == 0) p.part_count[c1] = 0;
  }
  if (!alive) return;
#pragma unroll
  for (int i = 0; i < kMine; ++i)
    if (out[i] != nullptr) *out[i] = old[i] + sum[i];
}

template <bool kFp8>
__device__ void load_keys(const WeightsParams& p, TcSmem& sm, Walk w, bool causal, int line, int ctas) {
  const PageView& pv = p.pv;
  const int lane = threadIdx.x & 31;
  constexpr int kLanes = kFp8 ? 8 : 16;           // lanes of a row, 16 bytes each
  constexpr int kRowsPass = 32 / kLanes;          // rows of a warp's pass
  constexpr int kMine = kKeys / kLoadThreads;     // rows a lane looks up
  const int first = (threadIdx.x - kSumThreads) / 32 * (kKeys / 2);  // this warp's half of the rows
  const int ch = lane % kLanes, sub = lane / kLanes;
  const uint8_t* pages = static_cast<const uint8_t*>(p.k_pages);
  Walk done = w;  // the segment whose sums are written out next
  int written = 0;
  bool alive = true;
  for (int n = 0; w.more(); w.next(p, causal), ++n) {
    const int ks = n % kKStages;
    if (n >= kKStages)
      alive = alive && __all_sync(kAll, mbar_wait(&sm.k_empty[ks], (n / kKStages - 1) & 1, pv.err, &sm.abort));
    auto place = [&](int row, int c16) {  // 16-byte piece c16 (0..15) of a bf16 row
      return sm.k[ks] + (c16 >> 3) * kKHalfBytes + row * 128 + (((c16 & 7) ^ (row & 7)) << 4);
    };
    if (alive) {
      // each lane looks up four rows (one memory latency for all 256), the passes below fetch them by shuffle
      int at[kMine];  // row of the page pool (128 elements each), -1: no key
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int key = w.kt * kKeys + first + lane + 32 * i;
        int page, slot;
        at[i] = -1;
        if (key < w.g.lkv && locate(pv, w.g.kv0, key, page, slot))
          at[i] = int(kv_offset(pv, page, slot, w.head) / kHeadDim);
      }
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        constexpr int kBatch = kFp8 ? 8 : 16;  // passes of 32 rows: 8 with e4m3 codes, 16 without
#pragma unroll
        for (int k0 = 0; k0 < kBatch; k0 += 4) {
          uint4 v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r = (k0 + k) * kRowsPass + sub, row = first + 32 * i + r;
            const int src = __shfl_sync(kAll, at[i], r);
            const uint8_t* from = pages + (long long)src * (kHeadDim * (kFp8 ? 1 : 2)) + 16 * ch;
            if constexpr (kFp8) {
              v[k] = src >= 0 ? __ldg(reinterpret_cast<const uint4*>(from)) : make_uint4(0, 0, 0, 0);
            } else {
              if (src >= 0)
                cp_async_16(place(row, ch), from);
              else
                *reinterpret_cast<uint4*>(place(row, ch)) = make_uint4(0, 0, 0, 0);
            }
          }
          if constexpr (kFp8) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int row = first + 32 * i + (k0 + k) * kRowsPass + sub;
              const uint2 a = widen4(v[k].x), b = widen4(v[k].y), c = widen4(v[k].z), d = widen4(v[k].w);
              *reinterpret_cast<uint4*>(place(row, 2 * ch)) = make_uint4(a.x, a.y, b.x, b.y);
              *reinterpret_cast<uint4*>(place(row, 2 * ch + 1)) = make_uint4(c.x, c.y, d.x, d.y);
            }
          }
        }
      }
    }
    cp_async_wait_all();
    fence_proxy_async_smem();
    if (alive) mbar_arrive(&sm.k_full[ks]);
    // k_empty says that segment n - 2's products are done: its sums are near.  (Written out before the wait for the
    // copies, they held the next keys up: 383 against 338 us for 128 requests of 16 tokens.)
    if (n >= kKStages) {
      write_sums(p, sm, done, written++, line, ctas, alive);
      done.next(p, causal);
    }
  }
  for (; done.more(); done.next(p, causal)) write_sums(p, sm, done, written++, line, ctas, alive);
}

__device__ void load_queries(const WeightsParams& p, TcSmem& sm, Walk w, bool causal, const CUtensorMap* tm_q) {
  const uint32_t bytes = uint32_t(2 * 128 * p.tile_tokens * p.group);
  int n = 0;
  bool ok = true;
  for (; ok && w.more(); w.next(p, causal)) {
    for (int qt = w.q0; qt < w.q1; ++qt, ++n) {
      const int qs = n % kQStages;
      if (n >= kQStages) ok = mbar_wait(&sm.q_empty[qs], (n / kQStages - 1) & 1, p.pv.err, &sm.abort);
      if (!ok) break;
      mbar_arrive_expect_tx(&sm.q_full[qs], bytes);
      const int tok0 = w.g.q0 + w.t0 + qt * p.tile_tokens;
      tc::tma_load_3d(sm.q[qs], tm_q, 0, w.head * p.group, tok0, &sm.q_full[qs]);
      tc::tma_load_3d(sm.q[qs] + kQHalfBytes, tm_q, 64, w.head * p.group, tok0, &sm.q_full[qs]);
    }
  }
  // never leave with tensor copies still landing in this CTA's shared memory
  for (int k = max(0, n - kQStages); k < n; ++k) mbar_wait_bounded(&sm.q_full[k % kQStages], (k / kQStages) & 1);
}

// One lane of the warp, the same each time; the branch on it keeps the warp's control flow uniform, so
// descriptors stay in uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t on;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(on));
  return on != 0;
}

// Issues the products, one thread of a warp that walks together (issued from a branch on the lane number a
// product took 131 clocks of its thread, whatever its size).  The descriptors of a stage are the first
// stage's plus an address step in 16-byte units.
__device__ void issue(const WeightsParams& p, TcSmem& sm, Walk w, bool causal, uint32_t tmem) {
  constexpr uint32_t idesc = tc::idesc_bf16_f32(kRows, kKeys, 0, 0);  // A = query rows, B = keys, both K-major
  const uint64_t q_desc = tc::smem_desc(smem_u32(sm.q[0]), 16, 1024, tc::kLayoutSw128);
  const uint64_t k_desc = tc::smem_desc(smem_u32(sm.k[0]), 16, 1024, tc::kLayoutSw128);
  int n = 0;
  for (int seg = 0; w.more(); w.next(p, causal), ++seg) {
    const int ks = seg % kKStages;
    if (!__all_sync(kAll, mbar_wait(&sm.k_full[ks], (seg / kKStages) & 1, p.pv.err, &sm.abort))) return;
    const uint64_t kd = k_desc + uint64_t(ks * (2 * kKHalfBytes / 16));
    for (int qt = w.q0; qt < w.q1; ++qt, ++n) {
      const int qs = n % kQStages, b = n % kSBufs;
      if (!__all_sync(kAll, mbar_wait(&sm.q_full[qs], (n / kQStages) & 1, p.pv.err, &sm.abort))) return;
      if (n >= kSBufs && !__all_sync(kAll, mbar_wait(&sm.s_empty[b], (n / kSBufs - 1) & 1, p.pv.err, &sm.abort))) return;
      tc::fence_after_sync();
      const uint64_t qd = q_desc + uint64_t(qs * (2 * kQHalfBytes / 16));
      if (elect_one()) {
        const uint32_t d = tmem + uint32_t(b * kKeys);
#pragma unroll
        for (int k = 0; k < 8; ++k)  // 16 dims: 32 bytes of the swizzled rows
          tc::mma_ss(d, qd + uint64_t(((k >> 2) * kQHalfBytes + (k & 3) * 32) / 16),
                     kd + uint64_t(((k >> 2) * kKHalfBytes + (k & 3) * 32) / 16), idesc, k != 0 ? 1u : 0u);
        tc::commit(&sm.s_full[b]);
        tc::commit(&sm.q_empty[qs]);
      }
      __syncwarp();
    }
    if (elect_one()) tc::commit(&sm.k_empty[ks]);
    __syncwarp();
  }
}

constexpr int kChunk = 8;  // scores a thread loads at a time; the next chunk is in flight meanwhile
__device__ __forceinline__ void load_scores(uint32_t taddr, uint32_t (&r)[kChunk]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
// Waits for the tensor-memory loads in flight.  The registers pass through, so that nothing that uses
// them can be scheduled before the wait.
__device__ __forceinline__ void wait_scores(uint32_t (&r)[kChunk]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])::"memory");
}

// The soft-cap's tanh takes two of the three special-function results of a score, and that pipe bounds it,
// so it comes two ways, a quarter of the scores the first and the others the second (measured on 509 new
// tokens over 16 K keys: all by the first 249 us, half 190, a quarter 182, none 188):
//   1 - 2 / (1 + 2^(2 y log2 e)), absolute error 1.5e-7 (the hardware's exponential and reciprocal);
//   y P(y^2) on the multiply-add pipe, P of degree 4 fitted to tanh(y) / y for |y| <= 0.6 so that the largest
//   error of y P is least: 2e-8, 7e-8 in fp32.  A warp with a larger |y| among them takes the first way.
__device__ __forceinline__ float2 tanh2_exp(float2 y) {
  const float2 e = __fmul2_rn(y, make_float2(2.f * kLog2e, 2.f * kLog2e));
  const float2 d = __fadd2_rn(make_float2(fast_exp2(e.x), fast_exp2(e.y)), make_float2(1.f, 1.f));
  float2 r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(d.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(d.y));
  return __ffma2_rn(r, make_float2(-2.f, -2.f), make_float2(1.f, 1.f));
}
constexpr float kPolyReach = 0.36f;  // of y^2
constexpr int kPolyPairs = 3;        // of a chunk's 4 pairs
__device__ __forceinline__ float2 tanh2_poly(float2 y, float2 u) {
  constexpr float c[5] = {0.99999964f, -0.3333121f, 0.1329921f, -0.05169674f, 0.014976956f};
  float2 t = make_float2(c[4], c[4]);
#pragma unroll
  for (int i = 3; i >= 0; --i) t = __ffma2_rn(t, u, make_float2(c[i], c[i]));
  return __fmul2_rn(t, y);
}

// Soft-cap of a kernel: none, the two ways above, or a cap so large that their absolute error would show
// (kExpTanhMostCap), where every score takes the series or the exponentials by its own |y|.
enum Cap { kCapNone = 0, kCapMixed, kCapWide };
__device__ __forceinline__ float2 tanh2_wide(float2 y) {
  const float2 u = __fmul2_rn(y, y), near = __fmul2_rn(tanh_near_factor(u), y), far = tanh2_exp(y);
  return make_float2(u.x <= kNearReach ? near.x : far.x, u.y <= kNearReach ? near.y : far.y);
}

// A chunk of the row's scores -> added to the column sums.  With kMasked, columns outside [lo, hi) get
// nothing whatever their score is.
template <bool kMasked, int kCap>
__device__ __forceinline__ void add_chunk(const uint32_t (&s)[kChunk], float nl, int lo, int hi, const WeightsParams& p,
                                          float2* acc) {
  float2 th[kChunk / 2];
  if constexpr (kCap == kCapWide) {
    const float in = p.scale_log2 * p.inv_cap_log2;
    float2 y[kChunk / 2];
    float far = 0.f;
#pragma unroll
    for (int i = 0; i < kChunk / 2; ++i) {
      y[i] = __fmul2_rn(make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), make_float2(in, in));
      far = fmaxf(far, fmaxf(fabsf(y[i].x), fabsf(y[i].y)));
    }
    // (a NaN passes fmaxf by and goes through the series as a NaN)
    if (!__any_sync(kAll, far * far > kNearReach)) {
#pragma unroll
      for (int i = 0; i < kChunk / 2; ++i) th[i] = __fmul2_rn(tanh_near_factor(__fmul2_rn(y[i], y[i])), y[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kChunk / 2; ++i) th[i] = tanh2_wide(y[i]);
    }
  } else if constexpr (kCap == kCapMixed) {
    const float in = p.scale_log2 * p.inv_cap_log2;
    float2 y[kChunk / 2], u[kPolyPairs];
#pragma unroll
    for (int i = 0; i < kChunk / 2; ++i)
      y[i] = __fmul2_rn(make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), make_float2(in, in));
    float far = 0.f;
#pragma unroll
    for (int i = 0; i < kPolyPairs; ++i) {
      u[i] = __fmul2_rn(y[i], y[i]);
      far = fmaxf(far, fmaxf(u[i].x, u[i].y));
    }
    const bool poly = !__any_sync(kAll, far > kPolyReach);
#pragma unroll
    for (int i = kPolyPairs; i < kChunk / 2; ++i) th[i] = tanh2_exp(y[i]);
    if (poly) {
#pragma unroll
      for (int i = 0; i < kPolyPairs; ++i) th[i] = tanh2_poly(y[i], u[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kPolyPairs; ++i) th[i] = tanh2_exp(y[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < kChunk / 2; ++i) {
    float2 x = make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1]));
    if constexpr (kCap != kCapNone) {
      x = __ffma2_rn(th[i], make_float2(p.cap_log2, p.cap_log2), make_float2(nl, nl));
    } else {
      x = __ffma2_rn(x, make_float2(p.scale_log2, p.scale_log2), make_float2(nl, nl));
    }
    if constexpr (kMasked) {
      if (2 * i < lo || 2 * i >= hi) x.x = -INFINITY;
      if (2 * i + 1 < lo || 2 * i + 1 >= hi) x.y = -INFINITY;
    }
    acc[i] = __fadd2_rn(acc[i], make_float2(fast_exp2(x.x), fast_exp2(x.y)));
  }
}

// The row's 64 scores of a tile.
template <bool kMasked, int kCap>
__device__ __forceinline__ void add_tile(uint32_t t_s, float nl, int lo, int hi, const WeightsParams& p, uint64_t* s_empty,
                                         float2 (&acc)[kCols / 2]) {
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
      if ((threadIdx.x & 31) == 0) mbar_arrive(s_empty);
    }
    add_chunk<kMasked, kCap>(s[c & 1], nl, lo - kChunk * c, hi - kChunk * c, p, acc + c * (kChunk / 2));
  }
}

template <bool kWin, int kCap>
__device__ void sum_weights(const WeightsParams& p, TcSmem& sm, bool causal, uint32_t tmem) {
  const PageView& pv = p.pv;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = threadIdx.x & (kRows - 1);   // query row of the tile: TMEM lane
  const int col0 = (warp >> 2) * kCols;        // first key of this warp
  const uint32_t t_lane = tmem + (uint32_t((warp & 3) * 32) << 16) + uint32_t(col0);
  const int win = sm.walk.win;
  int n = 0;
  bool alive = true;
  for (int i = 0; sm.seg[i & 1].tiles > 0; ++i) {
    const Segment g = sm.seg[i & 1];
    named_bar_sync(1, kSumThreads);  // all have read it, and what the one after it overwrites
    if (threadIdx.x == 0) {  // the next segment; its readers come to it after the barriers below
      sm.walk.next(p, causal);
      sm.walk.publish(p, sm.seg[(i + 1) & 1]);
    }
    __syncwarp();
    float2 acc[kCols / 2];
#pragma unroll
    for (int k = 0; k < kCols / 2; ++k) acc[k] = make_float2(0.f, 0.f);
    const int my_tok = row / p.group;
    int pos = g.pos + my_tok - col0;                                     // the row sees columns up to this one
    int left = my_tok < p.tile_tokens ? g.tokens - my_tok : 0;           // rows from here on, in tokens
    const float* lse_at = p.lse + g.lse + (long long)my_tok * p.hqo + (row - my_tok * p.group);
    // lse of the thread's row in the next tile, -inf where there is none.  Nothing looks at it before the
    // next tile: a use here would wait for the load (600 clocks a tile).
    float lse = -INFINITY;
    if (left > 0) lse = __ldg(lse_at);
    const int n_end = n + g.tiles;
    for (; n < n_end; ++n) {
      const int b = n % kSBufs;
      const float nl = -kLog2e * lse;
      int lo = 0, hi = kCols;  // the columns the row sees
      if (causal) {
        hi = min(kCols, pos + 1);
        if (kWin && win >= 0) lo = max(0, pos - win);
      }
      if (lse == -INFINITY) hi = 0;  // no such row, or one that saw no key
      const bool masked = __any_sync(kAll, lo > 0 || hi < kCols);
      pos += p.tile_tokens;
      left -= p.tile_tokens;
      lse_at += (long long)p.tile_tokens * p.hqo;
      lse = -INFINITY;
      if (n + 1 < n_end && left > 0) lse = __ldg(lse_at);
      alive = alive && __all_sync(kAll, mbar_wait(&sm.s_full[b], (n / kSBufs) & 1, pv.err, &sm.abort));
      if (alive) {
        tc::fence_after_sync();
        const uint32_t t_s = t_lane + uint32_t(b * kKeys);
        if (masked)
          add_tile<true, kCap>(t_s, nl, lo, hi, p, &sm.s_empty[b], acc);
        else
          add_tile<false, kCap>(t_s, nl, 0, kCols, p, &sm.s_empty[b], acc);
      }
    }
    // 64 column sums in each of 32 lanes -> two in each: at every step a lane keeps one half of its columns
    // and gives the other to its partner
    float* v = reinterpret_cast<float*>(acc);
#pragma unroll
    for (int m = 0; m < 5; ++m) {
      const int half = kCols >> (m + 1);
      const bool up = (lane >> (4 - m)) & 1;
#pragma unroll
      for (int k = 0; k < half; ++k) {
        const float give = up ? v[k] : v[k + half], keep = up ? v[k + half] : v[k];
        v[k] = keep + __shfl_xor_sync(kAll, give, 16 >> m);
      }
    }
    // lane l now holds columns 2 l and 2 l + 1; the four groups of rows add theirs in turn
    if (i >= 2) alive = alive && __all_sync(kAll, mbar_wait(&sm.red_empty[i & 1], ((i >> 1) - 1) & 1, pv.err, &sm.abort));
#pragma unroll 1
    for (int k = 0; k < 4; ++k) {
      if ((warp & 3) == k) {
        float2* at = reinterpret_cast<float2*>(sm.red[i & 1] + col0) + lane;
        *at = k == 0 ? make_float2(v[0], v[1]) : __fadd2_rn(*at, make_float2(v[0], v[1]));
      }
      named_bar_sync(1, kSumThreads);
    }
    if (alive && threadIdx.x == 0) mbar_arrive(&sm.red_full[i & 1]);
  }
}

template <bool kFp8, bool kWin, int kCap>
__global__ void __launch_bounds__(kTcThreads, 1)
    weights_tc_kernel(const __grid_constant__ WeightsParams p, const __grid_constant__ CUtensorMap tm_q) {
  // the kernel has no static shared memory, so this starts at the CTA's first (1024-byte aligned) address;
  // the check below holds it to that, the swizzled tiles need it
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  TcSmem& sm = *reinterpret_cast<TcSmem*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(&sm.k_full[i], kLoadThreads);
      mbar_init(&sm.k_empty[i], 1);
    }
    for (int i = 0; i < kQStages; ++i) {
      mbar_init(&sm.q_full[i], 1);
      mbar_init(&sm.q_empty[i], 1);
    }
    for (int i = 0; i < kSBufs; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.s_empty[i], kSumThreads / 32);
      mbar_init(&sm.red_full[i], 1);
      mbar_init(&sm.red_empty[i], kLoadThreads);
    }
    sm.abort = 0;
    fence_mbar_init();
  }
  if (p.tile_tokens * p.group < kRows) {  // rows of the Q stages that no copy fills
    for (int i = threadIdx.x; i < int(sizeof(sm.q) / 16); i += kTcThreads)
      reinterpret_cast<uint4*>(sm.q[0])[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  if (warp == 18 && lane == 0) tc::tma_prefetch_desc(&tm_q);
  if (warp == 19) {
    tc::tmem_alloc(&sm.tmem_base, kTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  wait_prior_grid();
  const uint32_t tmem = sm.tmem_base;
  const GeoHead plan = load_head(p.pv.geo);
  const bool causal = plan.causal != 0;
  const int line = plan.work;
  const int ctas = min(int(gridDim.x), line);
  if ((tmem & 0xFFFFu) + kTmemCols > 512u || (smem_u32(smem_raw) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicOr(p.pv.err, FI_DEVERR_TMEM);
  } else if (int(blockIdx.x) < ctas) {
    Walk w;
    w.init(p, plan, int((long long)line * blockIdx.x / ctas), int((long long)line * (blockIdx.x + 1) / ctas));
    if (warp < 16) {
      if (threadIdx.x == 0) {
        sm.walk = w;
        w.publish(p, sm.seg[0]);
      }
      named_bar_sync(1, kSumThreads);
      tc::regs_increase<kSumRegs>();
      sum_weights<kWin, kCap>(p, sm, causal, tmem);
    } else {
      tc::regs_decrease<kControlRegs>();
      if (warp < 18)
        load_keys<kFp8>(p, sm, w, causal, line, ctas);
      else if (warp == 18 && lane == 0)
        load_queries(p, sm, w, causal, &tm_q);
      else if (warp == 19)
        issue(p, sm, w, causal, tmem);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 19) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

// Tensor map of the queries [total_q][hqo][128] for tiles of `tokens` tokens x `heads` heads: a box is
// 64 dims of tokens * heads rows, token by token, 128-byte swizzled.  Rows behind total_q read as zeros.
// Returns false if the driver's encoder is missing or refuses the map.
bool make_query_map(CUtensorMap* m, const void* q, int hqo, int total_q, int heads, int tokens) {
  static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) == cudaSuccess &&
        found == cudaDriverEntryPointSuccess)
      encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  if (encode == nullptr) return false;
  const cuuint64_t row = cuuint64_t(kHeadDim) * 2;
  const cuuint64_t dims[3] = {cuuint64_t(kHeadDim), cuuint64_t(hqo), cuuint64_t(total_q)}, strides[2] = {row, row * hqo};
  const cuuint32_t box[3] = {64u, cuuint32_t(heads), cuuint32_t(tokens)}, step[3] = {1u, 1u, 1u};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

int launch_weights_tc(const WeightsParams& p, int total_q, bool fp8, int num_sms, cudaStream_t stream) {
  CUtensorMap tq;
  if (!make_query_map(&tq, p.q, p.hqo, total_q, p.group, p.tile_tokens)) return FI_ERR_INVALID_ARG;
  constexpr size_t smem = sizeof(TcSmem);
  static_assert(smem <= 227 * 1024, "shared memory exceeds the per-CTA limit");
  static_assert(kSBufs * kKeys <= int(kTmemCols) && kKeys == 4 * kCols, "score buffers, columns of the summing warps");
  using Kernel = void (*)(const WeightsParams, const CUtensorMap);
  static const Kernel kernels[12] = {
      weights_tc_kernel<false, false, kCapNone>, weights_tc_kernel<false, false, kCapMixed>, weights_tc_kernel<false, false, kCapWide>,
      weights_tc_kernel<false, true, kCapNone>,  weights_tc_kernel<false, true, kCapMixed>,  weights_tc_kernel<false, true, kCapWide>,
      weights_tc_kernel<true, false, kCapNone>,  weights_tc_kernel<true, false, kCapMixed>,  weights_tc_kernel<true, false, kCapWide>,
      weights_tc_kernel<true, true, kCapNone>,   weights_tc_kernel<true, true, kCapMixed>,   weights_tc_kernel<true, true, kCapWide>};
  static std::once_flag once;
  static cudaError_t attr = cudaSuccess;
  std::call_once(once, [] {
    for (int i = 0; i < 12 && attr == cudaSuccess; ++i)
      attr = cudaFuncSetAttribute(kernels[i], cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  });
  if (attr != cudaSuccess) return record_cuda_error(attr, "cudaFuncSetAttribute(weights_tc_kernel)");
  const int cap = p.cap_log2 > 0.f ? (p.wide_cap ? kCapWide : kCapMixed) : kCapNone;
  const Kernel k = kernels[(fp8 ? 6 : 0) + (p.window_left >= 0 ? 3 : 0) + cap];
  const cudaError_t e = launch_dependent(k, unsigned(num_sms), kTcThreads, smem, 1, stream, p, tq);
  return e == cudaSuccess ? 0 : record_cuda_error(e, "weights_tc_kernel launch");
}

}  // namespace fi
