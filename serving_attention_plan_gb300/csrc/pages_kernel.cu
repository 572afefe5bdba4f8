// Attention over pages that a cheap score selects: bounds of the keys of a page, the pages' scores for each query, the
// choice under a budget, and the work plan of the attention over the chosen pages.
#include <cuda_fp8.h>

#include <algorithm>

#include "cache_common.cuh"
#include "prefill_launch.h"
#include "tree_ops.h"

namespace fi {
namespace {

constexpr unsigned kAll = 0xffffffffu;

// The kernels below read the plan before wait_prior_grid: it was there before the kernel that they wait for, which a copy of the plan
// cannot lie behind.  What an earlier kernel may have written is read behind the wait, and every CTA waits, those without
// work too: a grid that ended before the one it depends on would let its own followers start.

// Last request r whose value of(r) (non-decreasing) is <= x, of(0) <= x; a whole warp, 32 probes a round.
template <typename F>
__device__ __forceinline__ int last_at_most(int n, int x, F of) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) >> 5;
    const int at = lo + lane * step;
    const unsigned le = __ballot_sync(kAll, at < hi && of(min(at, n - 1)) <= x);
    lo += (__popc(le) - 1) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

__device__ __forceinline__ int pages_of(const PageView& pv, int keys) {
  return pv.page_shift >= 0 ? (keys + pv.page_size - 1) >> pv.page_shift : (keys + pv.page_size - 1) / pv.page_size;
}

// The request of query token t < total_q.  In a decode batch that is entry t itself, so it is looked at first; a whole warp calls.
__device__ __forceinline__ Geo request_of(const Geo* geo, int batch, int t, int& r) {
  r = min(t, batch - 1);
  Geo g = load_geo(geo, r);
  if (t < g.q0 || t >= g.q0 + g.lq) {
    r = find_request(geo, batch, &Geo::q0, t);
    g = load_geo(geo, r);
  }
  return g;
}

// ---- bounds ------------------------------------------------------------------------------------------
//   bounds[page][head][0][d] = min, [1][d] = max over the page's keys of K[key][d]   (e4m3: of the codes' values)
// NaN wins, so that a page with a NaN key ranks first and its attention shows it.  Exact: a minimum is one of its inputs, and every
// e4m3 value is a bf16 value.  The keys are read once, 512 bytes a page and head are written: traffic is the bound.  A warp
// takes one (page, head) at a time, 16 bytes a lane and load, up to eight loads in flight, compared two by two in
// their 16-bit form.

__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b, bool f16) {
  uint32_t r;
  if (f16)
    asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b, bool f16) {
  uint32_t r;
  if (f16)
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t widen2(uint32_t two_codes) {
  uint32_t h;
  const uint16_t v = static_cast<uint16_t>(two_codes);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(v));
  return h;
}
__device__ __forceinline__ uint32_t f16x2_to_bf16x2(uint32_t h) {
  const __half2 v = *reinterpret_cast<const __half2*>(&h);
  const float2 f = __half22float2(v);
  return f2_to_bf16x2(f.x, f.y);
}

constexpr int kBoundsThreads = 256;
constexpr int kBoundsAhead = 8;

// One step: up to kBoundsAhead loads of a (page, head), which takes more than one if its page is long.
struct BoundsStep {
  int page, keys, head, k0;  // page -1: nothing to read
};

// Words of two dims that a lane holds: 4 of bf16, or 8 of f16 (16 codes).  The loads of a step are under way while the one before it
// is compared (13 prompts of 8 to 36 K keys, 610 MB: 116 -> 97 us, 0.94 of the copy bandwidth).
template <bool kFp8>
__global__ void __launch_bounds__(kBoundsThreads) bounds_kernel(const __grid_constant__ BoundsParams p) {
  constexpr int kLanes = kFp8 ? 8 : 16, kSide = 32 / kLanes, kWords = kFp8 ? 8 : 4, kRowsStep = kBoundsAhead * kSide;
  const PageView& pv = p.pv;
  const GeoHead plan = load_head(pv.geo);
  if (plan.batch == 0) return wait_prior_grid();
  const int lane = threadIdx.x & 31, sub = lane % kLanes, side = lane / kLanes;
  // a task is a page entry (or, for new keys, a query token) and a head; heads of a page are neighbours in memory
  const long long units = p.new_keys ? plan.total_q : __ldg(&pv.geo[plan.batch].kv0);
  const long long tasks = units * pv.hkv, warps = (long long)gridDim.x * (kBoundsThreads / 32);
  const long long me = (long long)blockIdx.x * (kBoundsThreads / 32) + (threadIdx.x >> 5);
  const long long t0 = tasks * me / warps, t1 = tasks * (me + 1) / warps;
  if (t0 >= t1) return wait_prior_grid();
  int unit = int(t0 / pv.hkv);
  long long task = t0;
  int r = p.new_keys ? 0 : find_request(pv.geo, plan.batch, &Geo::kv0, unit);
  Geo g = p.new_keys ? request_of(pv.geo, plan.batch, unit, r) : load_geo(pv.geo, r);
  BoundsStep next = {-1, 0, int(t0 - (long long)unit * pv.hkv), 0};
  auto look_up = [&]() {  // the page of `unit`
    int e;
    next.page = -1;
    next.keys = 0;
    if (p.new_keys) {
      while (unit >= g.q0 + g.lq) g = load_geo(pv.geo, ++r);
      const int t = unit - g.q0, j = g.lkv - g.lq + t;
      // the first new token of its page speaks for the page
      const bool first = j >= 0 && (t == 0 || j == 0 || j % pv.page_size == 0);
      e = first ? j / pv.page_size : -1;
    } else {
      while (unit >= g.kv0 + pages_of(pv, g.lkv)) g = load_geo(pv.geo, ++r);
      e = unit - g.kv0;
    }
    if (e < 0) return;
    next.keys = min(pv.page_size, g.lkv - e * pv.page_size);
    next.page = __ldg(pv.kv_indices + g.kv0 + e);
    if (static_cast<unsigned>(next.page) >= static_cast<unsigned>(pv.num_pages)) {
      atomicOr(pv.err, FI_DEVERR_PAGE_OOB);
      next.page = -1;
    }
  };
  auto advance = [&]() {  // to the step after `next`; false behind the last
    if (next.page >= 0 && next.k0 + kRowsStep < next.keys) {
      next.k0 += kRowsStep;
      return true;
    }
    next.k0 = 0;
    if (++task >= t1) return false;
    if (++next.head == pv.hkv) {
      next.head = 0;
      ++unit;
      look_up();
    }
    return true;
  };
  const long long step = pv.tok_stride * (kFp8 ? 1 : 2);
  auto fetch = [&](uint4 (&x)[kBoundsAhead]) {
    if (next.page < 0) return;
    const char* src = static_cast<const char*>(p.k_pages) + kv_offset(pv, next.page, 0, next.head) * (kFp8 ? 1 : 2) + sub * 16;
#pragma unroll
    for (int i = 0; i < kBoundsAhead; ++i)  // a row behind the last key stands for the last
      if (next.k0 + i * kSide < next.keys)
        x[i] = __ldcs(reinterpret_cast<const uint4*>(src + min(next.k0 + i * kSide + side, next.keys - 1) * step));
  };
  uint4 x[2][kBoundsAhead];
  uint32_t lo[kWords], hi[kWords];
  look_up();
  wait_prior_grid();
  fetch(x[0]);
  bool more = true;
  auto turn = [&](uint4 (&now)[kBoundsAhead], uint4 (&ahead)[kBoundsAhead]) {
    const BoundsStep c = next;
    more = advance();
    if (more) fetch(ahead);
    if (c.page < 0) return;
#pragma unroll
    for (int i = 0; i < kBoundsAhead; ++i) {
      if (c.k0 + i * kSide >= c.keys) break;
      const uint32_t w[4] = {now[i].x, now[i].y, now[i].z, now[i].w};
#pragma unroll
      for (int k = 0; k < kWords; ++k) {
        const uint32_t v = kFp8 ? widen2(k & 1 ? w[k / 2] >> 16 : w[k / 2]) : w[k & 3];
        lo[k] = c.k0 > 0 || i > 0 ? min2(lo[k], v, kFp8) : v;
        hi[k] = c.k0 > 0 || i > 0 ? max2(hi[k], v, kFp8) : v;
      }
    }
    if (c.k0 + kRowsStep < c.keys) return;
#pragma unroll
    for (int m = kLanes; m < 32; m <<= 1) {
#pragma unroll
      for (int k = 0; k < kWords; ++k) {
        lo[k] = min2(lo[k], __shfl_xor_sync(kAll, lo[k], m), kFp8);
        hi[k] = max2(hi[k], __shfl_xor_sync(kAll, hi[k], m), kFp8);
      }
    }
    uint4* to = reinterpret_cast<uint4*>(p.bounds + ((long long)c.page * pv.hkv + c.head) * 2 * kHeadDim);
    if constexpr (kFp8) {  // the row's four lanes of a sub take a half of its 16 minima or maxima each
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t a = side & 1 ? lo[4 + k] : lo[k], b = side & 1 ? hi[4 + k] : hi[k];
        w[k] = f16x2_to_bf16x2(side & 2 ? b : a);
      }
      to[(side >> 1) * 16 + sub * 2 + (side & 1)] = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      to[side * 16 + sub] = side ? make_uint4(hi[0], hi[1], hi[2], hi[3]) : make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
  };
  while (more) {
    turn(x[0], x[1]);
    if (more) turn(x[1], x[0]);
  }
}

// ---- scores --------------------------------------------------------------------------------------------
//   score(t, h, e) = scale * max over the query heads of h's group of  sum_d  min(q_d, 0) lo_d + max(q_d, 0) hi_d
// no less than the logit of any key of page e; -inf for a page that token t does not see.  The sum is a product of 256 terms
// whose one factor [lo, hi] is the page's row as it lies in memory, so it runs on warp-level products: 16 pages on the rows,
// eight (token, head) columns.  Sums are fp32.  Reading the bounds once is the bound; what it takes is warps, and few steps in each:
//  * a warp stays with one request and KV head for its run of page blocks, so that q's operands stay in registers;
//  * the order of the 256 terms is free, so a lane's 16 bytes of a row are taken as they come from memory, as the A operands
//    of two products, and q is read in the same order: no shared memory, no shuffle;
//  * the next block's lo halves are asked for when this one's have gone into the products, then the hi halves;
//  * the first page entries of all requests are read at once, where a search through them cost one latency a step.
// (Blocks on their way to rings in shared memory, one or two ahead, with nine to twelve warps an SM: 31 and 34 us for
// 128 decode requests of 1 to 8 K keys; sixteen warps that took a page's heads in turn, with nothing ahead: 26.)
// Measured: those requests 25 us (154 MB, 0.92 of the copy bandwidth).
constexpr int kScoreThreads = 128;
constexpr int kScoreCtas = 4;
constexpr int kScorePages = 16;
constexpr int kScoreList = 1024;  // requests whose first entries a CTA reads at once

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 16 pages of one KV head of a request.
struct ScoreBlock {
  Geo g;
  int r, room, pages;  // blocks that the line has for each head of the request, pages it has
  int head, block;
  int id;              // of page 16 block + lane % 16, -1 for none
  int id_after;        // of the place after it, if that is of the same request
};

// The line: for every request and KV head a place for each block.  Request r's begin at (its first entry) / 16 + r blocks,
// which leaves room for all of its own (and at times one more).
struct ScoreLine {
  const PageView& pv;
  const int* firsts;
  int batch, entries;

  __device__ __forceinline__ int begins(int k) const {
    return ((k == batch ? entries : k < kScoreList ? firsts[k] : __ldg(&pv.geo[k].kv0)) >> 4) + k;
  }
  __device__ __forceinline__ void enter(ScoreBlock& x) const {
    x.g = load_geo(pv.geo, x.r);
    x.room = begins(x.r + 1) - begins(x.r);
    x.pages = pages_of(pv, x.g.lkv);
  }
  __device__ __forceinline__ int ids_at(const ScoreBlock& x, int block) const {
    const int e = block * kScorePages + int(threadIdx.x & 15);
    return e < x.pages ? __ldg(pv.kv_indices + x.g.kv0 + e) : -1;
  }
  __device__ __forceinline__ void look_up(ScoreBlock& x, int id) const {
    x.id = id;
    if (id != -1 && static_cast<unsigned>(id) >= static_cast<unsigned>(pv.num_pages)) {
      atomicOr(pv.err, FI_DEVERR_PAGE_OOB);
      x.id = -1;
    }
    x.id_after = ids_at(x, x.block + 1 == x.room ? 0 : x.block + 1);
  }
  __device__ __forceinline__ void start(ScoreBlock& x, long long task) const {
    x.r = last_at_most(batch, int(task / pv.hkv), [&](int k) { return begins(k); });
    enter(x);
    const int in = int(task - (long long)begins(x.r) * pv.hkv);
    x.head = in / x.room;
    x.block = in - x.head * x.room;
    look_up(x, ids_at(x, x.block));
  }
  __device__ __forceinline__ void step(ScoreBlock& x) const {
    if (++x.block == x.room) {
      x.block = 0;
      if (++x.head == pv.hkv) {
        x.head = 0;
        ++x.r;
        enter(x);
        x.id_after = ids_at(x, 0);
      }
    }
    look_up(x, x.id_after);
  }
};

// Requests of up to eight columns (in a replay: of any number, eight at a time).  kHeads: heads of a group, 1, 2, 4 or 8; 0: any other
// number below 8, by a loop over the set's tokens.
template <int kHeads>
__global__ void __launch_bounds__(kScoreThreads, kScoreCtas) scores_kernel(const __grid_constant__ ScoreParams p) {
  __shared__ int firsts[kScoreList];
  const int lane = threadIdx.x & 31, row = lane >> 2, c = lane & 3;
  const PageView& pv = p.pv;
  for (int i = threadIdx.x; i < min(kScoreList, p.most_batch); i += kScoreThreads) firsts[i] = __ldg(&pv.geo[i].kv0);
  const GeoHead plan = load_head(pv.geo);
  if (plan.batch == 0) return wait_prior_grid();
  const int entries = __ldg(&pv.geo[plan.batch].kv0);
  __syncthreads();
  const ScoreLine line = {pv, firsts, plan.batch, entries};
  const long long tasks = (long long)line.begins(plan.batch) * pv.hkv, warps = (long long)gridDim.x * (kScoreThreads / 32);
  const long long me = (long long)blockIdx.x * (kScoreThreads / 32) + (threadIdx.x >> 5);
  long long task = tasks * me / warps;
  const long long t1 = tasks * (me + 1) / warps;
  if (task >= t1) return wait_prior_grid();
  const int heads = kHeads ? kHeads : p.group;
  const int fit = 8 / heads;                                // tokens of a set of eight columns
  const int col_tok = row / heads, col_head = row % heads;  // of column `row`

  ScoreBlock next;
  line.start(next, task);
  uint4 a[8], b[8];  // this lane's pieces of rows `row` and `row + 8`: 64-byte chunks 0-3 are lo, 4-7 hi
  auto fetch = [&](int k0) {
    const int ia = __shfl_sync(kAll, next.id, row), ib = __shfl_sync(kAll, next.id, row + 8);
    const uint4* pa = reinterpret_cast<const uint4*>(p.bounds + ((long long)max(ia, 0) * pv.hkv + next.head) * 2 * kHeadDim) + c;
    const uint4* pb = reinterpret_cast<const uint4*>(p.bounds + ((long long)max(ib, 0) * pv.hkv + next.head) * 2 * kHeadDim) + c;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (k < k0 || k >= k0 + 4) continue;
      a[k] = ia >= 0 ? __ldcs(pa + 4 * k) : make_uint4(0, 0, 0, 0);
      b[k] = ib >= 0 ? __ldcs(pb + 4 * k) : make_uint4(0, 0, 0, 0);
    }
  };
  wait_prior_grid();
  fetch(0);
  fetch(4);
  uint4 q[4];         // column `row` of the set at hand
  int q_key = -1;     // the (request, head) whose first set q holds
  for (; task < t1; ++task) {
    const ScoreBlock now = next;
    const bool more = task + 1 < t1;
    if (more) line.step(next);
    const int lq = now.g.lq;
    if (now.block * kScorePages >= now.pages || lq == 0) {  // an empty place
      if (more) {
        fetch(0);
        fetch(4);
      }
      continue;
    }
    const int ia = __shfl_sync(kAll, now.id, row), ib = __shfl_sync(kAll, now.id, row + 8);
    // column `row` of a set: (token, head of the group)
    auto query = [&](int tok) {
      const int ct = tok + col_tok;
      const bool on = col_tok < fit && ct < lq;
      const uint4* pq = reinterpret_cast<const uint4*>(p.q + ((long long)(now.g.q0 + (on ? ct : 0)) * p.hqo + now.head * p.group + (on ? col_head : 0)) * kHeadDim) + c;
#pragma unroll
      for (int k = 0; k < 4; ++k) q[k] = __ldg(pq + 4 * k);
    };
    const bool one = lq <= fit;  // one set of columns: q stays
    const int key = now.r * pv.hkv + now.head;
    if (!one || key != q_key) query(0);
    q_key = one ? key : -1;
    for (int tok = 0; tok < lq; tok += fit) {
      const int tok2 = tok + fit;
      float lo[4] = {0.f, 0.f, 0.f, 0.f}, hi[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t neg[4] = {min2(q[k].x, 0u, false), min2(q[k].y, 0u, false), min2(q[k].z, 0u, false), min2(q[k].w, 0u, false)};
        const uint32_t l0[4] = {a[k].x, b[k].x, a[k].y, b[k].y}, l1[4] = {a[k].z, b[k].z, a[k].w, b[k].w};
        mma_16816(lo, l0, neg[0], neg[1]);
        mma_16816(hi, l1, neg[2], neg[3]);
      }
      if (tok2 >= lq && more) fetch(0);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t pos[4] = {max2(q[k].x, 0u, false), max2(q[k].y, 0u, false), max2(q[k].z, 0u, false), max2(q[k].w, 0u, false)};
        const uint32_t h0[4] = {a[k + 4].x, b[k + 4].x, a[k + 4].y, b[k + 4].y}, h1[4] = {a[k + 4].z, b[k + 4].z, a[k + 4].w, b[k + 4].w};
        mma_16816(lo, h0, pos[0], pos[1]);
        mma_16816(hi, h1, pos[2], pos[3]);
      }
      if (tok2 >= lq && more) fetch(4);
      if (tok2 < lq) query(tok2);
      const float best[2][2] = {{lo[0] + hi[0], lo[1] + hi[1]}, {lo[2] + hi[2], lo[3] + hi[3]}};  // [page row][column 2 c, 2 c + 1]
      const int e0 = now.block * kScorePages + row;
      auto put = [&](int f, int half, float v) {  // the score of token tok + f and page e0 + 8 half
        const int e = e0 + 8 * half;
        if (f >= fit || tok + f >= lq || e >= now.pages || e >= p.row_pages) return;
        const int limit = plan.causal ? now.g.lkv - lq + tok + f : now.g.lkv - 1;
        const bool seen = (half ? ib : ia) >= 0 && (long long)e * pv.page_size <= limit;
        p.scores[((long long)(now.g.q0 + tok + f) * pv.hkv + now.head) * p.row_pages + e] = seen ? v * p.scale : -INFINITY;
      };
      if constexpr (kHeads == 1) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          put(2 * c + k, 0, best[0][k]);
          put(2 * c + k, 1, best[1][k]);
        }
      } else if constexpr (kHeads != 0) {
        // a token's columns are those of 1, 2 or 4 lanes; two of them write, or one both
        float v0 = max_nan(best[0][0], best[0][1]), v1 = max_nan(best[1][0], best[1][1]);
#pragma unroll
        for (int m = 1; m < kHeads / 2; m <<= 1) {
          v0 = max_nan(v0, __shfl_xor_sync(kAll, v0, m));
          v1 = max_nan(v1, __shfl_xor_sync(kAll, v1, m));
        }
        const int f = 2 * c / kHeads, at = c % (kHeads / 2);
        if (kHeads == 2) {
          put(f, 0, v0);
          put(f, 1, v1);
        } else if (at < 2) {
          put(f, at, at ? v1 : v0);
        }
      } else {
        for (int f = 0; f < fit && tok + f < lq; ++f) {
          float v0 = -INFINITY, v1 = -INFINITY;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const bool its = 2 * c + k >= f * heads && 2 * c + k < (f + 1) * heads;
            v0 = max_nan(v0, its ? best[0][k] : -INFINITY);
            v1 = max_nan(v1, its ? best[1][k] : -INFINITY);
          }
#pragma unroll
          for (int m = 1; m < 4; m <<= 1) {
            v0 = max_nan(v0, __shfl_xor_sync(kAll, v0, m));
            v1 = max_nan(v1, __shfl_xor_sync(kAll, v1, m));
          }
          if (c < 2) put(f, c, c ? v1 : v0);
        }
      }
    }
  }
}

// Requests of more columns, sixteen at a time.  There the instructions of a block count, not only the bounds' bytes, so q's columns are
// the rows of a product and the pages its columns: the words of a page are its operand as they come from memory, where as rows
// of a product four of them have to be moved together for each set (a fifth of all instructions), and 16 pages take two products an
// operand of q.  q streams by, a piece ahead (all of it in registers, the block's were spilled).  Both forms measured, two contexts of
// 131 K keys, 64/8 heads: 4 tokens each 19.2 us eight at a time, 16.0 sixteen (74 MB of bounds are 11); 16 tokens 55.8 and 39.2;
// four of 65 K, 16 heads a group, 16 tokens 99 and 87.  What is left is latency: no pipe is busy for a third of the time, DRAM for half
// of it, with twelve warps an SM and two chains of sixteen dependent products a set.  128 decode requests of four heads a group: 25 eight at a time, 32 sixteen.
// kHeads: heads of a group, 1, 2, 4 or 8; 16: more than 8, 16 at a time; 0: any other number below 8, by a loop over the set's tokens.
constexpr int kScoreWideCtas = 3;
constexpr int kScoreMostParts = 16;

template <int kHeads, bool kSplit>
__global__ void __launch_bounds__(kScoreThreads, kScoreWideCtas) scores_wide_kernel(const __grid_constant__ ScoreParams p) {
  constexpr int kValues = kHeads == 16 ? 4 : 8;  // that a lane gets of a set, the two halves of a token's 16 heads joined
  __shared__ int firsts[kScoreList];
  const int lane = threadIdx.x & 31, row = lane >> 2, c = lane & 3;
  const PageView& pv = p.pv;
  for (int i = threadIdx.x; i < min(kScoreList, p.most_batch); i += kScoreThreads) firsts[i] = __ldg(&pv.geo[i].kv0);
  const GeoHead plan = load_head(pv.geo);
  if (plan.batch == 0) return wait_prior_grid();
  const int entries = __ldg(&pv.geo[plan.batch].kv0);
  __syncthreads();
  const ScoreLine line = {pv, firsts, plan.batch, entries};
  // kSplit: a warp's piece of the line begins and ends within a block; part j of `parts` of it are the sets of every parts-th tokens
  // from the j-th on.
  const int parts = kSplit ? p.parts : 1;
  const long long units = (long long)line.begins(plan.batch) * pv.hkv * parts, warps = (long long)gridDim.x * (kScoreThreads / 32);
  const long long me = (long long)blockIdx.x * (kScoreThreads / 32) + (threadIdx.x >> 5);
  const long long u0 = units * me / warps, u1 = units * (me + 1) / warps, t0 = u0 / parts, t1 = (u1 + parts - 1) / parts;
  if (u0 >= u1) return wait_prior_grid();
  const int heads = kHeads ? kHeads : p.group;
  const int fit = kHeads == 16 ? 1 : 16 / heads;            // tokens of a set
  const int sets = kHeads == 16 ? (p.group + 15) / 16 : 1;  // sets of a token
  ScoreBlock next;
  line.start(next, t0);
  uint4 a[8], b[8];  // this lane's pieces of pages `row` and `row + 8`: 64-byte chunks 0-3 are lo, 4-7 hi
  const uint4 *pa = nullptr, *pb = nullptr;
  bool on_a = false, on_b = false;
  auto rows_of = [&]() {
    const int ia = __shfl_sync(kAll, next.id, row), ib = __shfl_sync(kAll, next.id, row + 8);
    pa = reinterpret_cast<const uint4*>(p.bounds + ((long long)max(ia, 0) * pv.hkv + next.head) * 2 * kHeadDim) + c;
    pb = reinterpret_cast<const uint4*>(p.bounds + ((long long)max(ib, 0) * pv.hkv + next.head) * 2 * kHeadDim) + c;
    on_a = ia >= 0;
    on_b = ib >= 0;
  };
  auto fetch = [&](int k) {
    a[k] = on_a ? __ldcs(pa + 4 * k) : make_uint4(0, 0, 0, 0);
    b[k] = on_b ? __ldcs(pb + 4 * k) : make_uint4(0, 0, 0, 0);
  };
  auto fetch_all = [&]() {
    rows_of();
#pragma unroll
    for (int k = 0; k < 8; ++k) fetch(k);
  };
  wait_prior_grid();
  fetch_all();
  uint4 q[2][2];  // columns `row` and `row + 8`: the piece at hand and the next
  for (long long task = t0; task < t1; ++task) {
    const ScoreBlock now = next;
    const bool more = task + 1 < t1;
    if (more) line.step(next);
    const int lq = now.g.lq;
    const int first = kSplit && task == t0 ? int(u0 - t0 * parts) : 0, end = kSplit && task + 1 == t1 ? int(u1 - task * parts) : parts;  // its parts
    auto after = [&](int tok) {  // the next tokens of those parts
      if (!kSplit) return tok + fit;
      const int g = tok / fit + 1, part = g & (parts - 1);
      return (part < first ? g - part + first : part >= end ? g - part + parts + first : g) * fit;
    };
    if (now.block * kScorePages >= now.pages || first * fit >= lq) {  // an empty place, or nothing in its parts
      if (more) fetch_all();
      continue;
    }
    auto column = [&](int half, int tok, int set) {  // q's pieces, four apart
      const int col = row + 8 * half, ct = tok + (kHeads == 16 ? 0 : col / heads), ch = kHeads == 16 ? set * 16 + col : col % heads;
      const bool on = ct < min(tok + fit, lq) && ch < p.group;
      return reinterpret_cast<const uint4*>(p.q + ((long long)(now.g.q0 + (on ? ct : 0)) * p.hqo + now.head * p.group + (on ? ch : 0)) * kHeadDim) + c;
    };
    const uint4* pq[2] = {column(0, first * fit, 0), column(1, first * fit, 0)};
    q[0][0] = __ldg(pq[0]);
    q[1][0] = __ldg(pq[1]);
    float best[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};  // 16 heads at a time: of the sets so far
    for (int tok = first * fit, set = 0; tok < lq;) {
      const bool last = set + 1 == sets;
      const int tok2 = last ? after(tok) : tok, set2 = last ? 0 : set + 1;
      const bool refill = tok2 >= lq && more;
      if (refill) rows_of();
      float s[2][4] = {};  // [page half]: [column half][page 2 c, 2 c + 1]
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint4 x = q[0][k & 1], y = q[1][k & 1];
        if (k < 3) {
          q[0][(k & 1) ^ 1] = __ldg(pq[0] + 4 * (k + 1));
          q[1][(k & 1) ^ 1] = __ldg(pq[1] + 4 * (k + 1));
        } else if (tok2 < lq) {
          pq[0] = column(0, tok2, set2);
          pq[1] = column(1, tok2, set2);
          q[0][0] = __ldg(pq[0]);
          q[1][0] = __ldg(pq[1]);
        }
        const uint32_t n0[4] = {min2(x.x, 0u, false), min2(y.x, 0u, false), min2(x.y, 0u, false), min2(y.y, 0u, false)};
        const uint32_t n1[4] = {min2(x.z, 0u, false), min2(y.z, 0u, false), min2(x.w, 0u, false), min2(y.w, 0u, false)};
        mma_16816(s[0], n0, a[k].x, a[k].y);
        mma_16816(s[1], n0, b[k].x, b[k].y);
        mma_16816(s[0], n1, a[k].z, a[k].w);
        mma_16816(s[1], n1, b[k].z, b[k].w);
        if (refill) fetch(k);
        const uint32_t p0[4] = {max2(x.x, 0u, false), max2(y.x, 0u, false), max2(x.y, 0u, false), max2(y.y, 0u, false)};
        const uint32_t p1[4] = {max2(x.z, 0u, false), max2(y.z, 0u, false), max2(x.w, 0u, false), max2(y.w, 0u, false)};
        mma_16816(s[0], p0, a[k + 4].x, a[k + 4].y);
        mma_16816(s[1], p0, b[k + 4].x, b[k + 4].y);
        mma_16816(s[0], p1, a[k + 4].z, a[k + 4].w);
        mma_16816(s[1], p1, b[k + 4].z, b[k + 4].w);
        if (refill) fetch(k + 4);
      }
      // The best of v's columns that differ in the lowest `bits` bits of `row`: each step leaves a lane half of the values, as long as it
      // has more than one.  put(f, index, value) for those that it is left with.
      auto join = [&](auto& v, int n, int bits, auto&& put) {
        int at = 0;
        bool mine = true;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          if (k >= bits) continue;
          const bool upper = lane >> (2 + k) & 1;
          if (n > 1) {
            n /= 2;
#pragma unroll
            for (int i = 0; i < kValues / 2; ++i) {
              if (i >= n) continue;
              const float keep = upper ? v[i + n] : v[i], give = upper ? v[i] : v[i + n];
              v[i] = max_nan(keep, __shfl_xor_sync(kAll, give, 4 << k));
            }
            at += upper ? n : 0;
          } else {
            v[0] = max_nan(v[0], __shfl_xor_sync(kAll, v[0], 4 << k));
            mine = mine && !upper;
          }
        }
#pragma unroll
        for (int i = 0; i < kValues; ++i)
          if (i < n) put(at + i, mine, v[i]);
      };
      // the score of token tok + f and the page of value `index`
      auto put = [&](int f, int index, bool mine, float v) {
        const int page = (index >> 1 & 1) * 8 + 2 * c + (index & 1), e = now.block * kScorePages + page;
        const int id = __shfl_sync(kAll, now.id, page);
        if (!mine || f >= fit || tok + f >= lq || e >= now.pages || e >= p.row_pages) return;
        const int limit = plan.causal ? now.g.lkv - lq + tok + f : now.g.lkv - 1;
        const bool seen = id >= 0 && (long long)e * pv.page_size <= limit;
        p.scores[((long long)(now.g.q0 + tok + f) * pv.hkv + now.head) * p.row_pages + e] = seen ? v * p.scale : -INFINITY;
      };
      if constexpr (kHeads == 16) {
        // 16 heads of one token, or what is left of them
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float x = set * 16 + row < p.group ? s[k >> 1][k & 1] : -INFINITY, y = set * 16 + row + 8 < p.group ? s[k >> 1][2 + (k & 1)] : -INFINITY;
          best[k] = max_nan(best[k], max_nan(x, y));
        }
        if (last) {
          join(best, 4, 3, [&](int index, bool mine, float v) { put(0, index, mine, v); });
#pragma unroll
          for (int k = 0; k < 4; ++k) best[k] = -INFINITY;
        }
      } else if constexpr (kHeads != 0) {
        float v[kValues];  // [column half][page half][page 2 c + j of it]
#pragma unroll
        for (int k = 0; k < kValues; ++k) v[k] = s[k >> 1 & 1][(k >> 2) * 2 + (k & 1)];
        constexpr int kBits = kHeads == 8 ? 3 : kHeads == 4 ? 2 : kHeads == 2 ? 1 : 0;
        join(v, kValues, kBits, [&](int index, bool mine, float x) { put((row >> kBits) + (index >> 2) * (8 >> kBits), index, mine, x); });
      } else {
        for (int f = 0; f < fit && tok + f < lq; ++f) {
          auto its = [&](int col) { return col >= f * heads && col < (f + 1) * heads; };
          float v[kValues];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            v[k] = max_nan(its(row) ? s[k >> 1][k & 1] : -INFINITY, its(row + 8) ? s[k >> 1][2 + (k & 1)] : -INFINITY);
          join(v, 4, 3, [&](int index, bool mine, float x) { put(f, index, mine, x); });
        }
      }
      tok = tok2;
      set = set2;
    }
  }
}

// ---- choice --------------------------------------------------------------------------------------------
// Of the n pages that a (token, KV head) row sees, the first `sink`, the last `recent` and the best of the rest, budget in
// all.  The threshold, the K-th largest score, is found from the top, two bits at a time: scores as integers of the same order, and at
// each step the counts of those at or above three candidates, which a warp sums as ten bits each of one number.  With more than one
// warp a step costs a barrier; once at most 512 scores are left to decide about, one warp goes on with them alone.  It ends once
// exactly K are counted.  Nothing depends on scheduling.  A warp holds a run of positions, so the chosen come out in order by counting.
// Rows longer than the CTA holds are read again for each count, a bit at a time.
// Bound by the chain of all this.  Measured: 64 x 8 rows of 128 to 512 pages 5.2 us (one bit a step, page ids where they are chosen, two votes
// a position: 7.7), 32 rows of 8193 9.6 (12.8, and 14.8 with every bit by all warps).
constexpr int kPickEach = 16;  // scores of a thread
constexpr int kPickMostWarps = 32;
constexpr uint32_t kPickFew = 32 * kPickEach;

// Order-preserving map; -0 counts as 0 and every NaN as the largest.
__device__ __forceinline__ uint32_t score_key(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// How many of a warp's (at most 512) scores are at or above x + 2^(bit - 1), x + 2^bit and x + both, ten bits each.
__device__ __forceinline__ uint32_t count_three(const uint32_t (&v)[kPickEach], uint32_t x, int bit) {
  const uint32_t x1 = x + (1u << (bit - 1)), x2 = x + (1u << bit), x3 = x2 + (1u << (bit - 1));
  uint32_t c[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < kPickEach; ++i) c[i & 1] += (v[i] >= x1 ? 1u : 0u) + (v[i] >= x2 ? 1u << 10 : 0u) + (v[i] >= x3 ? 1u << 20 : 0u);
  return __reduce_add_sync(kAll, c[0] + c[1]);
}
// The largest of the three and of x itself with at least `need` scores at or above it; whether they are exactly so many.
__device__ __forceinline__ bool narrow(uint32_t& x, int bit, uint32_t need, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t& from, uint32_t& above) {
  if (c1 < need) {
    above = c1;
    return false;
  }
  const uint32_t c = c3 >= need ? c3 : c2 >= need ? c2 : c1;
  x += (c2 >= need ? 1u << bit : 0u) + (c3 >= need || c2 < need ? 1u << (bit - 1) : 0u);
  above = c3 >= need ? above : c2 >= need ? c3 : c2;
  from = c;
  return c == need;
}

// kMost: the warps that it is compiled for, 1, 20 (96 registers a thread, 10240 pages) or 32 (64: 8193 pages 9.9 us in place
// of 9.6).
template <int kMost>
__global__ void __launch_bounds__(32 * kMost) pick_kernel(const __grid_constant__ PickParams p) {
  constexpr bool kOne = kMost == 1;
  __shared__ uint32_t counts[2][kPickMostWarps];
  __shared__ uint2 runs[kPickMostWarps];
  __shared__ uint32_t list[kOne ? 1 : kPickFew], list_end;
  const PageView& pv = p.pv;
  const GeoHead plan = load_head(pv.geo);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = kOne ? 1 : int(blockDim.x >> 5);
  const long long rows = (long long)plan.total_q * pv.hkv;
  Geo g = {};
  int r;
  if (blockIdx.x < rows) g = request_of(pv.geo, plan.batch, int(blockIdx.x / pv.hkv), r);
  wait_prior_grid();
  int turn = 0;
  auto total = [&](uint32_t v) {  // over the CTA; every thread gets it
    v = __reduce_add_sync(kAll, v);
    if (kOne) return v;
    if (lane == 0) counts[turn][warp] = v;
    __syncthreads();
    v = __reduce_add_sync(kAll, lane < warps ? counts[turn][lane] : 0u);
    turn ^= 1;
    return v;
  };
  for (long long row = blockIdx.x; row < rows; row += gridDim.x) {
    const int t = int(row / pv.hkv);
    const float* scores = p.scores + row * p.row_pages;
    const int span = warps * 32 * kPickEach;
    // this thread's scores of the run of positions that begins at `base`, as far as the row has room
    auto read = [&](int base, float (&w)[kPickEach]) {
#pragma unroll
      for (int i = 0; i < kPickEach; ++i) {
        const int pos = base + (warp * kPickEach + i) * 32 + lane;
        w[i] = pos < p.row_pages ? __ldg(scores + pos) : 0.f;
      }
    };
    float w0[kPickEach];
    read(0, w0);  // on their way while the request is looked up
    if (row != blockIdx.x) g = request_of(pv.geo, plan.batch, t, r);
    const int limit = plan.causal ? g.lkv - g.lq + (t - g.q0) : g.lkv - 1;  // the last key that the token sees
    const int n = limit < 0 ? 0 : p.row_pages > 0 ? min(pages_of(pv, limit + 1), p.row_pages) : 0;
    const int32_t* ids = pv.kv_indices + g.kv0;
    int32_t* out = p.selected + row * p.budget;
    const int kept = min(n, p.budget);
    for (unsigned i = unsigned(kept) + threadIdx.x; i < unsigned(p.budget); i += blockDim.x) out[i] = -1;
    if (n <= p.budget) {
      for (int i = threadIdx.x; i < n; i += blockDim.x) out[i] = __ldg(ids + i);
      continue;
    }
    const int f0 = p.sink, f1 = n - p.recent;  // positions that the scores decide about
    const uint32_t need = uint32_t(p.budget - p.sink - p.recent);
    // no score maps to 0, which stands for none
    auto keys_of = [&](int base, const float (&w)[kPickEach], uint32_t (&key)[kPickEach]) {
#pragma unroll
      for (int i = 0; i < kPickEach; ++i) {
        const int pos = base + (warp * kPickEach + i) * 32 + lane;
        key[i] = pos >= f0 && pos < f1 ? score_key(w[i]) : 0u;
      }
    };
    auto fetch = [&](int base, uint32_t (&key)[kPickEach]) {
      float w[kPickEach];
      read(base, w);
      keys_of(base, w, key);
    };
    uint32_t key[kPickEach];
    keys_of(0, w0, key);
    // The page ids of the run at hand, all of them: asked for where one is chosen, each took a latency of its own (4000 clocks).
    // Up to 20 warps ask before the search, where they cost nothing; more have no registers for that.
    int id[kPickEach];
    auto look_up = [&](int base) {
#pragma unroll
      for (int i = 0; i < kPickEach; ++i) {
        const int pos = base + (warp * kPickEach + i) * 32 + lane;
        id[i] = pos < n ? __ldg(ids + pos) : 0;
      }
    };
    if (kMost <= 20) look_up(0);
    auto at_least = [&](uint32_t x) {
      uint32_t k = 0;
      if (n <= span) {
#pragma unroll
        for (int i = 0; i < kPickEach; ++i) k += key[i] >= x;
      } else {
        for (int base = 0; base < n; base += span) {
          uint32_t some[kPickEach];
          fetch(base, some);
#pragma unroll
          for (int i = 0; i < kPickEach; ++i) k += some[i] >= x;
        }
      }
      return total(k);
    };
    uint32_t limit_key = 0;  // the largest x with at least `need` scores at or above it
    bool exact = need == 0;
    if (exact) limit_key = 0xffffffffu;
    uint32_t from = uint32_t(n), above = 0;  // scores at or above limit_key (at most), and at or above limit_key + 2^(bit + 1)
    int bit = 31;
    if (n <= span) {
      for (; bit >= 0 && !exact; bit -= 2) {  // two bits at a time
        if (!kOne && from - above <= kPickFew) break;
        const uint32_t c = count_three(key, limit_key, bit);  // of a warp
        uint32_t c1 = c & 1023u, c2 = c >> 10 & 1023u, c3 = c >> 20;
        if (!kOne) {
          if (lane == 0) counts[turn][warp] = c;
          __syncthreads();
          const uint32_t v = lane < warps ? counts[turn][lane] : 0u;
          const uint32_t two = __reduce_add_sync(kAll, (v & 1023u) | (v >> 10 & 1023u) << 16);
          c1 = two & 0xffffu;
          c2 = two >> 16;
          c3 = __reduce_add_sync(kAll, v >> 20);
          turn ^= 1;
        }
        exact = narrow(limit_key, bit, need, c1, c2, c3, from, above);
      }
    } else {
      for (; bit >= 0 && !exact; --bit) {
        const uint32_t x = limit_key | (1u << bit);
        const uint32_t k = at_least(x);
        if (k >= need) limit_key = x;
        exact = k == need;
      }
    }
    // scores above the limit stay, of those at it the first few; if exactly `need` are at or above it, all of them
    uint32_t ties = exact && need != 0 ? 0xffffffffu : 0u;
    if (!kOne && !exact && bit >= 0) {
      // the few that the remaining bits decide about, to one warp
      if (threadIdx.x == 0) list_end = 0;
      __syncthreads();
      const uint32_t low = max(limit_key, 1u);  // low .. limit_key + 2^(bit + 1) - 1, but never 0
      const uint32_t size = (bit == 31 ? 0u : limit_key + (2u << bit)) - low;
      auto in = [&](uint32_t v) { return v - low < size; };
      uint32_t mine = 0;
#pragma unroll
      for (int i = 0; i < kPickEach; ++i) mine += in(key[i]);
      uint32_t to = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(kAll, to, o);
        to += lane >= o ? v : 0u;
      }
      uint32_t base = 0;
      if (lane == 31) base = atomicAdd(&list_end, to);  // (their order does not matter, only how many lie where)
      to += __shfl_sync(kAll, base, 31) - mine;
#pragma unroll
      for (int i = 0; i < kPickEach; ++i)
        if (in(key[i])) list[to++] = key[i];
      __syncthreads();
      if (warp == 0) {
        uint32_t some[kPickEach];
#pragma unroll
        for (int i = 0; i < kPickEach; ++i) some[i] = uint32_t(32 * i + lane) < list_end ? list[32 * i + lane] : 0u;
        auto count = [&](uint32_t x) {
          uint32_t k = 0;
#pragma unroll
          for (int i = 0; i < kPickEach; ++i) k += some[i] >= x;
          return __reduce_add_sync(kAll, k);
        };
        const uint32_t left = need - above;
        bool done = false;
        uint32_t unused = 0;
        for (; bit >= 0 && !done; bit -= 2) {
          const uint32_t c = count_three(some, limit_key, bit);
          done = narrow(limit_key, bit, left, c & 1023u, c >> 10 & 1023u, c >> 20, unused, unused);
        }
        ties = done ? 0xffffffffu : left - (limit_key == 0xffffffffu ? 0u : count(limit_key + 1));
        if (lane == 0) runs[0] = make_uint2(limit_key, ties);
      }
      __syncthreads();
      limit_key = runs[0].x;
      ties = runs[0].y;
    } else if (!exact) {
      ties = need - (limit_key == 0xffffffffu ? 0u : at_least(limit_key + 1));
    }
    uint32_t before = 0, ties_before = 0;  // chosen positions and ties in the runs before
    for (int base = 0; base < n; base += span) {
      if (base > 0) fetch(base, key);
      if (kMost > 20 || base > 0) look_up(base);
      uint32_t stays = 0, ties_here = 0;  // bit i: of position i of this thread
#pragma unroll
      for (int i = 0; i < kPickEach; ++i) {
        const int pos = base + (warp * kPickEach + i) * 32 + lane;
        if (pos < f0 || (pos >= f1 && pos < n) || key[i] > limit_key) stays |= 1u << i;
        if (key[i] == limit_key && key[i] != 0u) ties_here |= 1u << i;
      }
      const uint32_t sure = __reduce_add_sync(kAll, __popc(stays)), tied = __reduce_add_sync(kAll, __popc(ties_here));  // of this warp
      uint32_t my_sure = before, my_ties = ties_before;
      if (!kOne) {
        __syncthreads();  // the last reads of `runs` and `counts`
        if (lane == 0) runs[warp] = make_uint2(sure, tied);
        __syncthreads();
        const uint2 v = lane < warps ? runs[lane] : make_uint2(0u, 0u);
        my_sure += __reduce_add_sync(kAll, lane < warp ? v.x : 0u);
        my_ties += __reduce_add_sync(kAll, lane < warp ? v.y : 0u);
        before += __reduce_add_sync(kAll, v.x);
        ties_before += __reduce_add_sync(kAll, v.y);
      } else {
        before += sure;
        ties_before += tied;
      }
      uint32_t at = my_sure + min(my_ties, ties);
      uint32_t take = ties - min(my_ties, ties);  // of this warp's ties the first so many
      const unsigned below = (1u << lane) - 1;
      if (take >= tied) {
        stays |= ties_here;
      } else if (take > 0) {
#pragma unroll
        for (int i = 0; i < kPickEach; ++i) {
          const unsigned there = __ballot_sync(kAll, ties_here >> i & 1u);
          if ((ties_here >> i & 1u) && __popc(there & below) < take) stays |= 1u << i;
          take -= min(take, uint32_t(__popc(there)));
        }
      }
#pragma unroll
      for (int i = 0; i < kPickEach; ++i) {
        const unsigned there = __ballot_sync(kAll, stays >> i & 1u);
        if (stays >> i & 1u) out[at + __popc(there & below)] = id[i];
        at += __popc(there);
      }
    }
    if (!kOne) __syncthreads();
  }
}

// ---- the attention's work --------------------------------------------------------------------------------
// A unit is a (query token, KV head) row with its own page list.  The lists form one line, counted in steps of block_pages
// pages (a request's units by its own number of pages, or the budget if that is less), and every CTA gets an equal piece.
// Unit u's piece in CTA c is item u + c: both grow along the line, so the items need no scan; where a CTA begins with
// a unit, one number stays free and gets an item without rows.  A unit that spans CTAs a .. b is split unit a, with the slots
// 2 a, 2 a + 1, ...: the next split unit begins in CTA b at the earliest, and b > a.
// A warp reads a unit's list: the pages in it, and whether the page where the token's keys end comes last.
// Bound by its chain of look-ups.  Measured with the attention behind it: 3 requests of 32 pages 10.6 us; 128 of 128 pages 169
// (1.08 GB, 0.95 of the copy bandwidth).
constexpr int kPlanThreads = 256;
constexpr int kPlanWarps = kPlanThreads / 32;

__device__ __forceinline__ void put_item(int32_t* items, long long at, int page_base, int q_start, int q_len, int head, int lo, int hi, int slot) {
  reinterpret_cast<int4*>(items)[2 * at] = make_int4(page_base, q_start, q_len, head);
  reinterpret_cast<int4*>(items)[2 * at + 1] = make_int4(lo, hi, kNotCausalDiag, slot);
}
__device__ __forceinline__ void put_unit(int32_t* units, int at, int slot, int n, int q_start, int q_len, int head) {
  reinterpret_cast<int4*>(units)[2 * at] = make_int4(slot, n, q_start, q_len);
  reinterpret_cast<int4*>(units)[2 * at + 1] = make_int4(head, 0, 0, 0);
}

__global__ void __launch_bounds__(kPlanThreads) list_plan_kernel(const __grid_constant__ ListPlanParams p) {
  __shared__ long long sums[2][kPlanWarps];
  const PageView& pv = p.pv;
  const GeoHead plan = load_head(pv.geo);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long units = (long long)plan.total_q * pv.hkv;
  // (a replay may bring more tokens than the list numbers have room for)
  const bool room = units * p.budget <= INT32_MAX;
  if (units == 0 || !room) {
    wait_prior_grid();
    if (blockIdx.x == 0) {
      if (threadIdx.x == 0) p.header[H_NUM_UNITS] = p.ctas;
      for (int c = threadIdx.x; c <= p.ctas; c += kPlanThreads) p.cta_indptr[c] = 0;
      for (int c = threadIdx.x; c < p.ctas; c += kPlanThreads) put_unit(p.units, c, 0, 0, 0, 0, 0);
      if (threadIdx.x == 0 && !room) atomicOr(pv.err, FI_DEVERR_KEPT);
    }
    return;
  }
  const long long u0 = units * blockIdx.x / gridDim.x, u1 = units * (blockIdx.x + 1) / gridDim.x;
  if (u0 >= u1) return wait_prior_grid();
  auto steps_of = [&](const Geo& g) {
    const int pages = min(pages_of(pv, g.lkv), p.budget);
    return max(1, (pages + p.block_pages - 1) / p.block_pages);
  };
  // the line's length, and its part before the request of this CTA's first unit
  int r;
  Geo g = request_of(pv.geo, plan.batch, int(u0 / pv.hkv), r);
  long long all = 0, before = 0;
  for (int k = threadIdx.x; k < plan.batch; k += kPlanThreads) {
    const Geo x = load_geo(pv.geo, k);
    const long long n = (long long)x.lq * pv.hkv * steps_of(x);
    all += n;
    if (k < r) before += n;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    all += __shfl_xor_sync(kAll, all, o);
    before += __shfl_xor_sync(kAll, before, o);
  }
  if (lane == 0) {
    sums[0][warp] = all;
    sums[1][warp] = before;
  }
  __syncthreads();
  all = before = 0;
#pragma unroll
  for (int k = 0; k < kPlanWarps; ++k) {
    all += sums[0][k];
    before += sums[1][k];
  }
  const long long per = max((long long)p.least, (all + p.ctas - 1) / p.ctas);
  const int used = int((all + per - 1) / per);

  int steps = steps_of(g);
  wait_prior_grid();
  for (long long u = u0 + warp; u < u1; u += kPlanWarps) {
    const int t = int(u / pv.hkv), head = int(u - (long long)t * pv.hkv);
    while (t >= g.q0 + g.lq) {
      before += (long long)g.lq * pv.hkv * steps;
      g = load_geo(pv.geo, ++r);
      steps = steps_of(g);
    }
    const long long a = before + (u - (long long)g.q0 * pv.hkv) * steps, b = a + steps;
    const int first = int(a / per), last = int((b - 1) / per);
    // the list: pages up to the first -1, the page of the token's last key at its end or not at all
    const int limit = plan.causal ? g.lkv - g.lq + (t - g.q0) : g.lkv - 1;
    const int32_t* list = p.selected + u * p.budget;
    const int end_page = limit >= 0 ? __ldg(pv.kv_indices + g.kv0 + limit / pv.page_size) : -1;
    const int end_keys = limit >= 0 ? limit % pv.page_size + 1 : 0;
    int n = 0;
    unsigned found = 0, at_end = 0;  // places of the end page among the last 32 read, whether it is the last of the list
    bool early = false;
    if (limit >= 0) {
      constexpr int kAhead = 4;
      for (int k0 = 0; k0 < p.budget; k0 += 32 * kAhead) {
        int id[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int k = k0 + 32 * i + lane;
          id[i] = k >= k0 && k < p.budget ? __ldg(list + k) : -1;
        }
        bool over = false;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          if (over) continue;
          const unsigned there = __ballot_sync(kAll, id[i] >= 0);
          const int here = there == kAll ? 32 : __ffs(~there) - 1;
          found = __ballot_sync(kAll, lane < here && id[i] == end_page);
          if (here > 0) {
            early = early || at_end != 0 || (found & ~(1u << (here - 1))) != 0;
            at_end = found >> (here - 1) & 1u;
          }
          n += here;
          over = here < 32;
        }
        if (over || k0 > p.budget - 32 * kAhead) break;
      }
    }
    // (the slots behind the token's last key are not keys: such a page is only read as the last of a list)
    const bool wrong = early && end_keys < pv.page_size;
    if (wrong && lane == 0) atomicOr(pv.err, FI_DEVERR_KEPT);
    const int keys = wrong ? 0 : int(min((long long)INT32_MAX / 2, (long long)n * pv.page_size)) - (at_end ? pv.page_size - end_keys : 0);
    for (int c = first + lane; c <= last; c += 32) {
      const long long x0 = max(a, c * per) - a, x1 = min(b, (c + 1) * per) - a;
      const long long step_keys = (long long)p.block_pages * pv.page_size;
      const int lo = int(min((long long)keys, x0 * step_keys));
      const int hi = c == last ? keys : int(min((long long)keys, x1 * step_keys));
      put_item(p.items, u + c, int(u) * p.budget, t, 1, head, lo, hi, first == last ? -1 : 2 * first + (c - first));
      if (first != last) p.slot_unit[2 * first + (c - first)] = first;
      if (c * per >= a) {  // the CTA begins here
        p.cta_indptr[c] = int(u) + c;
        const bool inside = c * per > a;
        if (!inside && c > 0) put_item(p.items, u + c - 1, 0, 0, 0, 0, 0, 0, -1);
        if (c > 0) {
          if (inside && c - 1 == first)
            put_unit(p.units, first, 2 * first, last - first + 1, t, 1, head);
          else
            put_unit(p.units, c - 1, 0, 0, 0, 0, 0);
        }
      }
    }
    if (u == units - 1) {  // (whose CTA is not always the first: a captured grid may have more CTAs than there are units)
      if (lane == 0) p.header[H_NUM_UNITS] = p.ctas;
      for (int c = used + lane; c <= p.ctas; c += 32) {
        p.cta_indptr[c] = int(units) + used - 1;
        put_unit(p.units, c - 1, 0, 0, 0, 0, 0);
      }
    }
  }
}

}  // namespace

int launch_bounds(const BoundsParams& p, int64_t tasks, bool fp8, int num_sms, cudaStream_t stream) {
  constexpr int kWarps = kBoundsThreads / 32;
  const unsigned grid = unsigned(std::max<int64_t>(1, std::min<int64_t>((tasks + kWarps - 1) / kWarps, int64_t(num_sms) * 2)));
  const cudaError_t e = fp8 ? launch_dependent(bounds_kernel<true>, grid, kBoundsThreads, 0, 1, stream, p)
                            : launch_dependent(bounds_kernel<false>, grid, kBoundsThreads, 0, 1, stream, p);
  return e == cudaSuccess ? FI_OK : record_cuda_error(e, "bounds_kernel launch");
}

int launch_scores(ScoreParams p, int64_t tasks, int num_sms, cudaStream_t stream) {
  constexpr int kWarps = kScoreThreads / 32;
  using Kernel = void (*)(const ScoreParams);
  static const Kernel kernels[3][6] = {
      {scores_kernel<0>, scores_kernel<1>, scores_kernel<2>, scores_kernel<4>, scores_kernel<8>, nullptr},
      {scores_wide_kernel<0, false>, scores_wide_kernel<1, false>, scores_wide_kernel<2, false>, scores_wide_kernel<4, false>,
       scores_wide_kernel<8, false>, scores_wide_kernel<16, false>},
      {scores_wide_kernel<0, true>, scores_wide_kernel<1, true>, scores_wide_kernel<2, true>, scores_wide_kernel<4, true>,
       scores_wide_kernel<8, true>, scores_wide_kernel<16, true>}};
  const int heads = p.group > 8 ? 5 : p.group == 8 ? 4 : p.group == 4 ? 3 : p.group == 2 ? 2 : p.group == 1 ? 1 : 0;
  const bool wide = int64_t(std::max(1, p.most_lq)) * p.group > 8;
  // Blocks' sets are shared out where there are fewer than two blocks a warp (one context of 16 K keys, 512 tokens of 32/8 heads 109 -> 47 us,
  // two of 32 K, 64 tokens of 64/8 55 -> 41; with more, a block read by two warps costs more than even pieces save: two of 131 K, 16 tokens
  // 39 and 42).
  const int fit = p.group > 8 ? 1 : 16 / p.group;
  p.parts = 1;
  if (wide && tasks < int64_t(num_sms) * kScoreWideCtas * kWarps * 2)
    while (p.parts < kScoreMostParts && 2 * int64_t(p.parts) * fit <= p.most_lq) p.parts *= 2;
  tasks *= p.parts;
  const Kernel kernel = kernels[wide ? 1 + (p.parts > 1) : 0][heads];
  const unsigned grid = unsigned(std::max<int64_t>(1, std::min<int64_t>((tasks + kWarps - 1) / kWarps, int64_t(num_sms) * (wide ? kScoreWideCtas : kScoreCtas))));
  const cudaError_t e = launch_dependent(kernel, grid, kScoreThreads, 0, 1, stream, p);
  return e == cudaSuccess ? FI_OK : record_cuda_error(e, "scores_kernel launch");
}

int launch_pick(const PickParams& p, int64_t rows, int most_pages, int num_sms, cudaStream_t stream) {
  const int warps = std::min(kPickMostWarps, std::max(1, (most_pages + 32 * kPickEach - 1) / (32 * kPickEach)));
  const unsigned grid = unsigned(std::max<int64_t>(1, std::min<int64_t>(rows, int64_t(num_sms) * std::min(32, 64 / warps))));
  const auto kernel = warps == 1 ? pick_kernel<1> : warps <= 20 ? pick_kernel<20> : pick_kernel<32>;
  const cudaError_t e = launch_dependent(kernel, grid, unsigned(warps) * 32, 0, 1, stream, p);
  return e == cudaSuccess ? FI_OK : record_cuda_error(e, "pick_kernel launch");
}

int launch_list_plan(const ListPlanParams& p, int64_t units, int num_sms, cudaStream_t stream) {
  const unsigned grid = unsigned(std::max<int64_t>(1, std::min<int64_t>((units + kPlanWarps - 1) / kPlanWarps, int64_t(num_sms) * 4)));
  const cudaError_t e = launch_dependent(list_plan_kernel, grid, kPlanThreads, 0, 1, stream, p);
  return e == cudaSuccess ? FI_OK : record_cuda_error(e, "list_plan_kernel launch");
}

}  // namespace fi
