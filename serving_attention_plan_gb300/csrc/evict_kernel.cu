// Selection of the keys to keep, and their compaction, per (request, KV head).
#include <algorithm>
#include <mutex>
#include <type_traits>

#include "cache_common.cuh"
#include "prefill_launch.h"

namespace fi {
namespace {

constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ unsigned cluster_size() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// An arrival that publishes no writes.  It says that this thread's reads have come back, and rests on a wait that comes
// before it (cp.async.wait_group, or a use of the value): the barrier itself orders nothing then.  (The release form
// waits for the thread's stores as well.)
__device__ __forceinline__ void cluster_arrive_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync_all() {
  cluster_arrive();
  cluster_wait();
}
// Reads a 32-bit word at the same shared-memory place of another CTA of the cluster.
__device__ __forceinline__ uint32_t peer_word(const void* local, unsigned rank) {
  uint32_t at, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(local)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

// ---- selection -----------------------------------------------------------------------------------
// The free range of a row is its keys [sink, L - recent); of those the K = budget - sink - recent
// largest stay, ties to the lowest position.  A radix select finds the K-th largest exactly: the
// weights are mapped to 32-bit integers in the same order, and three passes of 11, 11 and 10 bits
// narrow the threshold down by counting.  Counts are integers, so shared-memory atomics do not
// change the result.  A pass ends the search when all keys of its bin stay, which without many equal weights
// the second does.  The kept positions come out ascending by ranking (greater, equal) counts over the range in
// order, four positions a thread.  Measured: 64 x 8 rows of 2 to 4 K keys 15.2 us, 8 rows of 131 K 17.8 us; the look-ups and
// weights of a row take a third of that, the rest is a chain of counting steps.  Weights are read from memory once (the slice of the range that a CTA owns
// stays in shared memory); a cluster of CTAs shares a row when there are few rows.
//   Where pages hold whole groups of four slots, a thread fetches four weights at a time (one page id, one 16-byte
// load); one at a time the instructions around the loads took most of the time.  In a cluster every CTA
// reads its peers' counts in two steps, 64 coarse bins and then the 32 bins of the one that holds the threshold:
// reading all bins of all peers took 4 us a pass with 8 CTAs.
constexpr int kBins = 2048;
constexpr int kCoarse = kBins / 32;
constexpr int kFetch = 8;  // weights a thread has in flight

struct SelectSmem {
  uint32_t hist[3][kBins];
  uint32_t coarse[3][kCoarse];  // cluster: the histogram in runs of 32 bins
  uint32_t row[kCoarse + 32];   // cluster: the row's coarse counts, and the 32 of the hit
  uint32_t scan[2][32];         // the warps' counts of a chunk
  uint32_t total_gt, total_eq;  // of this CTA's slice
  uint32_t digit[3], above, within;  // result of a pass: the bin, the keys above it and in it
};

// Order-preserving map; -0 counts as 0 and every NaN as the largest.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 1024 ? 1 : 6) select_kernel(const __grid_constant__ SelectParams p, int cap) {
  extern __shared__ __align__(16) uint32_t keys[];  // [cap]: the CTA's slice of the row
  __shared__ SelectSmem sm;
  constexpr int kWarps = kThreads / 32;
  auto clear = [&]() {
    for (int i = threadIdx.x; i < 3 * kBins; i += kThreads) (&sm.hist[0][0])[i] = 0;
    if (threadIdx.x == 0) sm.total_gt = sm.total_eq = sm.digit[0] = sm.digit[1] = sm.digit[2] = sm.above = sm.within = 0;
  };
  clear();
  __syncthreads();
  wait_prior_grid();
  const PageView& pv = p.pv;
  const int batch = load_head(pv.geo).batch;
  const unsigned nr = cluster_size(), rank = cluster_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rows = batch * pv.hkv;
  for (int row = blockIdx.x / nr; row < rows; row += gridDim.x / nr) {
    const int r = row / pv.hkv, head = row - r * pv.hkv;
    const Geo g = load_geo(pv.geo, r);
    int32_t* kept = p.kept + (long long)row * p.budget;
    if (g.lkv <= p.budget) {
      // (a budget may be as large as 2^31 - 1, where a signed counter would overflow)
      for (unsigned i = rank * kThreads + tid; i < unsigned(p.budget); i += nr * kThreads)
        kept[i] = i < unsigned(g.lkv) ? int(i) : -1;
      continue;  // the same for every CTA of the cluster
    }
    const int f0 = p.sink, f1 = g.lkv - p.recent;
    const int need = p.budget - p.sink - p.recent;
    for (int i = rank * kThreads + tid; i < p.sink + p.recent; i += nr * kThreads) {
      if (i < p.sink)
        kept[i] = i;
      else
        kept[p.budget - p.recent + i - p.sink] = g.lkv - p.recent + i - p.sink;
    }
    if (need == 0) continue;
    // this CTA's slice of whole steps of 32 positions; key 0, which no weight maps to, marks positions outside
    // the free range
    const int a0 = f0 & ~31;
    const int per = (((f1 - a0 + int(nr) - 1) / int(nr)) + 31) & ~31;
    const int s0 = min(f1, a0 + int(rank) * per), n = min(f1, s0 + per) - s0;
    const bool in_smem = n <= cap;
    auto fetch_one = [&](int i) -> uint32_t {
      int page, slot;
      if (s0 + i < f0 || i >= n || !locate(pv, g.kv0, s0 + i, page, slot)) return 0u;
      return order_key(__ldg(p.weights + weight_offset(pv, page, slot, head)));
    };
    // kFetch keys: kFetch / kVec groups of kVec positions, `apart` groups between them; all page ids first
    auto fetch = [&](int group, int apart, uint32_t (&x)[kFetch], auto vec) {
      constexpr int kVec = decltype(vec)::value;
      int at[kFetch / kVec];  // a pool holds fewer than 2^31 rows: its K alone takes 128 bytes each
#pragma unroll
      for (int k = 0; k < kFetch / kVec; ++k) {
        const int i = (group + k * apart) * kVec;
        int page, slot;
        at[k] = -1;
        if (i < n && s0 + i + kVec > f0 && locate(pv, g.kv0, s0 + i, page, slot))
          at[k] = int(weight_offset(pv, page, slot, head));
      }
#pragma unroll
      for (int k = 0; k < kFetch / kVec; ++k) {
        float w[kVec];
        if (at[k] >= 0) {
          if constexpr (kVec == 4)
            *reinterpret_cast<float4*>(w) = __ldg(reinterpret_cast<const float4*>(p.weights + at[k]));
          else
            w[0] = __ldg(p.weights + at[k]);
        }
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          const int i = (group + k * apart) * kVec + e;
          x[k * kVec + e] = at[k] >= 0 && i < n && s0 + i >= f0 ? order_key(w[e]) : 0u;
        }
      }
    };
    uint32_t prefix = 0;  // the digits found so far, in place
    uint32_t left = uint32_t(need);
    int passes = 0;
    bool all_in = false;  // every key of the last bin stays: there is no need to look into it
    int missing = 0;      // free places that no key takes: pages outside the pool hold the others (error bit set)
    for (int pass = 0; pass < 3 && !all_in; ++pass, ++passes) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t mask = pass == 2 ? 1023u : 2047u;
      const uint32_t known = pass == 0 ? 0u : pass == 1 ? 0xffe00000u : 0xfffffc00u;
      auto count = [&](uint32_t x) {
        if (x != 0 && (x & known) == prefix) atomicAdd(&sm.hist[pass][(x >> shift) & mask], 1u);
      };
      if (pass > 0 && in_smem) {
        for (int i = 4 * tid; i < n; i += 4 * kThreads) {
          const uint4 x = *reinterpret_cast<const uint4*>(keys + i);
          count(x.x);
          if (i + 1 < n) count(x.y);
          if (i + 2 < n) count(x.z);
          if (i + 3 < n) count(x.w);
        }
      } else {
        auto all = [&](auto vec) {
          constexpr int kVec = decltype(vec)::value;
          const int groups = (n + kVec - 1) / kVec;
          for (int q = tid; q < groups; q += kFetch / kVec * kThreads) {
            uint32_t x[kFetch];
            fetch(q, kThreads, x, vec);
#pragma unroll
            for (int k = 0; k < kFetch / kVec; ++k) {
              const int i = (q + k * kThreads) * kVec;
              if (i >= n) break;
              if (in_smem) {  // the slice's storage is a multiple of four
                if constexpr (kVec == 4)
                  *reinterpret_cast<uint4*>(keys + i) = make_uint4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
                else
                  keys[i] = x[k];
              }
#pragma unroll
              for (int e = 0; e < kVec; ++e) count(x[k * kVec + e]);
            }
          }
        };
        if (p.by_four)
          all(std::integral_constant<int, 4>());
        else
          all(std::integral_constant<int, 1>());
      }
      __syncthreads();
      // the bin that holds the `left`-th largest: first its run of 32 bins, then itself
#pragma unroll
      for (int k = 0; k < kCoarse / kWarps; ++k) {
        const uint32_t v = __reduce_add_sync(kAll, sm.hist[pass][(warp + kWarps * k) * 32 + lane]);
        if (lane == 0) sm.coarse[pass][warp + kWarps * k] = v;
      }
      if (nr > 1 && tid < kCoarse + 32) sm.row[tid] = 0;
      __syncthreads();
      const uint32_t* coarse = sm.coarse[pass];
      if (nr > 1) {
        cluster_sync_all();
        if (tid < kCoarse * int(nr)) {
          const int bin = tid & (kCoarse - 1);
          const uint32_t v = peer_word(&sm.coarse[pass][bin], unsigned(tid / kCoarse));
          if (v) atomicAdd(&sm.row[bin], v);
        }
        __syncthreads();
        coarse = sm.row;
      }
      {
        // every warp finds the run by itself: lane l takes runs 63 - 2 l and 62 - 2 l
        const uint32_t c0 = coarse[kCoarse - 1 - 2 * lane], c1 = coarse[kCoarse - 2 - 2 * lane];
        uint32_t upto = c0 + c1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t u = __shfl_up_sync(kAll, upto, o);
          if (lane >= o) upto += u;
        }
        // Fewer keys than places (the whole cluster sees the same sum): all that were counted stay.  Only the
        // first pass can find so, later ones look into a bin that holds enough.  The bins' own counts place the slices, as
        // after a pass whose bin 0 stays as a whole.
        const uint32_t counted = __shfl_sync(kAll, upto, 31);
        if (counted < left) {
          missing = int(left - counted);
          prefix = 1;
          all_in = true;
          passes = 1;
          break;  // sm.digit[0] is 0 still
        }
        const int hit = __ffs(__ballot_sync(kAll, left <= upto)) - 1;
        uint32_t skipped = __shfl_sync(kAll, upto - c0 - c1, hit);
        const uint32_t h0 = __shfl_sync(kAll, c0, hit);
        int run = kCoarse - 1 - 2 * hit;
        if (left > skipped + h0) {
          skipped += h0;
          --run;
        }
        const uint32_t* fine = &sm.hist[pass][run * 32];
        if (nr > 1) {
          if (tid < 32 * int(nr)) {
            const uint32_t v = peer_word(fine + lane, unsigned(warp));
            if (v) atomicAdd(&sm.row[kCoarse + lane], v);
          }
          __syncthreads();
          fine = sm.row + kCoarse;
        }
        if (warp == 0) {  // bins from the run's last down
          const uint32_t c = fine[31 - lane];
          uint32_t incl = c;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(kAll, incl, o);
            if (lane >= o) incl += u;
          }
          const uint32_t before = skipped + incl - c;
          if (before < left && left <= before + c) {
            sm.digit[pass] = uint32_t(run * 32 + 31 - lane);
            sm.above = before;
            sm.within = c;
          }
        }
      }
      __syncthreads();
      prefix |= sm.digit[pass] << shift;
      left -= sm.above;
      all_in = left == sm.within;
    }
    // `prefix` is the K-th largest weight: every greater key stays, and the first `left` equal ones; or, with
    // all_in, the least of its bin: every key from there on stays
    const uint32_t above = all_in ? prefix - 1 : prefix;  // (prefix > 0: no weight maps to the first bins)
    if (all_in) left = 0;
    uint32_t gt = 0, eq = 0;  // kept, and equal, before the chunk at work
    if (nr > 1) {
      // what the slices of the lower ranks hold follows from their own counts
      uint32_t mine = 0;
      for (int pass = 0; pass < passes; ++pass) {
        const uint32_t from = sm.digit[pass] + (all_in && pass == passes - 1 ? 0 : 1);
        for (uint32_t i = from + tid; i < kBins; i += kThreads) mine += sm.hist[pass][i];
      }
      mine = __reduce_add_sync(kAll, mine);
      if (lane == 0 && mine) atomicAdd(&sm.total_gt, mine);
      if (tid == 0 && !all_in) sm.total_eq = sm.hist[2][sm.digit[2]];
      __syncthreads();
      cluster_sync_all();
      for (unsigned q = 0; q < rank; ++q) {
        gt += peer_word(&sm.total_gt, q);
        eq += peer_word(&sm.total_eq, q);
      }
      cluster_arrive();  // this CTA reads no peer from here on; the wait below lets it go on or leave
    }
    // chunks of four positions a thread, in order: (greater, equal) counts packed in one word, added up over the
    // warp by shuffles and over the warps through shared memory
    for (int c0 = 0, par = 0; c0 < n; c0 += 4 * kThreads, par ^= 1) {
      const int i = c0 + 4 * tid;
      uint32_t x[4] = {0, 0, 0, 0};
      if (in_smem) {
        if (i < n) {
          const uint4 v = *reinterpret_cast<const uint4*>(keys + i);
          x[0] = v.x;
          x[1] = i + 1 < n ? v.y : 0u;
          x[2] = i + 2 < n ? v.z : 0u;
          x[3] = i + 3 < n ? v.w : 0u;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = fetch_one(i + e);
      }
      uint32_t mine = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) mine += (x[e] > above ? 1u : 0u) + (x[e] == above && !all_in ? 0x10000u : 0u);
      uint32_t incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(kAll, incl, o);
        if (lane >= o) incl += v;
      }
      if (lane == 31) sm.scan[par][warp] = incl;
      __syncthreads();
      const uint32_t w = lane < kWarps ? sm.scan[par][lane] : 0u;
      const uint32_t before = incl - mine + __reduce_add_sync(kAll, lane < warp ? w : 0u);
      const uint32_t all = __reduce_add_sync(kAll, w);
      uint32_t my_gt = gt + (before & 0xffffu), my_eq = eq + (before >> 16);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool is_gt = x[e] > above, is_eq = x[e] == above && !all_in;
        const uint32_t at = my_gt + min(left, my_eq);
        // (the bound holds unless the weights change meanwhile)
        if ((is_gt || (is_eq && my_eq < left)) && at < uint32_t(need)) kept[p.sink + at] = s0 + i + e;
        my_gt += is_gt;
        my_eq += is_eq;
      }
      gt += all & 0xffffu;
      eq += all >> 16;
    }
    if (missing > 0) {  // the recent keys move up behind the free ones; their first places were written before the barriers
      for (int i = rank * kThreads + tid; i < missing + p.recent; i += nr * kThreads)
        kept[p.sink + need - missing + i] = i < p.recent ? g.lkv - p.recent + i : -1;
    }
    if (nr > 1) cluster_wait();
    if (row + int(gridDim.x / nr) < rows) {  // a further row starts over
      __syncthreads();
      clear();
      __syncthreads();
    }
  }
}

// ---- compaction ----------------------------------------------------------------------------------
// Row j of the first n slots receives row kept[j] >= j.  Steps go up in j, and the rows of a step are
// written only when all rows up to that step have been read: a write of step s lands at or below its
// last j, every later step reads at or above that, so nothing is overwritten before it has been read, and
// the copy is safe in place, however far reads run ahead.  The bound is memory traffic: each moved row is
// read once and written once, so reads run three steps (96 KB a CTA) ahead through shared memory, and the
// positions and page ids of the steps behind those are fetched one and two steps earlier still.  (Read and
// written step by step from registers, each step waited for four dependent loads: 310 us for 64 x 8
// rows of 2048 keys, now 164, 0.97 of the copy rate.)  A cluster shares a task (request, head, K or V) when there are few
// of them; its barrier then orders a step's reads before its writes.
constexpr int kCmpThreads = 256;
constexpr int kCmpVecs = 8;    // 16-byte pieces of a thread and step
constexpr int kCmpAhead = 3;   // steps in flight
constexpr int kIdxRing = kCmpAhead + 2;

struct CompactSmem {
  uint4 data[kCmpAhead][kCmpVecs][kCmpThreads];
  int2 idx[kIdxRing][kCmpThreads];  // (source, destination) row of the page pool; source -1: the row stays
};

// Checks entry j of a kept list of n entries; -1 for one that stays, is out of range or is behind the end.
__device__ __forceinline__ int kept_source(const CompactParams& p, int j, int k, int prev, int lkv) {
  if (k < j || k >= lkv || k <= prev) {
    atomicOr(p.pv.err, FI_DEVERR_KEPT);
    return -1;
  }
  return k == j ? -1 : k;
}

// The running weights of one (request, head): rows of four bytes, through registers.
__device__ void compact_weights(const CompactParams& p, const Geo& g, const int32_t* kept, int head, unsigned nr,
                                unsigned rank) {
  const PageView& pv = p.pv;
  const int n = p.budget, step = kCmpThreads * kCmpVecs;
  for (int s0 = 0; s0 < n; s0 += int(nr) * step) {
    const int j0 = s0 + int(rank) * step + threadIdx.x;
    int src[kCmpVecs];
    float v[kCmpVecs];
#pragma unroll
    for (int i = 0; i < kCmpVecs; ++i) {
      const int j = j0 + i * kCmpThreads;
      src[i] = j < n ? kept_source(p, j, __ldg(kept + j), j > 0 ? __ldg(kept + j - 1) : -1, g.lkv) : -1;
    }
#pragma unroll
    for (int i = 0; i < kCmpVecs; ++i) {
      int page, slot;
      if (src[i] >= 0 && locate(pv, g.kv0, src[i], page, slot))
        v[i] = __ldcg(p.weights + weight_offset(pv, page, slot, head));
      else
        src[i] = -1;
    }
    if (nr > 1)
      cluster_sync_all();
    else
      __syncthreads();
#pragma unroll
    for (int i = 0; i < kCmpVecs; ++i) {
      int page, slot;
      if (src[i] >= 0 && locate(pv, g.kv0, j0 + i * kCmpThreads, page, slot))
        p.weights[weight_offset(pv, page, slot, head)] = v[i];
    }
  }
}

template <bool kFp8>
__global__ void __launch_bounds__(kCmpThreads, 2) compact_kernel(const __grid_constant__ CompactParams p) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  CompactSmem& sm = *reinterpret_cast<CompactSmem*>(smem_raw);
  wait_prior_grid();
  const PageView& pv = p.pv;
  constexpr int kLanes = kFp8 ? 8 : 16;            // threads of one row
  constexpr int kRowBytes = kFp8 ? kHeadDim : 2 * kHeadDim;
  constexpr int kRowsPass = kCmpThreads / kLanes;  // rows one piece of all threads covers
  constexpr int kRowsStep = kRowsPass * kCmpVecs;
  static_assert(kRowsStep <= kCmpThreads, "one thread looks a row up");
  const int batch = load_head(pv.geo).batch;
  const unsigned nr = cluster_size(), rank = cluster_rank();
  const int sub = threadIdx.x / kLanes, l = threadIdx.x % kLanes;
  const int kinds = p.weights ? 3 : 2;
  const int tasks = batch * pv.hkv * kinds;
  for (int task = blockIdx.x / nr; task < tasks; task += gridDim.x / nr) {
    const int which = task % kinds, row = task / kinds;
    const int r = row / pv.hkv, head = row - r * pv.hkv;
    const Geo g = load_geo(pv.geo, r);
    if (g.lkv <= p.budget) continue;  // nothing moves
    const int n = p.budget;
    const int32_t* kept = p.kept + (long long)row * p.budget;
    if (which == 2) {
      compact_weights(p, g, kept, head, nr, rank);
      continue;
    }
    uint8_t* pages = static_cast<uint8_t*>(which ? p.v_pages : p.k_pages) + 16 * l;
    const int stride = int(nr) * kRowsStep;
    const int steps = (n + stride - 1) / stride;
    const bool looks = threadIdx.x < kRowsStep;
    const int mine = int(rank) * kRowsStep + int(threadIdx.x);  // the row of step 0 that this thread looks up
    const int32_t* list = pv.kv_indices + g.kv0;
    // rows of the pool (128 elements each, so they fit 32 bits): per page, slot and head
    const int page_rows = int(pv.page_stride / kHeadDim), slot_rows = int(pv.tok_stride / kHeadDim),
              head_row = head * int(pv.head_stride / kHeadDim);
    auto page_of = [&](int j) { return pv.page_shift >= 0 ? j >> pv.page_shift : j / pv.page_size; };

    // look-up of a step's rows, in three parts, so that no part waits for its own loads
    int k1 = 0, k1_prev = 0, src2 = -1, src_page = -1, dst_page = -1;  // later step's entry; its page ids
    auto fetch_entry = [&](int step) {
      const int j = step * stride + mine;
      k1 = j;  // stays
      k1_prev = -1;
      if (looks && j < n) {
        k1 = __ldg(kept + j);
        if (j > 0) k1_prev = __ldg(kept + j - 1);
      }
    };
    auto fetch_pages = [&](int step) {
      const int j = step * stride + mine;
      src2 = j < n ? kept_source(p, j, k1, k1_prev, g.lkv) : -1;
      if (looks && src2 >= 0) {
        src_page = __ldg(list + page_of(src2));
        dst_page = __ldg(list + page_of(j));
      }
    };
    auto put_rows = [&](int step, int at) {
      if (!looks) return;
      int2 rows = make_int2(-1, 0);
      if (src2 >= 0) {
        if (unsigned(src_page) < unsigned(pv.num_pages) && unsigned(dst_page) < unsigned(pv.num_pages)) {
          const int j = step * stride + mine;
          rows.x = src_page * page_rows + (src2 - page_of(src2) * pv.page_size) * slot_rows + head_row;
          rows.y = dst_page * page_rows + (j - page_of(j) * pv.page_size) * slot_rows + head_row;
        } else {
          atomicOr(pv.err, FI_DEVERR_PAGE_OOB);
        }
      }
      sm.idx[at][threadIdx.x] = rows;
    };
    // rows that stay are copied too, as nothing (no bytes read, none written): no branch in between
    auto read = [&](int step, int at, int to) {
      if (step < steps) {
        int src[kCmpVecs];
#pragma unroll
        for (int i = 0; i < kCmpVecs; ++i) src[i] = sm.idx[at][i * kRowsPass + sub].x;
#pragma unroll
        for (int i = 0; i < kCmpVecs; ++i)
          cp_async_16_or_none(&sm.data[to][i][threadIdx.x], pages + (long long)max(src[i], 0) * kRowBytes, src[i] >= 0);
      }
      cp_async_commit();
    };
    auto write = [&](int at, int from) {
      int2 rows[kCmpVecs];
#pragma unroll
      for (int i = 0; i < kCmpVecs; ++i) rows[i] = sm.idx[at][i * kRowsPass + sub];
#pragma unroll
      for (int i = 0; i < kCmpVecs; ++i) {
        const uint4 v = sm.data[from][i][threadIdx.x];
        if (rows[i].x >= 0) *reinterpret_cast<uint4*>(pages + (long long)rows[i].y * kRowBytes) = v;
      }
    };
    __syncthreads();  // the last task's look-ups are not read any more
    {
      // the first steps' look-ups, side by side
      int k[kCmpAhead + 2], prev[kCmpAhead + 2];
#pragma unroll
      for (int i = 0; i < kCmpAhead + 2; ++i) {
        fetch_entry(i);
        k[i] = k1;
        prev[i] = k1_prev;
      }
      int s2[kCmpAhead + 2], sp[kCmpAhead + 2], dp[kCmpAhead + 2];
#pragma unroll
      for (int i = 0; i < kCmpAhead + 2; ++i) {
        k1 = k[i];
        k1_prev = prev[i];
        fetch_pages(i);
        s2[i] = src2;
        sp[i] = src_page;
        dp[i] = dst_page;
      }
      fetch_entry(kCmpAhead + 2);
#pragma unroll
      for (int i = 0; i < kCmpAhead + 2; ++i) {
        src2 = s2[i];
        src_page = sp[i];
        dst_page = dp[i];
        if (i <= kCmpAhead) put_rows(i, i);  // the last one stays in the registers, as the loop below expects it
      }
    }
    __syncthreads();
    for (int i = 0; i < kCmpAhead; ++i) read(i, i, i);
    if (nr > 1) {
      cp_async_wait<kCmpAhead - 1>();
      cluster_arrive_relaxed();
    }
    // places in the rings of the step at work, and of the look-ups of steps ahead of it
    int at = 0, at_read = kCmpAhead, at_put = kCmpAhead + 1, data = 0;
    for (int step = 0; step < steps; ++step) {
      if (nr > 1) {
        // everybody has read this step; say so of the next one, whose barrier then runs beside the writes
        cluster_wait();
        __syncthreads();
        cp_async_wait<kCmpAhead - 2>();
        cluster_arrive_relaxed();
      } else {
        cp_async_wait<kCmpAhead - 1>();
        __syncthreads();
      }
      // the look-ups of step + ahead + 1 go into the place of step - 1's
      put_rows(step + kCmpAhead + 1, at_put);
      fetch_pages(step + kCmpAhead + 2);
      fetch_entry(step + kCmpAhead + 3);
      write(at, data);
      read(step + kCmpAhead, at_read, data);
      at = at + 1 == kIdxRing ? 0 : at + 1;
      at_read = at_read + 1 == kIdxRing ? 0 : at_read + 1;
      at_put = at_put + 1 == kIdxRing ? 0 : at_put + 1;
      data = data + 1 == kCmpAhead ? 0 : data + 1;
    }
    if (nr > 1) cluster_wait();
    cp_async_wait<0>();
  }
}

}  // namespace

int launch_select(SelectParams p, int batch, int most_batch, int max_lkv, int num_sms, cudaStream_t stream) {
  if (batch == 0) batch = most_batch;  // captured on an empty plan
  const int rows = batch * p.pv.hkv;
  p.by_four = p.pv.page_size % 4 == 0 && reinterpret_cast<uintptr_t>(p.weights) % 16 == 0;
  // a cluster shares a row while there are SMs for it (131 K keys of 8 heads: 8 CTAs 17.8 us), or as long as a slice does
  // not fit into shared memory and would be read again in each pass (16 x 8 rows of 100 K keys: 81 us, 121 without)
  unsigned cluster = 1;
  while (cluster < 8 && ((int64_t(rows) * cluster * 2 <= num_sms && max_lkv / int(cluster) > 4096) ||
                         max_lkv / int(cluster) > 48 * 1024 - 64))
    cluster *= 2;
  const int64_t want = (int64_t(max_lkv) / cluster + 64 + 31) / 32 * 32;
  const int cap = int(std::min<int64_t>(want, 48 * 1024));
  const size_t smem = size_t(cap) * 4;
  static std::once_flag once;
  static cudaError_t attr = cudaSuccess;
  std::call_once(once, [] {
    attr = cudaFuncSetAttribute(select_kernel<256>, cudaFuncAttributeMaxDynamicSharedMemorySize, 48 * 1024 * 4);
    if (attr == cudaSuccess)
      attr = cudaFuncSetAttribute(select_kernel<1024>, cudaFuncAttributeMaxDynamicSharedMemorySize, 48 * 1024 * 4);
  });
  if (attr != cudaSuccess) return record_cuda_error(attr, "cudaFuncSetAttribute(select_kernel)");
  // short rows take 256 threads, six to an SM up to 2900 keys and five to 4096; long ones, and clusters, 1024
  const bool wide = cluster > 1 || max_lkv > 4096;
  // rows of later plans of a captured launch: CTAs that fit the GPU at once, and that do nothing otherwise
  const int64_t later = std::min<int64_t>(int64_t(most_batch) * p.pv.hkv, std::max(1, wide ? num_sms / int(cluster) : 4 * num_sms));
  const unsigned grid = unsigned(std::max(std::min<int64_t>(rows, 4 * num_sms), later)) * cluster;
  const cudaError_t e = wide ? launch_dependent(select_kernel<1024>, grid, 1024, smem, cluster, stream, p, cap)
                             : launch_dependent(select_kernel<256>, grid, 256, smem, cluster, stream, p, cap);
  return e == cudaSuccess ? 0 : record_cuda_error(e, "select_kernel launch");
}

int launch_compact(const CompactParams& p, int batch, int most_batch, bool fp8, int num_sms, cudaStream_t stream) {
  if (batch == 0) batch = most_batch;  // captured on an empty plan
  const int64_t of_one = int64_t(p.pv.hkv) * (p.weights ? 3 : 2), tasks = batch * of_one;
  unsigned cluster = 1;
  while (cluster < 8 && tasks * cluster * 2 <= 2 * num_sms) cluster *= 2;
  static std::once_flag once;
  static cudaError_t attr = cudaSuccess;
  std::call_once(once, [] {
    attr = cudaFuncSetAttribute(compact_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(sizeof(CompactSmem)));
    if (attr == cudaSuccess)
      attr = cudaFuncSetAttribute(compact_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(sizeof(CompactSmem)));
  });
  if (attr != cudaSuccess) return record_cuda_error(attr, "cudaFuncSetAttribute(compact_kernel)");
  // as above; of clusters fewer than two CTAs an SM find room at once (38 clusters of 8: 145 us where 24 take 124)
  const int64_t later = std::min<int64_t>(most_batch * of_one, cluster > 1 ? std::max(1, num_sms / int(cluster)) : 2 * num_sms);
  const unsigned grid = unsigned(std::max(std::min<int64_t>(tasks, 64 * num_sms), later)) * cluster;
  const size_t smem = sizeof(CompactSmem);
  const cudaError_t e = fp8 ? launch_dependent(compact_kernel<true>, grid, kCmpThreads, smem, cluster, stream, p)
                            : launch_dependent(compact_kernel<false>, grid, kCmpThreads, smem, cluster, stream, p);
  return e == cudaSuccess ? 0 : record_cuda_error(e, "compact_kernel launch");
}

}  // namespace fi
