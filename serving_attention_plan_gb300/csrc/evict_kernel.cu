// Selection of the keys to keep, and their compaction, per (request, KV head).
#include <algorithm>
#include <mutex>

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
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
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
// change the result.  The kept positions come out ascending by ranking (greater, equal) counts over
// the range in order.  Weights are read from memory once (the slice of the range that a CTA owns
// stays in shared memory); a cluster of CTAs shares a row when there are few rows.
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;

struct SelectSmem {
  uint32_t hist[3][kBins];
  uint32_t warp_gt[kSelWarps], warp_eq[kSelWarps];
  uint32_t total_gt, total_eq;  // of this CTA's slice
  uint32_t digit, above;        // result of a pass
};

// Order-preserving map; -0 counts as 0 and every NaN as the largest.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kSelThreads) select_kernel(const __grid_constant__ SelectParams p, int cap) {
  extern __shared__ uint32_t keys[];  // [cap]: the CTA's slice of the row
  __shared__ SelectSmem sm;
  wait_prior_grid();
  const PageView& pv = p.pv;
  const int batch = __ldg(pv.header + H_BATCH);
  const unsigned nr = cluster_size(), rank = cluster_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rows = batch * pv.hkv;
  for (int row = blockIdx.x / nr; row < rows; row += gridDim.x / nr) {
    const int r = row / pv.hkv, head = row - r * pv.hkv;
    const Geo g = load_geo(pv.geo, r);
    int32_t* kept = p.kept + (long long)row * p.budget;
    if (g.lkv <= p.budget) {
      for (int i = rank * kSelThreads + tid; i < p.budget; i += nr * kSelThreads) kept[i] = i < g.lkv ? i : -1;
      continue;  // the same for every CTA of the cluster
    }
    const int f0 = p.sink, f1 = g.lkv - p.recent;
    const int need = p.budget - p.sink - p.recent;
    for (int i = rank * kSelThreads + tid; i < p.sink + p.recent; i += nr * kSelThreads) {
      if (i < p.sink)
        kept[i] = i;
      else
        kept[p.budget - p.recent + i - p.sink] = g.lkv - p.recent + i - p.sink;
    }
    if (need == 0) continue;
    // this CTA's slice, a multiple of a warp's step so that warps own whole steps
    const int per = (((f1 - f0 + int(nr) - 1) / int(nr)) + 31) & ~31;
    const int s0 = min(f1, f0 + int(rank) * per), s1 = min(f1, s0 + per);
    const int n = s1 - s0;
    const bool in_smem = n <= cap;
    auto fetch = [&](int i) -> uint32_t {  // key i of the slice, from memory
      int page, slot;
      if (!locate(pv, g.kv0, s0 + i, page, slot)) return 0u;
      return order_key(__ldg(p.weights + weight_offset(pv, page, slot, head)));
    };
    for (int i = tid; i < 3 * kBins; i += kSelThreads) (&sm.hist[0][0])[i] = 0;
    if (in_smem)
      for (int i = tid; i < n; i += kSelThreads) keys[i] = fetch(i);
    auto key = [&](int i) { return in_smem ? keys[i] : fetch(i); };
    __syncthreads();

    uint32_t prefix = 0;  // the digits found so far, in place
    uint32_t left = uint32_t(need);
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t mask = pass == 2 ? 1023u : 2047u;
      const uint32_t known = pass == 0 ? 0u : pass == 1 ? 0xffe00000u : 0xfffffc00u;
      for (int i = tid; i < n; i += kSelThreads) {
        const uint32_t x = key(i);
        if ((x & known) == prefix) atomicAdd(&sm.hist[pass][(x >> shift) & mask], 1u);
      }
      __syncthreads();
      if (nr > 1) cluster_sync_all();
      // thread t sums the row's counts of 4 bins, highest bins first
      uint32_t c[kBins / kSelThreads], mine = 0;
#pragma unroll
      for (int k = 0; k < kBins / kSelThreads; ++k) {
        const int bin = kBins - 1 - (tid * (kBins / kSelThreads) + k);
        uint32_t v = 0;
        if (nr == 1)
          v = sm.hist[pass][bin];
        else
          for (unsigned q = 0; q < nr; ++q) v += peer_word(&sm.hist[pass][bin], q);
        c[k] = v;
        mine += v;
      }
      uint32_t incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(kAll, incl, o);
        if (lane >= o) incl += v;
      }
      if (lane == 31) sm.warp_gt[warp] = incl;
      __syncthreads();
      uint32_t before = incl - mine;
      for (int w = 0; w < warp; ++w) before += sm.warp_gt[w];
#pragma unroll
      for (int k = 0; k < kBins / kSelThreads; ++k) {
        if (before < left && left <= before + c[k]) {
          sm.digit = uint32_t(kBins - 1 - (tid * (kBins / kSelThreads) + k));
          sm.above = before;
        }
        before += c[k];
      }
      __syncthreads();
      prefix |= sm.digit << shift;
      left -= sm.above;
      __syncthreads();
    }
    // `prefix` is the K-th largest weight; every greater key stays, and the first `left` equal ones.
    // Warps own consecutive steps of 32 keys.
    const int steps = (n + 31) >> 5;
    const int w0 = steps * warp / kSelWarps, w1 = steps * (warp + 1) / kSelWarps;
    uint32_t gt = 0, eq = 0;
    for (int st = w0; st < w1; ++st) {
      const int i = st * 32 + lane;
      const uint32_t x = i < n ? key(i) : 0u;
      gt += __popc(__ballot_sync(kAll, i < n && x > prefix));
      eq += __popc(__ballot_sync(kAll, i < n && x == prefix));
    }
    if (lane == 0) {
      sm.warp_gt[warp] = gt;
      sm.warp_eq[warp] = eq;
    }
    __syncthreads();
    if (tid == 0) {
      uint32_t a = 0, b = 0;
      for (int w = 0; w < kSelWarps; ++w) {
        a += sm.warp_gt[w];
        b += sm.warp_eq[w];
      }
      sm.total_gt = a;
      sm.total_eq = b;
    }
    __syncthreads();
    if (nr > 1) cluster_sync_all();
    gt = eq = 0;
    for (unsigned q = 0; q < rank; ++q) {
      gt += peer_word(&sm.total_gt, q);
      eq += peer_word(&sm.total_eq, q);
    }
    for (int w = 0; w < warp; ++w) {
      gt += sm.warp_gt[w];
      eq += sm.warp_eq[w];
    }
    const uint32_t below = (1u << lane) - 1u;
    for (int st = w0; st < w1; ++st) {
      const int i = st * 32 + lane;
      const uint32_t x = i < n ? key(i) : 0u;
      const unsigned bg = __ballot_sync(kAll, i < n && x > prefix), be = __ballot_sync(kAll, i < n && x == prefix);
      const uint32_t eq_before = eq + __popc(be & below);
      const bool keep = ((bg >> lane) & 1u) || (((be >> lane) & 1u) && eq_before < left);
      if (keep) kept[p.sink + gt + __popc(bg & below) + min(left, eq_before)] = s0 + i;
      gt += __popc(bg);
      eq += __popc(be);
    }
    // peers may still read this CTA's totals and counts; the next row overwrites them
    __syncthreads();
    if (nr > 1) cluster_sync_all();
  }
}

// ---- compaction ----------------------------------------------------------------------------------
// Row j of the first n slots receives row kept[j] >= j.  Steps go up in j, and within a step every
// row is read before any is written: a write of step s lands at or below its last j, every later
// step reads at or above that, so nothing is overwritten before it has been read, and the copy is
// safe in place.  The bound is memory traffic: each moved row is read once and written once.  Rows
// live in registers between the two halves of a step.  A cluster shares one (request, head, K or V) when there are few of them; its
// barrier then orders the step's reads before its writes.
constexpr int kCmpThreads = 256;
constexpr int kCmpVecs = 8;  // 16-byte pieces a thread carries

template <bool kFp8>
__global__ void __launch_bounds__(kCmpThreads) compact_kernel(const __grid_constant__ CompactParams p) {
  wait_prior_grid();
  const PageView& pv = p.pv;
  constexpr int kLanes = kFp8 ? 8 : 16;                         // threads of one row
  constexpr int kRowsPass = kCmpThreads / kLanes;               // rows one piece of all threads covers
  constexpr int kRowsStep = kRowsPass * kCmpVecs;
  const int batch = __ldg(pv.header + H_BATCH);
  const unsigned nr = cluster_size(), rank = cluster_rank();
  const int sub = threadIdx.x / kLanes, l = threadIdx.x % kLanes;
  const int tasks = batch * pv.hkv * 2;
  for (int task = blockIdx.x / nr; task < tasks; task += gridDim.x / nr) {
    const int which = task & 1, row = task >> 1;
    const int r = row / pv.hkv, head = row - r * pv.hkv;
    const Geo g = load_geo(pv.geo, r);
    if (g.lkv <= p.budget) continue;  // nothing moves
    const int n = p.budget;
    const int32_t* kept = p.kept + (long long)row * p.budget;
    uint8_t* pages = static_cast<uint8_t*>(which ? p.v_pages : p.k_pages);
    float* weights = which ? nullptr : p.weights;
    const int stride = int(nr) * kRowsStep;

    uint4 v[kCmpVecs];
    float wv[kCmpVecs];
    int src[kCmpVecs];  // -1: row stays or is out of range
    auto read = [&](int j0) {
#pragma unroll
      for (int i = 0; i < kCmpVecs; ++i) {
        const int j = j0 + i * kRowsPass + sub;
        src[i] = -1;
        if (j < n) {
          const int k = __ldg(kept + j);
          const int prev = j > 0 ? __ldg(kept + j - 1) : -1;
          if (k < j || k >= g.lkv || k <= prev)
            atomicOr(pv.err, FI_DEVERR_KEPT);
          else if (k != j)
            src[i] = k;
        }
      }
#pragma unroll
      for (int i = 0; i < kCmpVecs; ++i) {
        int page, slot;
        if (src[i] < 0) continue;
        if (!locate(pv, g.kv0, src[i], page, slot)) {
          src[i] = -1;
          continue;
        }
        const uint8_t* at = pages + kv_offset(pv, page, slot, head) * (kFp8 ? 1 : 2) + 16 * l;
        v[i] = __ldcg(reinterpret_cast<const uint4*>(at));
        if (weights && l == 0) wv[i] = __ldcg(weights + weight_offset(pv, page, slot, head));
      }
    };
    auto write = [&](int j0) {
#pragma unroll
      for (int i = 0; i < kCmpVecs; ++i) {
        int page, slot;
        if (src[i] < 0 || !locate(pv, g.kv0, j0 + i * kRowsPass + sub, page, slot)) continue;
        uint8_t* at = pages + kv_offset(pv, page, slot, head) * (kFp8 ? 1 : 2) + 16 * l;
        *reinterpret_cast<uint4*>(at) = v[i];
        if (weights && l == 0) weights[weight_offset(pv, page, slot, head)] = wv[i];
      }
    };
    for (int s0 = 0; s0 < n; s0 += stride) {
      const int j0 = s0 + int(rank) * kRowsStep;
      read(j0);
      if (nr > 1)
        cluster_sync_all();
      else
        __syncthreads();
      write(j0);
    }
  }
}

}  // namespace

int launch_select(const SelectParams& p, int batch, int max_lkv, int num_sms, cudaStream_t stream) {
  const int rows = batch * p.pv.hkv;
  unsigned cluster = 1;
  while (cluster < 8 && rows * int(cluster) * 2 <= num_sms && max_lkv / int(cluster) > 4096) cluster *= 2;
  const int64_t want = (int64_t(max_lkv) / cluster + 64 + 31) / 32 * 32;
  const int cap = int(std::min<int64_t>(want, 48 * 1024));
  const size_t smem = size_t(cap) * 4;
  static std::once_flag once;
  static cudaError_t attr = cudaSuccess;
  std::call_once(once, [] {
    attr = cudaFuncSetAttribute(select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 48 * 1024 * 4);
  });
  if (attr != cudaSuccess) return record_cuda_error(attr, "cudaFuncSetAttribute(select_kernel)");
  const unsigned grid = unsigned(std::min<int64_t>(rows, 4 * num_sms)) * cluster;
  const cudaError_t e = launch_dependent(select_kernel, grid, kSelThreads, smem, cluster, stream, p, cap);
  return e == cudaSuccess ? 0 : record_cuda_error(e, "select_kernel launch");
}

int launch_compact(const CompactParams& p, int batch, bool fp8, int num_sms, cudaStream_t stream) {
  const int64_t tasks = int64_t(batch) * p.pv.hkv * 2;
  unsigned cluster = 1;
  while (cluster < 8 && tasks * cluster * 2 <= num_sms) cluster *= 2;
  const unsigned grid = unsigned(std::min<int64_t>(tasks, 16 * num_sms)) * cluster;
  const cudaError_t e = fp8 ? launch_dependent(compact_kernel<true>, grid, kCmpThreads, 0, cluster, stream, p)
                            : launch_dependent(compact_kernel<false>, grid, kCmpThreads, 0, cluster, stream, p);
  return e == cudaSuccess ? 0 : record_cuda_error(e, "compact_kernel launch");
}

}  // namespace fi
