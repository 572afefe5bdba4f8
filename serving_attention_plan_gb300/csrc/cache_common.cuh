// Device helpers shared by the cache operators.
#pragma once

#include "cache_ops.h"
#include "device_common.cuh"
#include "plan.h"

namespace fi {

// Set-up may overlap the previous kernel on the stream (programmatic dependent launch); of global memory only the plan may be read before
// it has completed (a copy of the plan is no kernel, so a launch behind it waits for all of it), and followers are let go only after that.
__device__ __forceinline__ void wait_prior_grid() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <typename K, typename... A>
inline cudaError_t launch_dependent(K kernel, unsigned grid, unsigned threads, size_t smem, unsigned cluster,
                                    cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Last request whose `field` (non-decreasing over requests) is <= x; n >= 1 and the first request's
// field is <= x.  A whole warp calls it: 32 probes a round, so two rounds for up to 1024 requests.
__device__ __forceinline__ int find_request(const Geo* geo, int n, int32_t Geo::*field, int x) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) >> 5;
    const int at = lo + lane * step;
    const unsigned le = __ballot_sync(0xffffffffu, at < hi && __ldg(&(geo[min(at, n - 1)].*field)) <= x);
    lo += (__popc(le) - 1) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

__device__ __forceinline__ Geo load_geo(const Geo* geo, int r) {
  const int4 a = __ldg(reinterpret_cast<const int4*>(geo + r));
  const int4 b = __ldg(reinterpret_cast<const int4*>(geo + r) + 1);
  return Geo{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}

__device__ __forceinline__ GeoHead load_head(const Geo* geo) {
  const int4 a = __ldg(reinterpret_cast<const int4*>(geo) - 2);
  const int4 b = __ldg(reinterpret_cast<const int4*>(geo) - 1);
  return GeoHead{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}

// Page id and slot of key j of the request whose page list starts at kv0; false (with the error bit
// set) for a page outside the pool.
__device__ __forceinline__ bool locate(const PageView& pv, int kv0, int j, int& page, int& slot) {
  const int e = pv.page_shift >= 0 ? j >> pv.page_shift : j / pv.page_size;
  slot = j - e * pv.page_size;
  page = __ldg(pv.kv_indices + kv0 + e);
  if (static_cast<unsigned>(page) < static_cast<unsigned>(pv.num_pages)) return true;
  atomicOr(pv.err, FI_DEVERR_PAGE_OOB);
  return false;
}

// tanh(y) / y as the first terms of its series in u = y^2: 1e-8 relative up to kNearReach (|y| = 1/4).
constexpr float kNearReach = 0.0625f;
__device__ __forceinline__ float2 tanh_near_factor(float2 u) {
  constexpr float c[5] = {1.f, -1.f / 3.f, 2.f / 15.f, -17.f / 315.f, 62.f / 2835.f};
  float2 t = make_float2(c[4], c[4]);
#pragma unroll
  for (int i = 3; i >= 0; --i) t = __ffma2_rn(t, u, make_float2(c[i], c[i]));
  return t;
}

// 16 bytes global -> shared, or nothing (the source is not read, the destination gets zeros).
__device__ __forceinline__ void cp_async_16_or_none(void* dst_smem, const void* src_gmem, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst_smem)), "l"(src_gmem), "r"(on ? 16 : 0)
               : "memory");
}

__device__ __forceinline__ long long kv_offset(const PageView& pv, int page, int slot, int head) {
  return page * pv.page_stride + head * pv.head_stride + slot * pv.tok_stride;
}
__device__ __forceinline__ long long weight_offset(const PageView& pv, int page, int slot, int head) {
  return ((long long)page * pv.hkv + head) * pv.page_size + slot;
}

}  // namespace fi
