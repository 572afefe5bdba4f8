// Append: per-head RMS norm of q and k, rotary position, q to the dense query tensor, K and V into
// the plan's page slots, in one pass.
//
//   y = x / sqrt(mean(x^2) + eps) * w          (only with a weight)
//   (a, b) -> (a cos pf - b sin pf, a sin pf + b cos pf)   for the pair of frequency f at position p
//
// Every element is read once and written once, so the bound is memory traffic (and, for a decode
// step, the launch).  Half a warp owns one (token, head) row: 16 lanes x 8 dims, one 16-byte load
// and one store a lane; the norm is four shuffles, the partner of a rotated half sits
// rotary / 16 lanes away.  The angles of a token are computed once, by the warp that also finds the
// token's page slot, and shared by all its heads through shared memory: computed per head they
// would cost more issue slots than the rest of the row.
//
// Angles: a position times a frequency is taken in turns as a 64-bit fraction, p * F mod 2^64 with
// F = round(2^64 frac(f / 2 pi)): whole turns drop out exactly in the integer product, so the angle
// is right to 2^-33 turns + the rounding of F (p * 2^-65) at any position, where a 32-bit product
// loses the angle itself beyond some ten thousand positions.
#include <cuda_fp8.h>

#include "cache_common.cuh"
#include "prefill_launch.h"

namespace fi {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kHalfWarps = kAppendThreads / 16;
constexpr int kInFlight = 4;  // rows a half-warp has in flight

struct TokenPlace {
  long long off;  // element offset of KV head 0 in the pages, -1: no slot
};

__device__ __forceinline__ void unpack8(uint4 w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = bf16x2_to_f2(u[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(f2_to_bf16x2(x[0], x[1]), f2_to_bf16x2(x[2], x[3]), f2_to_bf16x2(x[4], x[5]),
                    f2_to_bf16x2(x[6], x[7]));
}

__device__ __forceinline__ uint2 pack8_e4m3(const float (&x)[8], float s) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i] * s, x[2 * i + 1] * s), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// kTok tokens a step: four for long batches (the sync and the request search are paid once for four
// tokens), one for decode steps, where tokens are few and each CTA should take one.
template <int kTok, bool kFp8>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendParams p) {
  // [parity][cos, sin][token][64]: frequency f of split pairs lies at 4 * (((f >> 2) & 1) * 8 + (f >> 3)) + (f & 3),
  // so the lanes' 16-byte reads fall into different banks; interleaved pairs are in order
  __shared__ float4 trig[2][2][kTok][16];
  __shared__ TokenPlace place[2][kTok];
  wait_prior_grid();
  const PageView& pv = p.pv;
  const int batch = __ldg(pv.header + H_BATCH);
  if (batch == 0) return;
  const int total = __ldg(&pv.geo[batch].q0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hw = threadIdx.x >> 4, l = threadIdx.x & 15;  // half-warp, lane in it
  const int heads = p.hqo + 2 * pv.hkv;
  const int half = p.rotary >> 1;  // frequencies
  const int hl = p.rotary >> 4;    // lanes of one rotated half
  // the lane's partner in the rotation of split halves (itself outside the rotated dims)
  const int partner = l < hl ? l + hl : (l < 2 * hl ? l - hl : l);
  uint4 wq = make_uint4(0, 0, 0, 0), wk = wq;
  if (p.q_weight) wq = __ldg(reinterpret_cast<const uint4*>(p.q_weight) + l);
  if (p.k_weight) wk = __ldg(reinterpret_cast<const uint4*>(p.k_weight) + l);
  uint64_t f0 = 0, f1 = 0;  // the lane's two frequencies
  if (warp < kTok) {
    if (lane < half) f0 = p.freq[lane];
    if (lane + 32 < half) f1 = p.freq[lane + 32];
  }

  auto src = [&](int row, int base) -> const uint4* {  // row of the step -> its 16 bytes
    const int t = row / heads, h = row - t * heads;
    const long long tok = base + t;
    const __nv_bfloat16* at;
    if (h < p.hqo)
      at = static_cast<const __nv_bfloat16*>(p.q) + tok * p.q_stride + h * kHeadDim;
    else if (h < p.hqo + pv.hkv)
      at = static_cast<const __nv_bfloat16*>(p.k) + tok * p.k_stride + (h - p.hqo) * kHeadDim;
    else
      at = static_cast<const __nv_bfloat16*>(p.v) + tok * p.v_stride + (h - p.hqo - pv.hkv) * kHeadDim;
    return reinterpret_cast<const uint4*>(at) + l;
  };

  int par = 0;
  for (int base = blockIdx.x * kTok; base < total; base += gridDim.x * kTok, par ^= 1) {
    const int rows = min(kTok, total - base) * heads;
    uint4 raw[kInFlight];
#pragma unroll
    for (int i = 0; i < kInFlight; ++i) {
      const int row = hw + i * kHalfWarps;
      if (row < rows) raw[i] = *src(row, base);
    }
    if (warp < kTok && base + warp < total) {
      const int tok = base + warp;
      const int r = find_request(pv.geo, batch, &Geo::q0, tok);
      const Geo g = load_geo(pv.geo, r);
      const int j = g.lkv - g.lq + tok - g.q0;
      const int pos = p.positions ? __ldg(p.positions + tok) : j;
      if (lane == 0) {
        long long off = -1;
        int page, slot;
        if (j >= 0 && locate(pv, g.kv0, j, page, slot)) off = kv_offset(pv, page, slot, 0);
        place[par][warp].off = off;
      }
      float* c = reinterpret_cast<float*>(trig[par][0][warp]);
      float* s = reinterpret_cast<float*>(trig[par][1][warp]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int f = lane + 32 * i;
        if (f < half) {
          const int32_t turn = int32_t(uint32_t((uint64_t(int64_t(pos)) * (i ? f1 : f0)) >> 32));
          float sn, cs;
          sincospif(float(turn) * 0x1p-31f, &sn, &cs);
          const int at = p.interleaved ? f : 4 * (((f >> 2) & 1) * 8 + (f >> 3)) + (f & 3);
          c[at] = cs;
          s[at] = sn;
        }
      }
    }
    __syncthreads();
    for (int row0 = hw; row0 < rows; row0 += kInFlight * kHalfWarps) {
      if (row0 != hw) {
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) {
          const int row = row0 + i * kHalfWarps;
          if (row < rows) raw[i] = *src(row, base);
        }
      }
#pragma unroll
      for (int i = 0; i < kInFlight; ++i) {
        const int row = row0 + i * kHalfWarps;
        // both halves of a warp go through the shuffles, whether or not their row is there
        const bool on = row < rows;
        const int t = on ? row / heads : 0, h = on ? row - t * heads : 0;
        const bool is_q = h < p.hqo, is_v = h >= p.hqo + pv.hkv;
        const void* wgt = is_v ? nullptr : (is_q ? p.q_weight : p.k_weight);
        float x[8];
        unpack8(on ? raw[i] : make_uint4(0, 0, 0, 0), x);
        if (p.q_weight || p.k_weight) {
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          if (wgt) {
            const float inv = 1.f / sqrtf(ss * (1.f / kHeadDim) + p.eps);
            float w[8];
            unpack8(is_q ? wq : wk, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = x[e] * inv * w[e];
          }
        }
        if (half > 0) {
          if (p.interleaved) {
            if (!is_v && l < 2 * hl) {
              const float4 c = trig[par][0][t][l], s = trig[par][1][t][l];
              const float cc[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float a = x[2 * e], b = x[2 * e + 1];
                x[2 * e] = a * cc[e] - b * sn[e];
                x[2 * e + 1] = a * sn[e] + b * cc[e];
              }
            }
          } else {
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = __shfl_sync(0xffffffffu, x[e], partner, 16);
            if (!is_v && l < 2 * hl) {
              const int k = l < hl ? l : l - hl;
              const float sign = l < hl ? -1.f : 1.f;
#pragma unroll
              for (int q4 = 0; q4 < 2; ++q4) {
                const float4 c = trig[par][0][t][q4 * 8 + k], s = trig[par][1][t][q4 * 8 + k];
                const float cc[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) x[4 * q4 + e] = x[4 * q4 + e] * cc[e] + sign * sn[e] * y[4 * q4 + e];
              }
            }
          }
        }
        if (!on) continue;
        if (is_q) {
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.q_out) + ((long long)(base + t) * p.hqo + h) * kHeadDim;
          reinterpret_cast<uint4*>(dst)[l] = pack8(x);
          continue;
        }
        const long long off0 = place[par][t].off;
        if (off0 < 0) continue;
        const long long off = off0 + (is_v ? h - p.hqo - pv.hkv : h - p.hqo) * pv.head_stride + 8 * l;
        void* pages = is_v ? p.v_pages : p.k_pages;
        if constexpr (kFp8)
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(pages) + off) =
              pack8_e4m3(x, is_v ? p.v_inv_scale : p.k_inv_scale);
        else
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(pages) + off) = pack8(x);
      }
    }
  }
}

}  // namespace

int launch_append(const AppendParams& p, int total_q, bool fp8, int num_sms, cudaStream_t stream) {
  const bool many = total_q >= 8 * num_sms;
  const unsigned grid = unsigned(many ? min((total_q + 3) / 4, 8 * num_sms) : total_q);
  cudaError_t e;
  if (many)
    e = fp8 ? launch_dependent(append_kernel<4, true>, grid, kAppendThreads, 0, 1, stream, p)
            : launch_dependent(append_kernel<4, false>, grid, kAppendThreads, 0, 1, stream, p);
  else
    e = fp8 ? launch_dependent(append_kernel<1, true>, grid, kAppendThreads, 0, 1, stream, p)
            : launch_dependent(append_kernel<1, false>, grid, kAppendThreads, 0, 1, stream, p);
  return e == cudaSuccess ? 0 : record_cuda_error(e, "append_kernel launch");
}

}  // namespace fi
