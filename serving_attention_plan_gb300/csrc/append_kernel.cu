// Append: per-head RMS norm of q and k, rotary position, q to the dense query tensor, K and V into
// the plan's page slots, in one pass.
//
//   y = x / sqrt(mean(x^2) + eps) * w          (only with a weight)
//   (a, b) -> (a cos pf - b sin pf, a sin pf + b cos pf)   for the pair of frequency f at position p
//
// Every element is read once and written once, so the bound is memory traffic (and, for a decode
// step, the launch).  Eight lanes own one (token, head) row, two 16-byte pieces each, chosen so that the
// two halves of a rotated pair lie in one lane: piece l and piece l + rotary / 16.  The norm is three
// shuffles, the rotation none, and all arithmetic is packed two by two.  (With 16 lanes of one piece, the
// partner's values fetched by shuffles, the issue slots bound it: 250 us for 26 K tokens of 32/8
// heads.  With one pass in flight in registers each pass waited for its own load: 125 us; now 110, 5.8 TB/s,
// 0.86 of the copy rate, and 4 % less without norm and rotation.)  The angles of a token are computed once, by the warp that also finds its page slot,
// one step ahead of the rows, and shared by all its heads through shared memory.
//
// Angles: a position times a frequency is taken in turns as a 64-bit fraction, p * F mod 2^64 with
// F = 2^64 frac(f / 2 pi): whole turns drop out exactly in the integer product.  What is left is the rounding of
// the product's upper half to 24 bits (2^-26 turns) and that of F, a quotient of doubles (p * 2^-55 turns for
// f <= 1: as much again at p = 2^29), where a 32-bit product loses the angle itself beyond some ten thousand positions.
#include <cuda_fp8.h>

#include <algorithm>
#include <mutex>

#include "cache_common.cuh"
#include "prefill_launch.h"

namespace fi {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kRowLanes = 8;
constexpr int kAppendCtasPerSm = 2;
// Passes in flight of a group: 96 KB a CTA for warps, a decode token's two or three for a whole CTA.
template <int kGroup>
constexpr int kPassesAhead = kGroup == 32 ? 12 : 3;

__device__ __forceinline__ void unpack8(uint4 w, float2 (&x)[4]) {
  x[0] = bf16x2_to_f2(w.x);
  x[1] = bf16x2_to_f2(w.y);
  x[2] = bf16x2_to_f2(w.z);
  x[3] = bf16x2_to_f2(w.w);
}

__device__ __forceinline__ uint4 pack8(const float2 (&x)[4]) {
  return make_uint4(f2_to_bf16x2(x[0].x, x[0].y), f2_to_bf16x2(x[1].x, x[1].y), f2_to_bf16x2(x[2].x, x[2].y),
                    f2_to_bf16x2(x[3].x, x[3].y));
}

__device__ __forceinline__ uint2 pack8_e4m3(const float2 (&x)[4], float s) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = __nv_cvt_float2_to_fp8x2(__fmul2_rn(x[i], make_float2(s, s)), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// 8 elements at element offset `off` of the pages.
template <bool kFp8>
__device__ __forceinline__ void put8(void* pages, long long off, const float2 (&x)[4], float inv_scale) {
  if constexpr (kFp8)
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(pages) + off) = pack8_e4m3(x, inv_scale);
  else
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(pages) + off) = pack8(x);
}

// Threads work in groups that take one token at a time: a warp for long batches, the whole CTA for decode steps,
// where tokens are few and a token's rows should go side by side.  A pass of a group is kGroup / 8 rows;
// kPassesAhead passes are in flight, across tokens, each lane's own 32 bytes of them by asynchronous copies
// into a ring of its own (in registers the ring spilled, and a spill waits for its load).
template <int kGroup, bool kFp8>
__global__ void __launch_bounds__(kAppendThreads, kAppendCtasPerSm) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kGroups = kAppendThreads / kGroup, kRowsPass = kGroup / kRowLanes, kDepth = kPassesAhead<kGroup>;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  uint4(*ring)[2][kAppendThreads] = reinterpret_cast<uint4(*)[2][kAppendThreads]>(smem_raw);  // [kDepth]
  // cos and sin of a token's frequencies: piece k of a split half holds frequencies 8 k .. 8 k + 7, its first
  // four at [k], the others at [8 + k], so the lanes' 16-byte reads fall into different banks; interleaved
  // pairs are in order, piece k holds [k]
  __shared__ float4 cosines[kGroups][2][16], sines[kGroups][2][16];
  __shared__ long long place[kGroups][2];  // element offset of KV head 0 in the pages, -1: no slot
  __shared__ uint4 norm_weight[2][16];     // of q and k
  wait_prior_grid();
  const PageView& pv = p.pv;
  const GeoHead plan = load_head(pv.geo);
  const int batch = plan.batch, total = plan.total_q;
  if (batch == 0) return;
  const int lane = threadIdx.x & 31, l = threadIdx.x % kRowLanes;
  const int group = threadIdx.x / kGroup, sub = threadIdx.x % kGroup / kRowLanes;
  const bool leads = threadIdx.x % kGroup < 32;  // the group's first warp looks slots and angles up
  auto sync = [&]() {
    if constexpr (kGroup == 32)
      __syncwarp();
    else
      __syncthreads();
  };
  const int half = p.rotary >> 1;  // frequencies
  const int hp = p.rotary >> 4;    // 16-byte pieces of a rotated half
  // the lane's two pieces: l and its partner of the other half, or two of the pieces that do not rotate;
  // interleaved pairs lie inside a piece.  Neighbouring lanes take neighbouring pieces, so that a copy's
  // 16 bytes a lane make whole sectors.
  const int pa = p.interleaved || l < hp ? l : hp + l;
  const int pb = p.interleaved ? l + 8 : (l < hp ? l + hp : l + 8);
  if (threadIdx.x < 32) {
    const void* w = threadIdx.x < 16 ? p.q_weight : p.k_weight;
    if (w) norm_weight[threadIdx.x >> 4][threadIdx.x & 15] = __ldg(static_cast<const uint4*>(w) + (threadIdx.x & 15));
  }
  // this group's run of tokens
  const long long me = (long long)blockIdx.x * kGroups + group, groups = (long long)gridDim.x * kGroups;
  const int s0 = int(total * me / groups), s1 = int(total * (me + 1) / groups);

  const int heads = p.hqo + 2 * pv.hkv;  // rows of a token: q, k, v
  int f_tok = s0, f_row = sub;  // what is fetched next
  auto fetch = [&](int slot) {
    const bool on = f_tok < s1 && f_row < heads;
    const long long tok = on ? f_tok : 0;
    const int row = on ? f_row : 0;
    const __nv_bfloat16* at = static_cast<const __nv_bfloat16*>(p.q) + tok * p.q_stride + row * kHeadDim;
    if (row >= p.hqo) at = static_cast<const __nv_bfloat16*>(p.k) + tok * p.k_stride + (row - p.hqo) * kHeadDim;
    if (row >= p.hqo + pv.hkv)
      at = static_cast<const __nv_bfloat16*>(p.v) + tok * p.v_stride + (row - p.hqo - pv.hkv) * kHeadDim;
    cp_async_16_or_none(&ring[slot][0][threadIdx.x], at + 8 * pa, on);
    cp_async_16_or_none(&ring[slot][1][threadIdx.x], at + 8 * pb, on);
    cp_async_commit();
    f_row += kRowsPass;
    if (f_row - sub >= heads) {
      f_row = sub;
      ++f_tok;
    }
  };
#pragma unroll
  for (int i = 0; i < kDepth; ++i) fetch(i);

  uint64_t f0 = 0, f1 = 0;  // the lane's two frequencies
  if (leads) {
    if (lane < half) f0 = p.freq[lane];
    if (lane + 32 < half) f1 = p.freq[lane + 32];
  }
  Geo g{};  // the request of the last token
  // slot and angles of a token, by the group's first warp
  auto prepare = [&](int tok, int par) {
    if (tok >= s1) return;
    if (tok < g.q0 || tok >= g.q0 + g.lq) g = load_geo(pv.geo, find_request(pv.geo, batch, &Geo::q0, tok));
    const int j = g.lkv - g.lq + tok - g.q0;
    const int pos = p.positions ? __ldg(p.positions + tok) : j;
    if (lane == 0) {
      long long off = -1;
      int page, slot;
      if (j >= 0 && locate(pv, g.kv0, j, page, slot)) off = kv_offset(pv, page, slot, 0);
      place[group][par] = off;
    }
    float* c = reinterpret_cast<float*>(cosines[group][par]);
    float* s = reinterpret_cast<float*>(sines[group][par]);
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
  };
  if (leads) prepare(s0, 0);
  __syncthreads();  // the norm weights

  int par = 0, slot = 0;
  for (int tok = s0; tok < s1; ++tok, par ^= 1) {
    sync();
    if (leads) prepare(tok + 1, par ^ 1);
    const float4 *cosine = cosines[group][par], *sine = sines[group][par];
    const long long off0 = place[group][par];
    for (int h = sub; h - sub < heads; h += kRowsPass) {
      cp_async_wait<kDepth - 1>();
      const uint4 raw[2] = {ring[slot][0][threadIdx.x], ring[slot][1][threadIdx.x]};
      fetch(slot);
      slot = slot + 1 == kDepth ? 0 : slot + 1;
      if (h >= heads) continue;
      float2 a[4], b[4];
      unpack8(raw[0], a);
      unpack8(raw[1], b);
      if (h >= p.hqo + pv.hkv) {  // v: as it is
        if (off0 < 0) continue;
        const long long off = off0 + (h - p.hqo - pv.hkv) * pv.head_stride;
        if constexpr (kFp8) {
          put8<true>(p.v_pages, off + 8 * pa, a, p.v_inv_scale);
          put8<true>(p.v_pages, off + 8 * pb, b, p.v_inv_scale);
        } else {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.v_pages) + off);
          dst[pa] = raw[0];
          dst[pb] = raw[1];
        }
        continue;
      }
      const bool is_q = h < p.hqo;
      if (is_q ? p.q_weight != nullptr : p.k_weight != nullptr) {
        float2 w[4], s2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < 4; ++e) s2 = __ffma2_rn(b[e], b[e], __ffma2_rn(a[e], a[e], s2));
        float ss = s2.x + s2.y;
        // the lanes of a row agree on all branches
        const unsigned mates = 0xffu << (lane & 24);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) ss += __shfl_xor_sync(mates, ss, o);
        const float inv = rsqrtf(fmaf(ss, 1.f / kHeadDim, p.eps));
        const float2 i2 = make_float2(inv, inv);
        unpack8(norm_weight[is_q ? 0 : 1][pa], w);
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] = __fmul2_rn(__fmul2_rn(a[e], i2), w[e]);
        unpack8(norm_weight[is_q ? 0 : 1][pb], w);
#pragma unroll
        for (int e = 0; e < 4; ++e) b[e] = __fmul2_rn(__fmul2_rn(b[e], i2), w[e]);
      }
      if (p.interleaved) {
        auto turn = [&](float2 (&x)[4], int piece) {
          if (piece >= 2 * hp) return;
          const float4 c = cosine[piece], s = sine[piece];
          const float cc[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            x[e] = make_float2(x[e].x * cc[e] - x[e].y * sn[e], x[e].x * sn[e] + x[e].y * cc[e]);
        };
        turn(a, pa);
        turn(b, pb);
      } else if (l < hp) {
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2) {
          const float4 c = cosine[8 * e2 + l], s = sine[8 * e2 + l];
          const float2 cc[2] = {make_float2(c.x, c.y), make_float2(c.z, c.w)};
          const float2 sn[2] = {make_float2(s.x, s.y), make_float2(s.z, s.w)};
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 x = a[2 * e2 + e], y = b[2 * e2 + e];
            const float2 ms = make_float2(-sn[e].x, -sn[e].y);
            a[2 * e2 + e] = __ffma2_rn(y, ms, __fmul2_rn(x, cc[e]));
            b[2 * e2 + e] = __ffma2_rn(x, sn[e], __fmul2_rn(y, cc[e]));
          }
        }
      }
      if (is_q) {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.q_out) +
                                              ((long long)tok * p.hqo + h) * kHeadDim);
        dst[pa] = pack8(a);
        dst[pb] = pack8(b);
      } else if (off0 >= 0) {
        const long long off = off0 + (h - p.hqo) * pv.head_stride;
        put8<kFp8>(p.k_pages, off + 8 * pa, a, p.k_inv_scale);
        put8<kFp8>(p.k_pages, off + 8 * pb, b, p.k_inv_scale);
      }
    }
  }
  cp_async_wait<0>();
}

}  // namespace

int launch_append(const AppendParams& p, int total_q, int most_q, bool fp8, int num_sms, cudaStream_t stream) {
  using Kernel = void (*)(const AppendParams);
  static const Kernel kernels[4] = {append_kernel<kAppendThreads, false>, append_kernel<kAppendThreads, true>,
                                    append_kernel<32, false>, append_kernel<32, true>};
  constexpr size_t ring = sizeof(uint4) * 2 * kAppendThreads;  // of one pass
  const size_t smem[2] = {ring * kPassesAhead<kAppendThreads>, ring * kPassesAhead<32>};
  static std::once_flag once;
  static cudaError_t attr = cudaSuccess;
  std::call_once(once, [&] {
    for (int i = 0; i < 4 && attr == cudaSuccess; ++i)
      attr = cudaFuncSetAttribute(kernels[i], cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem[i / 2]));
  });
  if (attr != cudaSuccess) return record_cuda_error(attr, "cudaFuncSetAttribute(append_kernel)");
  // a warp for each token once they fill the grid's warps
  const int ctas = kAppendCtasPerSm * num_sms;
  const bool many = total_q >= ctas * (kAppendThreads / 32);
  const cudaError_t e = launch_dependent(kernels[(many ? 2 : 0) + (fp8 ? 1 : 0)], unsigned(std::min(most_q, ctas)),
                                         kAppendThreads, smem[many ? 1 : 0], 1, stream, p);
  return e == cudaSuccess ? 0 : record_cuda_error(e, "append_kernel launch");
}

}  // namespace fi
