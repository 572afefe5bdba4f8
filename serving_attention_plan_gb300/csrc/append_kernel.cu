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
// heads, now 125: 5.1 TB/s, 0.76 of the copy rate.  Norm and rotation are 6 % of that; more passes in flight, more or fewer
// warps, a warp for each token and other token orders changed nothing.)  The angles of a token are computed once, by the warp that also finds its page slot,
// one step ahead of the rows, and shared by all its heads through shared memory.
//
// Angles: a position times a frequency is taken in turns as a 64-bit fraction, p * F mod 2^64 with
// F = round(2^64 frac(f / 2 pi)): whole turns drop out exactly in the integer product, so the angle
// is right to 2^-33 turns + the rounding of F (p * 2^-65) at any position, where a 32-bit product
// loses the angle itself beyond some ten thousand positions.
#include <cuda_fp8.h>

#include <algorithm>

#include "cache_common.cuh"
#include "prefill_launch.h"

namespace fi {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kRowLanes = 8;
constexpr int kRowsPass = kAppendThreads / kRowLanes;  // rows of a pass; the next pass is in flight meanwhile
constexpr int kAppendCtasPerSm = 3;

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

// A step is kTok tokens: four for long batches (the sync and the search for the request are paid once for four
// tokens), one for decode steps, where tokens are few and each CTA should take one.
template <int kTok, bool kFp8>
__global__ void __launch_bounds__(kAppendThreads, kAppendCtasPerSm) append_kernel(const __grid_constant__ AppendParams p) {
  // cos and sin of a token's frequencies: piece k of a split half holds frequencies 8 k .. 8 k + 7, its first
  // four at [k], the others at [8 + k], so the lanes' 16-byte reads fall into different banks; interleaved
  // pairs are in order, piece k holds [k]
  __shared__ float4 cosines[2][kTok][16], sines[2][kTok][16];
  __shared__ long long place[2][kTok];  // element offset of KV head 0 in the pages, -1: no slot
  wait_prior_grid();
  const PageView& pv = p.pv;
  const GeoHead plan = load_head(pv.geo);
  const int batch = plan.batch, total = plan.total_q;
  if (batch == 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = threadIdx.x / kRowLanes, l = threadIdx.x % kRowLanes;
  const int half = p.rotary >> 1;  // frequencies
  const int hp = p.rotary >> 4;    // 16-byte pieces of a rotated half
  // the lane's two pieces, and whether they rotate (together, or each by itself when interleaved)
  const int pa = p.interleaved ? l : (l < hp ? l : 2 * hp + 2 * (l - hp));
  const int pb = p.interleaved ? l + 8 : (l < hp ? l + hp : pa + 1);
  uint4 wq[2] = {}, wk[2] = {};
  if (p.q_weight) {
    wq[0] = __ldg(reinterpret_cast<const uint4*>(p.q_weight) + pa);
    wq[1] = __ldg(reinterpret_cast<const uint4*>(p.q_weight) + pb);
  }
  if (p.k_weight) {
    wk[0] = __ldg(reinterpret_cast<const uint4*>(p.k_weight) + pa);
    wk[1] = __ldg(reinterpret_cast<const uint4*>(p.k_weight) + pb);
  }
  // this CTA's run of steps
  const int steps = (total + kTok - 1) / kTok;
  const int s0 = int((long long)steps * blockIdx.x / gridDim.x), s1 = int((long long)steps * (blockIdx.x + 1) / gridDim.x);

  uint64_t f0 = 0, f1 = 0;  // the lane's two frequencies
  if (warp < kTok) {
    if (lane < half) f0 = p.freq[lane];
    if (lane + 32 < half) f1 = p.freq[lane + 32];
  }
  Geo g{};  // the request of the warp's last token
  // slot and angles of the step's token `warp`, by that warp
  auto prepare = [&](int step, int par) {
    const int tok = step * kTok + warp;
    if (step >= s1 || tok >= total) return;
    if (tok < g.q0 || tok >= g.q0 + g.lq) g = load_geo(pv.geo, find_request(pv.geo, batch, &Geo::q0, tok));
    const int j = g.lkv - g.lq + tok - g.q0;
    const int pos = p.positions ? __ldg(p.positions + tok) : j;
    if (lane == 0) {
      long long off = -1;
      int page, slot;
      if (j >= 0 && locate(pv, g.kv0, j, page, slot)) off = kv_offset(pv, page, slot, 0);
      place[par][warp] = off;
    }
    float* c = reinterpret_cast<float*>(cosines[par][warp]);
    float* s = reinterpret_cast<float*>(sines[par][warp]);
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
  if (warp < kTok) prepare(s0, 0);

  const int heads = p.hqo + 2 * pv.hkv;  // rows of a token: q, k, v
  uint4 next[2];
  int next_t = 0, next_h = -1;  // row of the step that `next` holds, -1: none
  auto load = [&](int step, int row) {
    next_h = -1;
    const int base = step * kTok;
    if (step >= s1 || row >= min(kTok, total - base) * heads) return;
    next_t = kTok == 1 ? 0 : int(__umulhi(unsigned(row), p.heads_inv));
    next_h = row - next_t * heads;
    const long long tok = base + next_t;
    const __nv_bfloat16* at;
    if (next_h < p.hqo)
      at = static_cast<const __nv_bfloat16*>(p.q) + tok * p.q_stride + next_h * kHeadDim;
    else if (next_h < p.hqo + pv.hkv)
      at = static_cast<const __nv_bfloat16*>(p.k) + tok * p.k_stride + (next_h - p.hqo) * kHeadDim;
    else
      at = static_cast<const __nv_bfloat16*>(p.v) + tok * p.v_stride + (next_h - p.hqo - pv.hkv) * kHeadDim;
    next[0] = __ldcs(reinterpret_cast<const uint4*>(at) + pa);
    next[1] = __ldcs(reinterpret_cast<const uint4*>(at) + pb);
  };
  load(s0, sub);
  int par = 0;
  for (int step = s0; step < s1; ++step, par ^= 1) {
    const int base = step * kTok, rows = min(kTok, total - base) * heads;
    __syncthreads();
    if (warp < kTok) prepare(step + 1, par ^ 1);
    for (int row = sub; row - sub < rows; row += kRowsPass) {
      const uint4 raw[2] = {next[0], next[1]};
      const int t = next_t, h = next_h;
      if (row - sub + kRowsPass < rows)
        load(step, row + kRowsPass);
      else
        load(step + 1, sub);
      if (h < 0) continue;
      float2 a[4], b[4];
      unpack8(raw[0], a);
      unpack8(raw[1], b);
      if (h >= p.hqo + pv.hkv) {  // v: as it is
        if (place[par][t] < 0) continue;
        const long long off = place[par][t] + (h - p.hqo - pv.hkv) * pv.head_stride;
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
        unpack8(is_q ? wq[0] : wk[0], w);
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] = __fmul2_rn(__fmul2_rn(a[e], i2), w[e]);
        unpack8(is_q ? wq[1] : wk[1], w);
#pragma unroll
        for (int e = 0; e < 4; ++e) b[e] = __fmul2_rn(__fmul2_rn(b[e], i2), w[e]);
      }
      if (p.interleaved) {
        auto turn = [&](float2 (&x)[4], int piece) {
          if (piece >= 2 * hp) return;
          const float4 c = cosines[par][t][piece], s = sines[par][t][piece];
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
          const float4 c = cosines[par][t][8 * e2 + l], s = sines[par][t][8 * e2 + l];
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
                                              ((long long)(base + t) * p.hqo + h) * kHeadDim);
        dst[pa] = pack8(a);
        dst[pb] = pack8(b);
      } else if (place[par][t] >= 0) {
        const long long off = place[par][t] + (h - p.hqo) * pv.head_stride;
        put8<kFp8>(p.k_pages, off + 8 * pa, a, p.k_inv_scale);
        put8<kFp8>(p.k_pages, off + 8 * pb, b, p.k_inv_scale);
      }
    }
  }
}

}  // namespace

int launch_append(AppendParams p, int total_q, bool fp8, int num_sms, cudaStream_t stream) {
  const bool many = total_q >= 8 * num_sms;
  const unsigned grid = unsigned(many ? std::min((total_q + 3) / 4, kAppendCtasPerSm * num_sms) : total_q);
  const unsigned heads = unsigned(p.hqo + 2 * p.pv.hkv);
  p.heads_inv = unsigned(((1ull << 32) + heads - 1) / heads);  // division by a high product: exact below 2^32 / heads
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
