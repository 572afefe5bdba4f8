// Attention of a tree of drafted tokens over a paged cache, and the move of the accepted path's keys.
//
//   o = softmax(x) V,  x = scale q.k (soft-cap: cap tanh(x / cap)),  over the keys that a row sees:
//   key j of a request of l_q tokens and l_kv keys is seen by token t if j < l_kv - l_q, or if bit
//   j - (l_kv - l_q) of t's mask is set.
//
// What bounds it: a tree has 8 to 64 tokens, so a KV head has 32 to 512 query rows; up to 128 rows a key costs
// 2 * 128 * 128 products for 512 bytes, which the tensor cores do in a third of the time that the bytes take.  The kernel
// is therefore built to stream keys past a tile of 128 rows of one KV head (rows are (token, head of the group) pairs), or
// past two such tiles at once: with one tile a pass, 256 rows read every key twice, and the second reading, from L2, took
// as long as the first.  Two tiles are bound by the rate at which the products take their operands: 32 score products of 128 x
// 64 at 76 clocks and 16 output products of 128 x 128 at 75 are 3600 of the 3900 clocks of 128 keys.
//
// Measured: 64 requests of 16 tokens over 265 K bf16 keys in all, 32/8 heads, 179 us (0.92 of the copy bandwidth), 128 of 8 tokens
// over 283 K 190; 32 of 64 tokens over 158 K 171 (256 rows); the 64 requests with e4m3 keys 155; 12 requests of 17 to 30
// tokens over 8 to 24 K e4m3 keys, 64/8 heads, 218.
//
// Split: the 128-key tiles of all (request, KV head, pair of row tiles) units form one line, and every CTA takes an equal
// piece of it, wherever that cuts a unit.  Nothing of this is planned on the host but the line's prefix per request, so a
// captured launch follows later plans.  A unit that was cut leaves partial states, which a second launch joins in order.
//
// One CTA an SM.  Two softmax groups, each with its own running maximum, sum and accumulator, keep the tensor cores
// and each other busy, 64 keys a step: with one row tile group h takes keys 64 h .. 64 h + 63 of every tile, and the two
// states are joined when the piece is written; with two it takes row tile h.
//   warps 0-3, 4-7    softmax of group 0 and 1; a thread owns a row (TMEM lane)
//   warps 8-11        a finished piece, to the output or to a partial slot; e4m3: Q as two e4m3 terms
//   warps 12-15       TMA of page boxes, every stage's boxes dealt to the four (one warp's issue ends at 4 TB/s)
//   warps 16, 17      issue of S = Q K^T and of O_h += P_h V
//   warp 18           the CTA's pieces, ahead of the others (found out by each warp for itself, the next piece cost 5000
//                     clocks of waiting for its request's entry)
//   warps 20-23       e4m3: V widened to f16
// TMEM: two score buffers of 2 x 64 columns (P overwrites a group's first 32), O_0 and O_1.
// Shared memory: two Q tiles; bf16: five K / V tiles; e4m3: six tiles of codes and two of widened V.
//
// e4m3 pages: K's codes go into the products as they are, against q as a sum of two e4m3 terms (each row scaled by a power
// of two that brings its largest element to 128 .. 256; the sum is exact for elements above 2^-9 of that, and right to 2^-17
// of it for the others), at the rate of as many bf16 products.  V is widened to f16, exactly, so that the weights keep 11
// bits.  (K and V both widened: the widening and the few f16 tiles that shared memory holds set the pace, 2800
// clocks a tile, where the bytes take 1450.)
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <mutex>

#include "cache_common.cuh"
#include "prefill_launch.h"
#include "tcgen05.cuh"
#include "tree_ops.h"

namespace fi {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kRows = kTreeRows;            // query rows of a tile
constexpr int kKeys = kTreeKeys;            // keys of a tile
constexpr int kHalfKeys = kKeys / 2;
constexpr int kHalfBytes = kRows * 128;     // one 64-dim half of a 128-row tile
constexpr int kTileBytes = 2 * kHalfBytes;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;             // O_h at 256 + 128 h, S_b at 128 b
constexpr float kRescaleThreshold = 8.f;    // O is rescaled when a row's maximum grows by more than 2^8
constexpr int kLoaders = 4;

// Registers of a thread per warpgroup.  Launched with 96 (bf16, 640 threads) or 80 (e4m3, 768); the shares below add up to
// that.
template <bool kFp8>
struct Shape {
  static constexpr int kThreads = kFp8 ? 768 : 640;
  static constexpr int kLaunchRegs = kFp8 ? 80 : 96;
  static constexpr uint32_t kSoftmaxRegs = kFp8 ? 136 : 144;
  static constexpr uint32_t kWriteRegs = kFp8 ? 72 : 80;
  static constexpr uint32_t kLoadRegs = kFp8 ? 40 : 56;
  static constexpr uint32_t kIssueRegs = 56;
  static constexpr uint32_t kWidenRegs = kFp8 ? 40 : 0;
  static_assert(2 * kSoftmaxRegs + kWriteRegs + kLoadRegs + kIssueRegs + kWidenRegs == kLaunchRegs * (kThreads / 128),
                "the warpgroups' registers are those of the launch");
  static constexpr int kRing = kFp8 ? 6 : 5;  // tiles that TMA fills, K and V in turn
  static constexpr int kTile = kFp8 ? kHalfBytes : kTileBytes;
  static constexpr int kWide = kFp8 ? 2 : 0;  // V tiles widened
  static constexpr int kReaders = 8 + 4 + kLoaders + 2 + (kFp8 ? 4 : 0);  // warps that read the pieces
};

// A run of tiles of one (request, KV head, pair of row tiles) unit.
struct Piece {
  int q0, nq;         // its first query token, tokens
  int kv0, lkv, lq;   // the request's first page entry, keys, tokens
  int head;
  int k0, k1;         // tiles [k0, k1) of the unit's; none: the pieces end here
  int slot;           // partial slot, or -1 for a whole unit
  int pad[3];
};
static_assert(sizeof(Piece) == 48, "three 16-byte words");
constexpr int kPieces = 4;  // found ahead

template <bool kFp8>
struct TreeSmem {
  uint8_t q[2][kTileBytes];  // [2 dim halves][128 rows][128 B] of bf16, 128B-swizzled; e4m3: then [2 terms][128 rows][128 codes]
  uint8_t kv[Shape<kFp8>::kRing][Shape<kFp8>::kTile];
  uint8_t wide[kFp8 ? Shape<kFp8>::kWide : 1][kFp8 ? kTileBytes : 16];
  float stat_m[2][kRows], stat_l[2][kRows];
  Piece pieces[kPieces];
  int8_t q_exp[2][kRows];  // e4m3: q = 2^exp (term 0 + term 1), kQuiet for a row that is not finite
  uint64_t piece_full[kPieces], piece_empty[kPieces];
  uint64_t q_full[2], q_empty[2], q_ready[2];
  uint64_t full[Shape<kFp8>::kRing], empty[Shape<kFp8>::kRing];
  uint64_t wide_full[2], wide_empty[2];
  uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];  // [group][buffer]
  uint64_t stat_full, stat_empty, o_free;
  uint32_t tmem_base;
  int abort;
};
constexpr int kQuiet = -128;

// Bounded wait for a barrier's phase: kTries tries that may each sleep for a microsecond, two seconds (60 ms if none of them
// slept; the longest wait, for the end of a piece, is 2 us a tile).  There are some forty waits: with a look at the clock
// in each, as in mbar_wait, the roles' code outgrew the instruction cache.
constexpr uint32_t kTries = 1u << 21;
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, int32_t* err, volatile int* abort) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\tmov.u32 n, 0;\n\t"
      "TRY:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000;\n\t"
      "@p bra DONE;\n\t"
      "add.u32 n, n, 1;\n\tsetp.lt.u32 q, n, %3;\n\t"
      "@q bra TRY;\n\t"
      "DONE:\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity), "n"(kTries)
      : "memory");
  if (done) return true;
  if (*abort == 0) atomicOr(err, FI_DEVERR_WAIT_TIMEOUT);
  *abort = 1;
  return false;
}

// ---- the line of tiles ---------------------------------------------------------------------------

struct Line {
  int total, per, ctas;  // tiles; of a CTA; CTAs that have any
  __device__ Line(int tiles, int grid) : total(tiles) {
    per = max(kTreeLeastTiles, (total + grid - 1) / grid);
    ctas = (total + per - 1) / per;
  }
};

// Warp 18: the pieces of the CTA's part [pos, end) of the line, which begins in request r, in order, into the ring.
template <bool kFp8>
__device__ void find_pieces(const TreeParams& p, TreeSmem<kFp8>& sm, const GeoHead& plan, const Line& line, int cta, int r) {
  const int lane = threadIdx.x & 31, hkv = p.pv.hkv, tokens = 2 * p.tile_tokens;
  int pos = cta * line.per;
  const int end = min(line.total, pos + line.per);
  Geo g = load_geo(p.pv.geo, r), after = load_geo(p.pv.geo, r + 1);  // (an entry lies behind the last request)
  int tiles = max(1, (g.lkv + kKeys - 1) / kKeys), sets = (g.lq + tokens - 1) / tokens;
  int unit = (pos - g.tree0) / tiles, at = pos - g.tree0 - unit * tiles;
  for (int n = 0;; ++n) {
    const int slot = n % kPieces;
    if (n >= kPieces && !__all_sync(kAll, wait_for(&sm.piece_empty[slot], (n / kPieces - 1) & 1, p.pv.err, &sm.abort))) return;
    Piece c = {};
    if (pos < end) {
      while (unit == hkv * sets) {
        g = after;
        after = load_geo(p.pv.geo, min(++r + 1, plan.batch));
        tiles = max(1, (g.lkv + kKeys - 1) / kKeys);
        sets = (g.lq + tokens - 1) / tokens;
        unit = at = 0;
      }
      const int set = unit % sets;
      c.head = unit / sets;
      c.q0 = g.q0 + set * tokens;
      c.nq = min(tokens, g.lq - set * tokens);
      c.kv0 = g.kv0;
      c.lkv = g.lkv;
      c.lq = g.lq;
      c.k0 = at;
      c.k1 = at + min(tiles - at, end - pos);
      const int a = pos - at, first = a / line.per;  // the unit's place on the line, the CTA that begins it
      c.slot = (a + tiles - 1) / line.per != first ? 2 * first + (cta - first) : -1;
      pos += c.k1 - c.k0;
      at = 0;
      ++unit;
    }
    if (lane == 0) {
      sm.pieces[slot] = c;
      mbar_arrive(&sm.piece_full[slot]);
    }
    __syncwarp();
    if (c.k0 == c.k1) return;
  }
}

// Piece number n, for a whole warp; false behind the last one.
template <bool kFp8>
__device__ __forceinline__ bool take(const TreeParams& p, TreeSmem<kFp8>& sm, int n, Piece& c) {
  const int slot = n % kPieces;
  const bool ok = __all_sync(kAll, wait_for(&sm.piece_full[slot], (n / kPieces) & 1, p.pv.err, &sm.abort));
  const int4* src = reinterpret_cast<const int4*>(&sm.pieces[slot]);
  const int4 x = src[0], y = src[1];
  c.q0 = x.x;
  c.nq = x.y;
  c.kv0 = x.z;
  c.lkv = x.w;
  c.lq = y.x;
  c.head = y.y;
  c.k0 = y.z;
  c.k1 = y.w;
  c.slot = src[2].x;
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&sm.piece_empty[slot]);
  return ok && c.k0 < c.k1;
}

// Steps of 64 keys a group that a piece takes.
__device__ __forceinline__ int steps_of(const Piece& c, bool two) {
  return two ? max(1, (min(c.k1 * kKeys, c.lkv) - c.k0 * kKeys + kHalfKeys - 1) / kHalfKeys) : c.k1 - c.k0;
}

__device__ __forceinline__ bool elect_one() {
  uint32_t on;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(on));
  return on != 0;
}

// ---- loads -----------------------------------------------------------------------------------------

// Loader warp `w` of four: its share of the boxes of every tile, K and V in turn.  A box is one page and KV head, 64 dims
// (bf16) or 128 codes (e4m3), 128B-swizzled; pages behind the request's last read as zeros.
template <bool kFp8>
__device__ void load_tiles(const TreeParams& p, TreeSmem<kFp8>& sm, const CUtensorMap* tm_q, const CUtensorMap* tm_k,
                           const CUtensorMap* tm_v, int w) {
  using S = Shape<kFp8>;
  const int lane = threadIdx.x & 31;
  const int ps = p.pv.page_size, pages = kKeys / ps;
  const int boxes = kFp8 ? pages : 2 * pages;
  const int mine = w + kLoaders * lane;  // this lane's box
  const int page = kFp8 ? mine : mine >> 1, half = kFp8 ? 0 : mine & 1;
  const uint32_t bytes = uint32_t((boxes - w + kLoaders - 1) / kLoaders) * uint32_t(ps) * 128u;
  const uint32_t place = uint32_t(half) * kHalfBytes + uint32_t(page * ps) * 128u;
  auto locate = [&](const Piece& c, int t) {  // the page of this lane's box, num_pages for none
    int z = p.pv.num_pages;
    const int e = t * pages + page;
    if (mine < boxes && e * ps < c.lkv) {
      const int id = __ldg(p.pv.kv_indices + c.kv0 + e);
      if (static_cast<unsigned>(id) < static_cast<unsigned>(p.pv.num_pages))
        z = id;
      else
        atomicOr(p.pv.err, FI_DEVERR_PAGE_OOB);
    }
    return z;
  };
  Piece c;
  int n = 0, nu = 0, nq = 0;  // tiles, pieces, Q tiles
  bool ok = true, more = take(p, sm, nu++, c);
  int t = c.k0;
  int z_next = more ? locate(c, t) : 0;
  while (more && ok) {
    const int z = z_next, head = c.head;
    int q0 = c.q0, q_left = t == c.k0 ? c.nq : 0;  // the piece's Q tiles come behind its first K tile, whose place is free before theirs
    if (++t == c.k1) {
      more = take(p, sm, nu++, c);
      t = c.k0;
    }
    if (more) z_next = locate(c, t);  // lands while this tile waits for its place
    for (int v = 0; v < 2; ++v, ++n) {
      const int slot = n % S::kRing;
      if (n >= S::kRing) ok = __all_sync(kAll, wait_for(&sm.empty[slot], (n / S::kRing - 1) & 1, p.pv.err, &sm.abort));
      if (!ok) break;
      if (lane == 0) mbar_arrive_expect_tx(&sm.full[slot], bytes);
      __syncwarp();
      if (mine < boxes) tc::tma_load_4d(sm.kv[slot] + place, v ? tm_v : tm_k, 64 * half, head, 0, z, &sm.full[slot]);
      for (; q_left > 0; q_left -= p.tile_tokens, q0 += p.tile_tokens, ++nq) {
        if (w != 0) continue;
        const int b = nq & 1;
        if (nq >= 2) ok = __all_sync(kAll, wait_for(&sm.q_empty[b], ((nq >> 1) - 1) & 1, p.pv.err, &sm.abort));
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&sm.q_full[b], p.q_tile_bytes);
          tc::tma_load_3d(sm.q[b], tm_q, 0, head * p.group, q0, &sm.q_full[b]);
          tc::tma_load_3d(sm.q[b] + kHalfBytes, tm_q, 64, head * p.group, q0, &sm.q_full[b]);
        }
        __syncwarp();
      }
      if (!ok) {
        ++n;
        break;
      }
    }
  }
  // no copy is left landing in this CTA's shared memory
  if (w == 0)
    for (int k = max(0, nq - 2); k < nq; ++k) mbar_wait_bounded(&sm.q_full[k & 1], (k >> 1) & 1);
  for (int k = max(0, n - S::kRing); k < n; ++k) mbar_wait_bounded(&sm.full[k % S::kRing], (k / S::kRing) & 1);
}

__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two_codes) {
  uint32_t h;
  const uint16_t v = static_cast<uint16_t>(two_codes);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(v));
  return h;
}
__device__ __forceinline__ uint32_t f2_to_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// e4m3: widening warp `w` of four takes 32 rows of every V tile: eight lanes read one row of codes and write it as f16 in the
// products' layout (16-byte chunk c of a 64-dim half's row r at c ^ (r % 8)).  The lanes of the second half write their odd
// chunk first, so that a row's eight lanes fill different banks.  Rows behind the last key become zeros: a page's unused
// slots may hold NaN, which a weight of zero would not cancel.
__device__ void widen_tiles(const TreeParams& p, TreeSmem<true>& sm, int w) {
  using S = Shape<true>;
  const int lane = threadIdx.x & 31, chunk = lane & 7;
  const uint32_t half_off = uint32_t(chunk >> 2) * kHalfBytes;
  const bool swap = chunk >= 4;
  const int m = (2 * chunk) & 7;
  const int r0 = 32 * w + (lane >> 3);
  Piece c;
  int tt = 0, nu = 0;
  bool ok = true;
  for (; ok && take(p, sm, nu, c); ++nu) {
    for (int t = c.k0; t < c.k1; ++t, ++tt) {
      const int lim = c.lkv - t * kKeys;
      const int n = 2 * tt + 1, from = n % S::kRing, to = tt % S::kWide;
      ok = __all_sync(kAll, wait_for(&sm.full[from], (n / S::kRing) & 1, p.pv.err, &sm.abort));
      if (!ok) break;
      const uint32_t src = smem_u32(sm.kv[from]) + uint32_t(r0 * 128), dst = smem_u32(sm.wide[to]) + half_off + uint32_t(r0 * 128);
#pragma unroll 1
      for (int i0 = 0; i0 < 8; i0 += 4) {
        uint32_t x[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(x[i][0]), "=r"(x[i][1]), "=r"(x[i][2]), "=r"(x[i][3])
                       : "r"(src + uint32_t(512 * (i0 + i) + 16 * (chunk ^ ((r0 + 4 * (i0 + i)) & 7))))
                       : "memory");
        if (i0 == 0) {
          if (tt >= S::kWide) ok = __all_sync(kAll, wait_for(&sm.wide_empty[to], (tt / S::kWide - 1) & 1, p.pv.err, &sm.abort));
          if (!ok) break;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = r0 + 4 * (i0 + i);
          const bool on = r < lim;
          const uint32_t lo[2] = {on ? x[i][0] : 0u, on ? x[i][1] : 0u}, hi[2] = {on ? x[i][2] : 0u, on ? x[i][3] : 0u};
          const uint32_t a[2] = {swap ? hi[0] : lo[0], swap ? hi[1] : lo[1]}, b[2] = {swap ? lo[0] : hi[0], swap ? lo[1] : hi[1]};
          const uint32_t row = dst + 512 * (i0 + i);
          const int ca = (swap ? m + 1 : m) ^ (r & 7), cb = (swap ? m : m + 1) ^ (r & 7);
          asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(row + 16 * ca), "r"(e4m3x2_to_f16x2(a[0])),
                       "r"(e4m3x2_to_f16x2(a[0] >> 16)), "r"(e4m3x2_to_f16x2(a[1])), "r"(e4m3x2_to_f16x2(a[1] >> 16))
                       : "memory");
          asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(row + 16 * cb), "r"(e4m3x2_to_f16x2(b[0])),
                       "r"(e4m3x2_to_f16x2(b[0] >> 16)), "r"(e4m3x2_to_f16x2(b[1])), "r"(e4m3x2_to_f16x2(b[1] >> 16))
                       : "memory");
        }
      }
      if (!ok) break;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sm.wide_full[to]);
        mbar_arrive(&sm.empty[from]);
      }
    }
  }
}

__device__ __forceinline__ uint32_t e4m3x2_of(float lo, float hi) {
  uint16_t v;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(hi), "f"(lo));
  return v;
}

// e4m3: Q tile number n from bf16 into its two terms, in place: warp `w` of four takes 32 rows, eight lanes a row, 16 of its
// bytes from each dim half.  A row's bytes are read by the lanes that write them, four rows a step.
__device__ bool split_q(const TreeParams& p, TreeSmem<true>& sm, int n, int w) {
  const int lane = threadIdx.x & 31, c = lane & 7, b = n & 1;
  if (!__all_sync(kAll, wait_for(&sm.q_full[b], (n >> 1) & 1, p.pv.err, &sm.abort))) return false;
  const uint32_t q = smem_u32(sm.q[b]);
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {
    const int r = 32 * w + 4 * i + (lane >> 3), sw = r & 7;
    const uint32_t row = q + uint32_t(r * 128);
    uint32_t x[8];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(x[4 * h]), "=r"(x[4 * h + 1]), "=r"(x[4 * h + 2]), "=r"(x[4 * h + 3])
                   : "r"(row + uint32_t(h * kHalfBytes + 16 * (c ^ sw)))
                   : "memory");
    uint32_t top = 0;  // the largest |element|'s bits
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max(top, max(x[k] & 0x7fffu, x[k] >> 16 & 0x7fffu));
#pragma unroll
    for (int m = 1; m < 8; m <<= 1) top = max(top, __shfl_xor_sync(kAll, top, m));
    const int e = int(top >> 7);  // its exponent field; the factor 2^(134 - e) brings it to 128 .. 256
    const int up = top == 0 ? 0 : min(134 - e, 126);
    const float f = __uint_as_float(uint32_t(up + 127) << 23);
    uint32_t t0[4], t1[4];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float2 v = __fmul2_rn(bf16x2_to_f2(x[k]), make_float2(f, f));
      const uint32_t a = e4m3x2_of(v.x, v.y);
      const uint32_t back = e4m3x2_to_f16x2(a);
      const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&back));
      const uint32_t rest = e4m3x2_of(v.x - g.x, v.y - g.y);
      t0[k >> 1] = k & 1 ? t0[k >> 1] | a << 16 : a;
      t1[k >> 1] = k & 1 ? t1[k >> 1] | rest << 16 : rest;
    }
    __syncwarp();
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // dims 64 h + 8 c .. : half of 16-byte chunk 4 h + c / 2
      const uint32_t at = row + uint32_t(16 * ((4 * h + (c >> 1)) ^ sw) + 8 * (c & 1));
      asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(at), "r"(t0[2 * h]), "r"(t0[2 * h + 1]) : "memory");
      asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(at + kHalfBytes), "r"(t1[2 * h]), "r"(t1[2 * h + 1]) : "memory");
    }
    if (c == 0) sm.q_exp[b][r] = int8_t(e == 255 ? kQuiet : -up);
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive(&sm.q_ready[b]);
  return true;
}

// ---- products ----------------------------------------------------------------------------------------
// One warp issues S, another O, by an elected lane of a uniform warp.  With two row tiles the scores of the two groups are
// products of their own (64 columns), and the groups fall out of step; with one they are one product of 128 columns (two of 64
// read Q twice: 197 against 194 us for 64 requests of 16 tokens).

// D (TMEM) [+]= A (shared memory) B (shared memory), e4m3 operands.
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// S = Q K^T from the descriptors of the Q tile's and the key rows' first products.  A later product's differ in the address alone,
// whose 14 bits (16-byte units) hold all of shared memory, so it is added (made anew, the descriptors took longer than the products).
template <bool kFp8>
__device__ __forceinline__ void score_products(uint32_t s, uint64_t q, uint64_t k, uint32_t idesc) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // 32 bytes of dims a product: 16 bf16 of either half, or 32 codes against either term
    const uint64_t qi = q + uint64_t((i >> 2) * (kHalfBytes / 16) + (i & 3) * 2);
    const uint64_t ki = k + uint64_t((kFp8 ? 0 : (i >> 2) * (kHalfBytes / 16)) + (i & 3) * 2);
    if constexpr (kFp8)
      mma_e4m3(s, qi, ki, idesc, i != 0 ? 1u : 0u);
    else
      tc::mma_ss(s, qi, ki, idesc, i != 0 ? 1u : 0u);
  }
}

// The scores of one piece; false after a wait that ran out.  (A piece's kind, kTwo row tiles or one, is settled outside the loop:
// the loop's code stays small, and a product's descriptors are constants but for their addresses.)
template <bool kFp8, bool kTwo>
__device__ bool issue_piece_scores(const TreeParams& p, TreeSmem<kFp8>& sm, uint32_t tmem, int steps, int& tt, int& ss, int& nq) {
  using S = Shape<kFp8>;
  // (an e4m3 descriptor's type fields are zero, as f16's are)
  constexpr int kN = kTwo ? kHalfKeys : kKeys;
  constexpr uint32_t idesc = kFp8 ? tc::idesc_f16_f32(kRows, kN, 0, 0) : tc::idesc_bf16_f32(kRows, kN, 0, 0);
  uint64_t* q_in = kFp8 ? sm.q_ready : sm.q_full;
  uint64_t q[kTwo ? 2 : 1];
#pragma unroll
  for (int h = 0; h < (kTwo ? 2 : 1); ++h) {
    if (!__all_sync(kAll, wait_for(&q_in[(nq + h) & 1], ((nq + h) >> 1) & 1, p.pv.err, &sm.abort))) return false;
    q[h] = tc::smem_desc(smem_u32(sm.q[(nq + h) & 1]), 16, 1024, tc::kLayoutSw128);
  }
  for (int s = 0; s < steps; ++s, ++ss) {
    const int n = 2 * tt, slot = n % S::kRing, b = ss & 1, sub = kTwo ? s & 1 : 0;
    // (Of an odd ring the place held V of a tile at least three steps back.  The step before this one has waited for the outputs of step
    // ss - 3, and those for that V: the wait cannot take its phase for this tile's.)
    if (sub == 0 && !__all_sync(kAll, wait_for(&sm.full[slot], (n / S::kRing) & 1, p.pv.err, &sm.abort))) return false;
    const uint64_t k = tc::smem_desc(smem_u32(sm.kv[slot]) + uint32_t(sub * kHalfKeys * 128), 16, 1024, tc::kLayoutSw128);
    const bool done = !kTwo || sub == 1 || s == steps - 1;  // with the tile
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // the buffer's last P has been read; with one row tile, both groups' are
      if (ss >= 2 && !__all_sync(kAll, wait_for(&sm.pv_done[h][b], ((ss >> 1) - 1) & 1, p.pv.err, &sm.abort))) return false;
      if (!kTwo && h == 0) continue;
      tc::fence_after_sync();
      if (elect_one()) {
        if constexpr (kTwo) {
          score_products<kFp8>(tmem + uint32_t(b * kKeys + h * kHalfKeys), q[h], k, idesc);
          tc::commit(&sm.s_full[h][b]);
        } else {
          score_products<kFp8>(tmem + uint32_t(b * kKeys), q[0], k, idesc);
          tc::commit(&sm.s_full[0][b]);
          tc::commit(&sm.s_full[1][b]);
        }
        if (h == 1 && done) tc::commit(&sm.empty[slot]);
        if (h == 1 && s == steps - 1) {
          tc::commit(&sm.q_empty[nq & 1]);
          if (kTwo) tc::commit(&sm.q_empty[(nq + 1) & 1]);
        }
      }
      __syncwarp();
    }
    if (done) ++tt;
  }
  nq += kTwo ? 2 : 1;
  return true;
}

template <bool kFp8>
__device__ void issue_scores(const TreeParams& p, TreeSmem<kFp8>& sm, uint32_t tmem) {
  Piece c;
  int tt = 0, ss = 0, nq = 0;  // tiles, steps, Q tiles
  bool ok = true;
  for (int nu = 0; ok && take(p, sm, nu, c); ++nu)
    ok = c.nq > p.tile_tokens ? issue_piece_scores<kFp8, true>(p, sm, tmem, steps_of(c, true), tt, ss, nq)
                              : issue_piece_scores<kFp8, false>(p, sm, tmem, steps_of(c, false), tt, ss, nq);
}

template <bool kFp8, bool kTwo>
__device__ bool issue_piece_outputs(const TreeParams& p, TreeSmem<kFp8>& sm, uint32_t tmem, int steps, int keys, int nu, int& tt, int& ss) {
  using S = Shape<kFp8>;
  constexpr uint32_t idesc = kFp8 ? tc::idesc_f16_f32(kRows, kHeadDim, 0, 1) : tc::idesc_bf16_f32(kRows, kHeadDim, 0, 1);
  const int lane = threadIdx.x & 31;
  for (int s = 0; s < steps; ++s, ++ss) {
    const int n = 2 * tt + 1, slot = kFp8 ? tt % 2 : n % S::kRing, b = ss & 1, sub = kTwo ? s & 1 : 0;
    uint8_t* tile = kFp8 ? sm.wide[kFp8 ? slot : 0] : sm.kv[slot];
    if (sub == 0) {
      if (!__all_sync(kAll, kFp8 ? wait_for(&sm.wide_full[slot & 1], (tt >> 1) & 1, p.pv.err, &sm.abort)
                                 : wait_for(&sm.full[slot], (n / S::kRing) & 1, p.pv.err, &sm.abort)))
        return false;
      const int lim = keys - (kTwo ? s >> 1 : s) * kKeys;
      if (!kFp8 && lim < kKeys) {
        // the box of the last page brought the slots behind the last key, which may hold NaN: a weight of zero would not
        // cancel it (the rows behind that page came in as zeros)
        const int stop = min(kKeys, (max(lim, 0) + p.pv.page_size - 1) / p.pv.page_size * p.pv.page_size);
        for (int i = max(lim, 0) * 16 + lane; i < stop * 16; i += 32)
          *reinterpret_cast<uint4*>(tile + ((i >> 3) & 1) * kHalfBytes + (i >> 4) * 128 + (i & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
        __syncwarp();
      }
    }
    const bool done = !kTwo || sub == 1 || s == steps - 1;  // with the tile
    // V as B (keys x dims), MN-major: 16 keys are two 8-row groups, the second 64 dims the leading step
    const uint64_t v0 = tc::smem_desc(smem_u32(tile), kHalfBytes, 1024, tc::kLayoutSw128);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      bool ok = wait_for(&sm.p_full[h][b], (ss >> 1) & 1, p.pv.err, &sm.abort);
      // the piece's first product overwrites O once the last piece's has been read out
      if (s == 0 && h == 0 && nu > 0) ok = ok && wait_for(&sm.o_free, (nu - 1) & 1, p.pv.err, &sm.abort);
      if (!__all_sync(kAll, ok)) return false;
      tc::fence_after_sync();
      if (elect_one()) {
        const uint64_t v = v0 + uint64_t((kTwo ? sub : h) * (kHalfKeys * 128 / 16));
#pragma unroll
        for (int i = 0; i < kHalfKeys / 16; ++i)
          tc::mma_ts(tmem + kColO + uint32_t(h * kHeadDim), tmem + uint32_t(b * kKeys + h * kHalfKeys + i * 8),
                     v + uint64_t(i * (2048 / 16)), idesc, (s != 0 || i != 0) ? 1u : 0u);
        tc::commit(&sm.pv_done[h][b]);
        if (h == 1 && done) tc::commit(kFp8 ? &sm.wide_empty[slot & 1] : &sm.empty[slot]);
      }
      __syncwarp();
    }
    if (done) ++tt;
  }
  return true;
}

template <bool kFp8>
__device__ void issue_outputs(const TreeParams& p, TreeSmem<kFp8>& sm, uint32_t tmem) {
  Piece c;
  int tt = 0, ss = 0;
  bool ok = true;
  for (int nu = 0; ok && take(p, sm, nu, c); ++nu) {
    const int keys = c.lkv - c.k0 * kKeys;  // of the piece's tiles on
    ok = c.nq > p.tile_tokens ? issue_piece_outputs<kFp8, true>(p, sm, tmem, steps_of(c, true), keys, nu, tt, ss)
                              : issue_piece_outputs<kFp8, false>(p, sm, tmem, steps_of(c, false), keys, nu, tt, ss);
  }
}

// ---- softmax ---------------------------------------------------------------------------------------

// Which of the 64 keys from `base` on a row sees: those before `off`, and of the lq drafted ones behind it the
// set bits of its mask.
__device__ __forceinline__ uint64_t seen_keys(const uint32_t* mask, int words, int base, int off, int lq) {
  const int d = off - base;
  if (d >= 64) return ~0ull;
  uint64_t seen = d > 0 ? (1ull << d) - 1 : 0;
  const int u0 = max(-d, 0), word = u0 >> 5, sh = u0 & 31;
  auto get = [&](int k) -> uint32_t { return k < words ? __ldg(mask + k) : 0u; };
  const uint32_t w0 = get(word), w1 = get(word + 1), w2 = get(word + 2);
  uint64_t bits = uint64_t(__funnelshift_r(w0, w1, sh)) | uint64_t(__funnelshift_r(w1, w2, sh)) << 32;  // tokens u0 ..
  const int left = lq - u0;  // of them there are so many
  if (left < 64) bits &= left > 0 ? (1ull << left) - 1 : 0;
  return seen | (d > 0 ? bits << d : bits);
}

template <int kCap, bool kF16>
__device__ __forceinline__ void softmax_half(const TreeParams& p, float scale, uint32_t t_s, uint32_t t_o, uint64_t seen, float& m, float& l,
                                             bool first, uint64_t* pv_done, int pv_parity, int32_t* err, int* abort, bool& alive) {
  uint32_t s[kHalfKeys];
  tc::tmem_ld32(t_s, *reinterpret_cast<uint32_t(*)[32]>(s));
  tc::tmem_ld32(t_s + 32, *reinterpret_cast<uint32_t(*)[32]>(s + 32));
  tc::tmem_wait_ld();
  if (kCap) {
    const float in = scale * p.inv_cap_log2;
#pragma unroll
    for (int j = 0; j < kHalfKeys; ++j) {
      const float y = __uint_as_float(s[j]) * in;
      float th = tanh_exp2(y);
      if (kCap == 2 && y * y < kNearReach) th = y * tanh_near_factor(make_float2(y * y, 0.f)).x;
      s[j] = __float_as_uint(p.cap_log2 * th);
    }
    scale = 1.f;
  }
  if (!__all_sync(kAll, seen == ~0ull)) {
#pragma unroll
    for (int j = 0; j < kHalfKeys; ++j) s[j] = (uint32_t(seen >> (j & 32)) >> (j & 31)) & 1u ? s[j] : __float_as_uint(-INFINITY);
  }
  float mx[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) mx[j] = -INFINITY;
#pragma unroll
  for (int j = 0; j < kHalfKeys; ++j) mx[j & 7] = fmaxf(mx[j & 7], __uint_as_float(s[j]));
  const float top = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7])));
  const float m_new = fmaxf(m, top * scale);
  float alpha = 1.f;
  bool need = false;
  if (first) {
    m = m_new;
  } else {
    need = m_new > m + kRescaleThreshold;  // also from -inf to a number
    if (need) {
      alpha = fast_exp2(m - m_new);
      l *= alpha;
      m = m_new;
    }
  }
  const float m_use = m == -INFINITY ? 0.f : m;
  const float2 sc2 = make_float2(scale, scale), nm2 = make_float2(-m_use, -m_use);
  float2 sum[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) sum[j] = make_float2(0.f, 0.f);
#pragma unroll
  for (int j = 0; j < kHalfKeys / 2; ++j) {
    const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])), sc2, nm2);
    const float2 e = make_float2(fast_exp2(x.x), fast_exp2(x.y));
    sum[j & 3] = __fadd2_rn(sum[j & 3], e);
    s[j] = kF16 ? f2_to_f16x2(e.x, e.y) : f2_to_bf16x2(e.x, e.y);  // the weights are rounded as fi_run rounds them; l is not
  }
  const float2 all = __fadd2_rn(__fadd2_rn(sum[0], sum[1]), __fadd2_rn(sum[2], sum[3]));
  l += all.x + all.y;
  tc::tmem_st32(t_s, *reinterpret_cast<uint32_t(*)[32]>(s));
  tc::tmem_wait_st();
  if (__any_sync(kAll, need)) {
    alive = alive && __all_sync(kAll, wait_for(pv_done, pv_parity, err, abort));
    tc::fence_after_sync();
#pragma unroll 1
    for (int k = 0; k < 4; ++k) {
      uint32_t o[32];
      tc::tmem_ld32(t_o + 32 * k, o);
      tc::tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
      tc::tmem_st32(t_o + 32 * k, o);
    }
    tc::tmem_wait_st();
  }
}

template <bool kFp8, int kCap>
__device__ void softmax_keys(const TreeParams& p, TreeSmem<kFp8>& sm, uint32_t tmem, int h) {
  const int row = threadIdx.x & (kRows - 1), lane = threadIdx.x & 31;
  const uint32_t mine = tmem + (uint32_t(row & ~31) << 16);
  const uint32_t t_o = mine + kColO + uint32_t(h * kHeadDim);
  const int row_token = row / p.group;
  Piece c;
  int ss = 0, nu = 0, nq = 0;
  bool alive = true;
  for (; take(p, sm, nu, c); ++nu) {
    const bool two = c.nq > p.tile_tokens;
    const int first = two && h == 1 ? p.tile_tokens : 0;              // this group's tokens of the piece
    const int tokens = min(p.tile_tokens, c.nq - first);
    const bool busy = (row & ~31) < tokens * p.group;  // the warp has rows of the piece
    const uint32_t* mask = p.mask + (long long)(c.q0 + first + min(row_token, tokens - 1)) * p.mask_words;
    const int off = c.lkv - c.lq, steps = steps_of(c, two);
    const int base0 = c.k0 * kKeys + (two ? 0 : h * kHalfKeys), base_step = two ? kHalfKeys : kKeys;
    float m = -INFINITY, l = 0.f, scale = p.scale_log2;
    for (int s = 0; s < steps; ++s, ++ss) {
      const int b = ss & 1;
      const uint64_t seen = busy ? seen_keys(mask, p.mask_words, base0 + s * base_step, off, c.lq) : 0;
      alive = alive && __all_sync(kAll, wait_for(&sm.s_full[h][b], (ss >> 1) & 1, p.pv.err, &sm.abort));
      if (kFp8 && s == 0) {  // the row's scale, once the products have seen the tile; then the Q tiles may go
        const int e = sm.q_exp[(nq + (two ? h : 0)) & 1][row];
        // (never 0, however small the row and k_scale: 0 times the -inf of an unseen key would be NaN)
        scale = e == kQuiet ? __uint_as_float(0x7fc00000u) : fmaxf(scale * __uint_as_float(uint32_t(e + 127) << 23), __uint_as_float(1u));
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.q_empty[nq & 1]);
        if (lane == 0 && two) mbar_arrive(&sm.q_empty[(nq + 1) & 1]);
        nq += two ? 2 : 1;
      }
      if (alive && busy) {
        tc::fence_after_sync();
        const uint32_t t_s = mine + uint32_t(b * kKeys + h * kHalfKeys);
        uint64_t* before = &sm.pv_done[h][b ^ 1];  // the product that wrote O last
        const int parity = ((ss - 1) >> 1) & 1;
        softmax_half<kCap, kFp8>(p, scale, t_s, t_o, seen, m, l, s == 0, before, parity, p.pv.err, &sm.abort, alive);
        tc::fence_before_sync();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.p_full[h][b]);
    }
    if (nu >= 1) alive = alive && __all_sync(kAll, wait_for(&sm.stat_empty, (nu - 1) & 1, p.pv.err, &sm.abort));
    sm.stat_m[h][row] = m;
    sm.stat_l[h][row] = l;
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.stat_full);
  }
}

__device__ __forceinline__ void tmem_ld16(uint32_t at, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(at));
}

// 16 dims of a row: to the output in bf16, or to a partial slot.  A slot takes 32 bytes a store, a whole sector; the caller's output is
// aligned to 16 bytes and takes two stores (32 requests of 64 tokens over 2 to 8 K keys: 171.6 us, 170.1 with one; 16 tokens: no difference).
__device__ __forceinline__ void put32(void* to, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]),
               "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ void put16(const TreeParams& p, bool whole, long long row, int dim, const float (&v)[16]) {
  uint32_t w[8];
  if (whole) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = f2_to_bf16x2(v[2 * j], v[2 * j + 1]);
    uint4* to = reinterpret_cast<uint4*>(p.o + row * kHeadDim + dim);
    to[0] = make_uint4(w[0], w[1], w[2], w[3]);
    to[1] = make_uint4(w[4], w[5], w[6], w[7]);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(v[8 * h + j]);
      put32(p.part_o + row * kHeadDim + dim + 8 * h, w);
    }
  }
}

// A finished piece, to the output or as a state to its slot: with one row tile the two groups' states of the same rows
// joined, with two each group's own.
template <bool kFp8>
__device__ void write_pieces(const TreeParams& p, TreeSmem<kFp8>& sm, uint32_t tmem) {
  const int row = threadIdx.x & (kRows - 1), lane = threadIdx.x & 31;
  const uint32_t mine = tmem + (uint32_t(row & ~31) << 16) + kColO;
  Piece c, ahead;
  int ss = 0, nu = 0, nq = 0;
  bool alive = true, more = take(p, sm, 0, ahead);
  auto split = [&]() {  // the Q tiles of the piece ahead, while the one at hand is worked on
    if constexpr (kFp8) {
      for (int left = ahead.nq; left > 0 && alive; left -= p.tile_tokens, ++nq) alive = split_q(p, sm, nq, (threadIdx.x >> 5) & 3);
    }
  };
  if (more) split();
  for (; more; ++nu) {
    c = ahead;
    more = take(p, sm, nu + 1, ahead);
    if (more) split();
    const bool two = c.nq > p.tile_tokens;
    alive = alive && __all_sync(kAll, wait_for(&sm.stat_full, nu & 1, p.pv.err, &sm.abort));
    float m[2] = {sm.stat_m[0][row], sm.stat_m[1][row]}, l[2] = {sm.stat_l[0][row], sm.stat_l[1][row]};
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.stat_empty);
    ss += steps_of(c, two);
    const int last = ss - 1;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      alive = alive && __all_sync(kAll, wait_for(&sm.pv_done[h][last & 1], (last >> 1) & 1, p.pv.err, &sm.abort));
    tc::fence_after_sync();
    const bool whole = c.slot < 0;
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      const int first = h * p.tile_tokens, rows = min(p.tile_tokens, c.nq - first) * p.group;  // of this pass
      if ((row & ~31) >= rows) break;
      // the states' weights: o = w0 O_0 + w1 O_1
      float w0, w1, lse2 = -INFINITY;
      const float m0 = two && h == 1 ? -INFINITY : m[0], m1 = two && h == 0 ? -INFINITY : m[1];
      const float top = fmaxf(m0, m1);
      w0 = w1 = 0.f;
      const float l0 = two && h == 1 ? 0.f : l[0], l1 = two && h == 0 ? 0.f : l[1];
      if (top != -INFINITY || l0 != l0 || l1 != l1) {  // (a row of NaN has no maximum and a sum of NaN)
        w0 = m0 == top ? 1.f : fast_exp2(m0 - top);
        w1 = m1 == top ? 1.f : fast_exp2(m1 - top);
        const float sum = w0 * l0 + w1 * l1;
        lse2 = top + fast_log2(sum);
        const float inv = p.v_scale / sum;
        w0 *= inv;
        w1 *= inv;
      }
      const bool write = row < rows;
      const long long at = whole ? (long long)(c.q0 + first + row / p.group) * p.hqo + c.head * p.group + row % p.group
                                 : ((long long)c.slot * 2 + h) * kRows + row;
#pragma unroll 1
      for (int k = 0; k < kHeadDim; k += 16) {
        // (a group without a seen key, or of other rows, has nothing to add, not even 0 x NaN)
        float v[16];
        uint32_t a[16], b[16];
        tmem_ld16(mine + k, a);
        tmem_ld16(mine + kHeadDim + k, b);
        tc::tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float x = w0 != 0.f ? __uint_as_float(a[j]) * w0 : 0.f;
          v[j] = w1 != 0.f ? fmaf(__uint_as_float(b[j]), w1, x) : x;
        }
        if (write) put16(p, whole, at, k, v);
      }
      if (write) {
        if (whole)
          p.lse[at] = lse2 * kLn2;
        else
          p.part_lse[at] = lse2;
      }
      if (!two) break;
    }
    tc::fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.o_free);
  }
}

template <bool kFp8, int kCap>
__global__ void __launch_bounds__(Shape<kFp8>::kThreads, 1)
    tree_kernel(const __grid_constant__ TreeParams p, const __grid_constant__ CUtensorMap tm_q,
                const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
  using S = Shape<kFp8>;
  // the kernel has no static shared memory, so this starts at the CTA's first (1024-byte aligned) address; the
  // check below holds it to that, the swizzled tiles need it
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  TreeSmem<kFp8>& sm = *reinterpret_cast<TreeSmem<kFp8>*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sm.q_full[b], 1);
      mbar_init(&sm.q_empty[b], kFp8 ? 1 + 8 : 1);  // the products; e4m3: and the softmax warps
      mbar_init(&sm.q_ready[b], 4);
      mbar_init(&sm.wide_full[b], 4);
      mbar_init(&sm.wide_empty[b], 1);
      for (int h = 0; h < 2; ++h) {
        mbar_init(&sm.s_full[h][b], 1);
        mbar_init(&sm.p_full[h][b], 4);
        mbar_init(&sm.pv_done[h][b], 1);
      }
    }
    for (int i = 0; i < S::kRing; ++i) {
      mbar_init(&sm.full[i], kLoaders);
      mbar_init(&sm.empty[i], kFp8 && i % 2 == 1 ? 4 : 1);  // e4m3: V's codes are read by the widening warps
    }
    for (int i = 0; i < kPieces; ++i) {
      mbar_init(&sm.piece_full[i], 1);
      mbar_init(&sm.piece_empty[i], S::kReaders);
    }
    mbar_init(&sm.stat_full, 8);
    mbar_init(&sm.stat_empty, 4);
    mbar_init(&sm.o_free, 4);
    sm.abort = 0;
    fence_mbar_init();
  }
  if (warp == 12 && lane == 0) {
    tc::tma_prefetch_desc(&tm_q);
    tc::tma_prefetch_desc(&tm_k);
    tc::tma_prefetch_desc(&tm_v);
  }
  if (warp == 16) {
    tc::tmem_alloc(&sm.tmem_base, kTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sm.tmem_base;
  const GeoHead plan = load_head(p.pv.geo);
  const int start = __ldg(p.starts + blockIdx.x);
  const Line line(plan.tree, int(gridDim.x));
  wait_prior_grid();  // (the plan was there before the kernel that this one waits for)
  if ((tmem & 0xFFFFu) + kTmemCols > 512u || (smem_u32(smem_raw) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicOr(p.pv.err, FI_DEVERR_TMEM);
  } else if (int(blockIdx.x) < line.ctas) {
    if (warp < 8) {
      tc::regs_increase<S::kSoftmaxRegs>();
      softmax_keys<kFp8, kCap>(p, sm, tmem, warp >> 2);
    } else if (warp < 12) {
      if constexpr (S::kWriteRegs < S::kLaunchRegs) tc::regs_decrease<S::kWriteRegs>();
      write_pieces<kFp8>(p, sm, tmem);
    } else if (warp < 16) {
      tc::regs_decrease<S::kLoadRegs>();
      load_tiles<kFp8>(p, sm, &tm_q, &tm_k, &tm_v, warp - 12);
    } else if (warp < 20) {
      tc::regs_decrease<S::kIssueRegs>();
      if (warp == 16)
        issue_scores<kFp8>(p, sm, tmem);
      else if (warp == 17)
        issue_outputs<kFp8>(p, sm, tmem);
      else if (warp == 18)
        find_pieces<kFp8>(p, sm, plan, line, int(blockIdx.x), start);
    } else if constexpr (kFp8) {
      tc::regs_decrease<S::kWidenRegs>();
      widen_tiles(p, sm, warp - 20);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 16) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

// ---- units that were cut -------------------------------------------------------------------------------
// kJoinCtas CTAs for each place where the line was cut; those of one unit's cuts share its rows and join their states in
// the pieces' order.  What a row has to read, n states of 516 bytes, lies in L2, and most units have two or three pieces, so
// latency counts: a warp takes two rows at a time, whose LSEs (sixteen lanes a row) and first states (all lanes, four dims each) are
// asked for at once.  (A row a warp: 30 us behind 160 us of 256-row units.)
constexpr int kJoinThreads = 256;
constexpr int kJoinCtas = 4;
constexpr int kJoinAhead = 4;

__global__ void __launch_bounds__(kJoinThreads, 4) tree_join_kernel(const __grid_constant__ TreeParams p, int grid) {
  // The plan was there before the kernel whose states this one joins, so it is read before the wait.  Every CTA waits, those
  // with nothing to join too: a grid that ended before the one it depends on would let its own followers start.
  const GeoHead plan = load_head(p.pv.geo);
  const Line line(plan.tree, grid);
  const int cut = int(blockIdx.x) / kJoinCtas + 1, part = int(blockIdx.x) % kJoinCtas;
  const int lane = threadIdx.x & 31, warp = int(threadIdx.x >> 5);
  const int x = cut * line.per;
  const Geo g = load_geo(p.pv.geo, cut < line.ctas ? __ldg(p.starts + cut) : 0);
  const int tokens = 2 * p.tile_tokens;
  const int tiles = max(1, (g.lkv + kKeys - 1) / kKeys), sets = (g.lq + tokens - 1) / tokens;
  const int unit = (x - g.tree0) / tiles, a = g.tree0 + unit * tiles;
  const int begins = a / line.per, n = (a + tiles - 1) / line.per - begins + 1;  // the CTA with the unit's first piece, pieces
  const long long first = 2ll * begins;
  const int head = unit / max(1, sets), set = unit - head * sets, q0 = g.q0 + set * tokens, nq = min(tokens, g.lq - set * tokens);
  // row k of the unit lies at 128 h + x of a slot, for row x of its row tile h
  const int tile_rows = p.tile_tokens * p.group, rows = nq * p.group;
  auto place = [&](int k) { return first * 2 * kRows + (k < tile_rows ? k : kRows + k - tile_rows); };
  const int warps = max(1, n - 1) * kJoinCtas * (kJoinThreads / 32);
  wait_prior_grid();
  if (cut >= line.ctas || a == x) return;  // nothing is cut here
  for (int k0 = 2 * (((cut - 1 - begins) * kJoinCtas + part) * (kJoinThreads / 32) + warp); k0 < rows; k0 += 2 * warps) {
    const long long at[2] = {place(k0), place(min(k0 + 1, rows - 1))};
    // sixteen lanes a row: lane (row, i) holds the LSE of state i, then its weight
    const float* lses = p.part_lse + (lane < 16 ? at[0] : at[1]);
    auto lse_of = [&](int i) { return i < n ? __ldcg(lses + (long long)i * 2 * kRows) : -INFINITY; };
    auto states = [&](int i0, float4 (&v)[2][kJoinAhead]) {  // states i0 .. of both rows, four dims a lane
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int e = 0; e < kJoinAhead; ++e)
          v[r][e] = i0 + e < n ? __ldcg(reinterpret_cast<const float4*>(p.part_o + (at[r] + (long long)(i0 + e) * 2 * kRows) * kHeadDim) + lane)
                               : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    const float own = lse_of(lane & 15);
    float4 v[2][kJoinAhead];
    states(0, v);  // the first states' numbers come with their LSEs
    float m = own;
    for (int i = 16 + (lane & 15); i < n; i += 16) m = fmaxf(m, lse_of(i));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
    m = m == -INFINITY ? 0.f : m;
    float sum = fast_exp2(own - m);
    for (int i = 16 + (lane & 15); i < n; i += 16) sum += fast_exp2(lse_of(i) - m);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;  // (no state of the row has seen a key)
    if ((lane & 15) == 0 && k0 + (lane >> 4) < rows) {
      const int k = k0 + (lane >> 4);
      p.lse[(long long)(q0 + k / p.group) * p.hqo + head * p.group + k % p.group] = sum == 0.f ? -INFINITY : (m + fast_log2(sum)) * kLn2;
    }
    float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    for (int i0 = 0; i0 < n; i0 += kJoinAhead) {
      if (i0 > 0) states(i0, v);
      const float w = (i0 < 16 ? fast_exp2(own - m) : fast_exp2(lse_of((i0 & ~15) + (lane & 15)) - m)) * inv;
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int e = 0; e < kJoinAhead; ++e) {
          const float we = __shfl_sync(kAll, w, 16 * r + ((i0 + e) & 15));
          if (we == 0.f) continue;
          acc[r].x = fmaf(we, v[r][e].x, acc[r].x);
          acc[r].y = fmaf(we, v[r][e].y, acc[r].y);
          acc[r].z = fmaf(we, v[r][e].z, acc[r].z);
          acc[r].w = fmaf(we, v[r][e].w, acc[r].w);
        }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int k = k0 + r;
      if (k >= rows) continue;
      const long long orow = (long long)(q0 + k / p.group) * p.hqo + head * p.group + k % p.group;
      *reinterpret_cast<uint2*>(p.o + orow * kHeadDim + 4 * lane) = make_uint2(f2_to_bf16x2(acc[r].x, acc[r].y), f2_to_bf16x2(acc[r].z, acc[r].w));
    }
  }
}

// ---- the accepted path ---------------------------------------------------------------------------------
// A warp a (request, KV head): the rows of up to 16 accepted tokens are read, K and V, before the first of them is
// written; path entries ascend, so a later entry's row is never one that an earlier entry has overwritten.  The bytes
// are few (a path of six tokens of 8 heads: 48 KB a request); what counts is the chain plan, path, page id, row (512 requests,
// up to 17 tokens, e4m3: 5.8 us; 32 requests 2.6).
constexpr int kCommitRows = 16;

template <bool kFp8>
__global__ void __launch_bounds__(128) commit_kernel(const __grid_constant__ CommitParams p) {
  constexpr int kElem = kFp8 ? 1 : 2, kLanes = kHeadDim * kElem / 16;  // lanes of a row
  constexpr int kSide = 32 / kLanes, kSteps = kCommitRows / kSide;     // rows at a time
  const PageView& pv = p.pv;
  const int batch = load_head(pv.geo).batch;
  wait_prior_grid();
  const int lane = threadIdx.x & 31;
  const long long tasks = (long long)batch * pv.hkv;
  for (long long task = (long long)blockIdx.x * 4 + (threadIdx.x >> 5); task < tasks; task += (long long)gridDim.x * 4) {
    const int r = int(task / pv.hkv), head = int(task % pv.hkv);
    const Geo g = load_geo(pv.geo, r);
    const int32_t* path = p.path + (long long)r * p.path_len;
    const int off = g.lkv - g.lq, most = min(p.path_len, g.lq);
    for (int j0 = 0; j0 < most; j0 += kCommitRows) {
      // lane j looks entry j0 + j up
      const int j = j0 + lane;
      int e = lane < kCommitRows && j < most ? __ldg(path + j) : -1;
      const unsigned ends = __ballot_sync(kAll, e < 0);  // the path ends at its first -1
      if (ends & ((2u << lane) - 1)) e = -1;
      long long from = -1, to = -1;
      if (e >= 0) {
        const int before = j > 0 ? __ldg(path + j - 1) : -1;
        int sp, ss, dp, ds;
        if (e <= before || e < j || e >= g.lq)
          atomicOr(pv.err, FI_DEVERR_KEPT);
        else if (e != j && off + j >= 0 && locate(pv, g.kv0, off + e, sp, ss) && locate(pv, g.kv0, off + j, dp, ds)) {
          from = kv_offset(pv, sp, ss, head);
          to = kv_offset(pv, dp, ds, head);
        }
      }
      const unsigned moved = __ballot_sync(kAll, from >= 0);
      if (moved != 0) {
        uint4 k[kSteps], v[kSteps];
        long long at[kSteps];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const int row = i * kSide + lane / kLanes;
          const long long src = __shfl_sync(kAll, from, row);
          at[i] = __shfl_sync(kAll, to, row);
          if (src >= 0) {
            const long long byte = src * kElem + (lane % kLanes) * 16;
            k[i] = __ldcg(reinterpret_cast<const uint4*>(static_cast<const char*>(p.k_pages) + byte));
            v[i] = __ldcg(reinterpret_cast<const uint4*>(static_cast<const char*>(p.v_pages) + byte));
          }
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          if (at[i] < 0) continue;
          const long long byte = at[i] * kElem + (lane % kLanes) * 16;
          *reinterpret_cast<uint4*>(static_cast<char*>(p.k_pages) + byte) = k[i];
          *reinterpret_cast<uint4*>(static_cast<char*>(p.v_pages) + byte) = v[i];
        }
        __syncwarp();
      }
      if (ends & ((1u << kCommitRows) - 1)) break;
    }
  }
}

// ---- launches ------------------------------------------------------------------------------------------

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &found) == cudaSuccess &&
        found == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// Pages of either layout as (dim, KV head, token in page, page); a box is one page and head, 64 dims of bf16 or 128 codes,
// 128B-swizzled.
bool page_map(CUtensorMap* m, const void* base, const PageView& pv, bool fp8) {
  const cuuint64_t e = fp8 ? 1 : 2;
  const cuuint64_t dims[4] = {cuuint64_t(kHeadDim), cuuint64_t(pv.hkv), cuuint64_t(pv.page_size), cuuint64_t(pv.num_pages)};
  const cuuint64_t strides[3] = {pv.head_stride * e, pv.tok_stride * e, pv.page_stride * e};
  const cuuint32_t box[4] = {fp8 ? 128u : 64u, 1u, cuuint32_t(pv.page_size), 1u}, step[4] = {1u, 1u, 1u, 1u};
  return encoder()(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims,
                   strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// q as (dim, head, token); a box is 64 dims of the rows of a tile.
bool query_map(CUtensorMap* m, const TreeParams& p, int total_q) {
  const cuuint64_t row = cuuint64_t(kHeadDim) * 2;
  const cuuint64_t dims[3] = {cuuint64_t(kHeadDim), cuuint64_t(p.hqo), cuuint64_t(total_q)}, strides[2] = {row, row * p.hqo};
  const cuuint32_t box[3] = {64u, cuuint32_t(p.group), cuuint32_t(p.tile_tokens)}, step[3] = {1u, 1u, 1u};
  return encoder()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<__nv_bfloat16*>(p.q), dims, strides, box, step,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

int launch_tree(const TreeParams& p, int total_q, bool fp8, int num_sms, cudaStream_t stream) {
  if (encoder() == nullptr) return record_cuda_error(cudaErrorNotSupported, "cuTensorMapEncodeTiled entry point");
  CUtensorMap tq, tk, tv;
  if (!query_map(&tq, p, total_q) || !page_map(&tk, p.k_pages, p.pv, fp8) || !page_map(&tv, p.v_pages, p.pv, fp8))
    return FI_ERR_INVALID_ARG;
  static_assert(sizeof(TreeSmem<false>) <= 227 * 1024 && sizeof(TreeSmem<true>) <= 227 * 1024, "shared memory of a CTA");
  using Kernel = void (*)(const TreeParams, const CUtensorMap, const CUtensorMap, const CUtensorMap);
  static const Kernel kernels[6] = {tree_kernel<false, 0>, tree_kernel<false, 1>, tree_kernel<false, 2>,
                                    tree_kernel<true, 0>,  tree_kernel<true, 1>,  tree_kernel<true, 2>};
  static PerDevice once;
  cudaError_t e = once.run([&] {
    cudaError_t st = cudaSuccess;
    for (int i = 0; i < 6 && st == cudaSuccess; ++i)
      st = cudaFuncSetAttribute(kernels[i], cudaFuncAttributeMaxDynamicSharedMemorySize,
                                int(i < 3 ? sizeof(TreeSmem<false>) : sizeof(TreeSmem<true>)));
    return st;
  });
  if (e != cudaSuccess) return record_cuda_error(e, "cudaFuncSetAttribute(tree_kernel)");
  const int cap = p.cap_log2 > 0.f ? (p.wide_cap ? 2 : 1) : 0;
  e = launch_dependent(kernels[(fp8 ? 3 : 0) + cap], unsigned(num_sms), fp8 ? Shape<true>::kThreads : Shape<false>::kThreads,
                       fp8 ? sizeof(TreeSmem<true>) : sizeof(TreeSmem<false>), 1, stream, p, tq, tk, tv);
  if (e != cudaSuccess) return record_cuda_error(e, "tree_kernel launch");
  if (num_sms == 1) return FI_OK;  // one piece of line: nothing is cut
  e = launch_dependent(tree_join_kernel, unsigned(num_sms - 1) * kJoinCtas, kJoinThreads, 0, 1, stream, p, num_sms);
  return e == cudaSuccess ? FI_OK : record_cuda_error(e, "tree_join_kernel launch");
}

int launch_commit(const CommitParams& p, int most_batch, bool fp8, int num_sms, cudaStream_t stream) {
  const long long ctas = ((long long)most_batch * p.pv.hkv + 3) / 4;
  const unsigned grid = unsigned(std::min<long long>(ctas, (long long)num_sms * 8));
  const cudaError_t e = fp8 ? launch_dependent(commit_kernel<true>, grid, 128, 0, 1, stream, p)
                            : launch_dependent(commit_kernel<false>, grid, 128, 0, 1, stream, p);
  return e == cudaSuccess ? FI_OK : record_cuda_error(e, "commit_kernel launch");
}

}  // namespace fi
