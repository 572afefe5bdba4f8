// Attention of a tree of drafted tokens over a paged cache, and the move of the accepted path's keys.
//
//   o = softmax(x) V,  x = scale q.k (soft-cap: cap tanh(x / cap)),  over the keys that a row sees:
//   key j of a request of l_q tokens and l_kv keys is seen by token t if j < l_kv - l_q, or if bit
//   j - (l_kv - l_q) of t's mask is set.
//
// What bounds it: a tree has 8 to 64 tokens, so a KV head has 32 to 512 query rows; up to 128 rows a key costs
// 2 * 128 * 128 products for 512 bytes, which the tensor cores do in a third of the time that the bytes take.  The tile is
// therefore 128 rows of one KV head (rows are (token, head of the group) pairs) and the kernel is built to
// stream keys; more rows are further tiles, whose keys come from L2.
//
// Split: the 128-key tiles of all (request, KV head, row tile) units form one line, and every CTA takes an equal piece
// of it, wherever that cuts a unit.  Nothing of this is planned on the host but the line's prefix per request, so a captured
// launch follows later plans.  A unit that was cut leaves partial states, which a second launch joins in order.
//
// One CTA an SM.  The keys of a tile are worked on in two halves of 64, each with its own running maximum,
// sum and accumulator, so that two softmax groups keep the tensor cores and each other busy; the halves are
// joined when the unit's piece is written.
//   warps 0-3, 4-7    softmax of keys 0-63 and 64-127 of every tile; a thread owns a row (TMEM lane)
//   warps 8-11        the two halves of a finished piece joined, to the output or to a partial slot
//   warps 12-15       TMA of page boxes, every stage's boxes dealt to the four (one warp's issue ends at 4 TB/s)
//   warp 16, 17       issue of S = Q K^T (128 x 128) and of O_h += P_h V_h
//   warps 20-23       e4m3 pages: codes widened to f16, exactly, from a ring of their own
// TMEM: two score buffers of 128 columns (P overwrites a half's first 32), O_0 and O_1.
// Shared memory: two Q tiles; bf16: five K / V tiles; e4m3: three widened tiles and four of codes.
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

// Registers of a thread per warpgroup.  Launched with 96 (bf16, 640 threads) or 80 (e4m3, 768), 480 for a thread of each
// warpgroup together; the shares below add up to that.
template <bool kFp8>
struct Shape {
  static constexpr int kThreads = kFp8 ? 768 : 640;
  static constexpr int kLaunchRegs = kFp8 ? 80 : 96;
  static constexpr uint32_t kSoftmaxRegs = kFp8 ? 144 : 160;
  static constexpr uint32_t kJoinRegs = 80;
  static constexpr uint32_t kLoadRegs = kFp8 ? 32 : 40;
  static constexpr uint32_t kIssueRegs = kFp8 ? 32 : 40;
  static constexpr uint32_t kWidenRegs = kFp8 ? 48 : 0;
  static_assert(2 * kSoftmaxRegs + kJoinRegs + kLoadRegs + kIssueRegs + kWidenRegs == kLaunchRegs * (kThreads / 128),
                "the warpgroups' registers are those of the launch");
  static constexpr int kTiles = kFp8 ? 3 : 5;  // K / V tiles that the products read
  static constexpr int kRaw = kFp8 ? 4 : 0;    // tiles of codes
  static constexpr int kRing = kFp8 ? kRaw : kTiles;  // tiles that TMA fills
};

template <bool kFp8>
struct TreeSmem {
  uint8_t q[2][kTileBytes];  // [2 dim halves][128 rows][128 B], 128B-swizzled
  uint8_t kv[Shape<kFp8>::kTiles][kTileBytes];
  uint8_t raw[kFp8 ? Shape<kFp8>::kRaw : 1][kFp8 ? kHalfBytes : 16];  // [128 keys][128 codes]
  float stat_m[2][kRows], stat_l[2][kRows];
  uint64_t q_full[2], q_empty[2], q_ready[2];
  uint64_t full[Shape<kFp8>::kRing], raw_empty[kFp8 ? Shape<kFp8>::kRaw : 1];
  uint64_t ready[Shape<kFp8>::kTiles], empty[Shape<kFp8>::kTiles];  // ready: e4m3, widened
  uint64_t s_full[2], p_full[2][2], pv_done[2][2];  // [half][buffer]
  uint64_t stat_full, stat_empty, o_free;
  uint32_t tmem_base;
  int abort;
};

// ---- the line of tiles ---------------------------------------------------------------------------

struct Line {
  int total, per, ctas;  // tiles; of a CTA; CTAs that have any
  __device__ Line(int tiles, int grid) : total(tiles) {
    per = max(kTreeLeastTiles, (total + grid - 1) / grid);
    ctas = (total + per - 1) / per;
  }
};

// A run of tiles of one (request, KV head, row tile) unit.
struct Piece {
  int q0, nq;         // its first query token, tokens
  int kv0, lkv, lq;   // the request's first page entry, keys, tokens
  int head;
  int k0, k1;         // tiles [k0, k1) of the unit's
  int slot;           // partial slot, or -1 for a whole unit
};

// The pieces of a part [pos, end) of the line, in order.
struct Walk {
  const Geo* geo;
  int batch, hkv, tokens;  // tokens of a row tile
  int pos, end, per, cta;
  int r, tiles, row_tiles, unit, at;  // request, tiles and row tiles of its units, the unit's number, next tile
  Geo g;

  __device__ __forceinline__ void enter() {
    g = load_geo(geo, r);
    tiles = max(1, (g.lkv + kKeys - 1) / kKeys);
    row_tiles = (g.lq + tokens - 1) / tokens;
  }
  // A whole warp; the part is not empty.
  __device__ void init(const TreeParams& p, const GeoHead& plan, const Line& line, int cta_) {
    geo = p.pv.geo;
    batch = plan.batch;
    hkv = p.pv.hkv;
    tokens = p.tile_tokens;
    per = line.per;
    cta = cta_;
    pos = cta * per;
    end = min(line.total, pos + per);
    r = find_request(geo, batch, &Geo::tree0, pos);
    enter();
    const int in = pos - g.tree0;
    unit = in / tiles;
    at = in - unit * tiles;
  }
  __device__ __forceinline__ bool next(Piece& c) {
    if (pos >= end) return false;
    while (unit == hkv * row_tiles) {
      ++r;
      unit = 0;
      at = 0;
      enter();
    }
    const int tile = unit % row_tiles;
    c.head = unit / row_tiles;
    c.q0 = g.q0 + tile * tokens;
    c.nq = min(tokens, g.lq - tile * tokens);
    c.kv0 = g.kv0;
    c.lkv = g.lkv;
    c.lq = g.lq;
    c.k0 = at;
    c.k1 = at + min(tiles - at, end - pos);
    const int a = pos - at, first = a / per;  // the unit's place on the line, the CTA that begins it
    c.slot = (a + tiles - 1) / per != first ? 2 * first + (cta - first) : -1;
    pos += c.k1 - c.k0;
    at = 0;
    ++unit;
    return true;
  }
};

__device__ __forceinline__ bool elect_one() {
  uint32_t on;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(on));
  return on != 0;
}

// ---- loads -----------------------------------------------------------------------------------------

// Loader warp `w` of four: its share of the boxes of every tile, K and V in turn.  A box is one page and KV head, 64 dims
// (bf16, 128B-swizzled) or 128 codes (e4m3); pages behind the request's last read as zeros.
template <bool kFp8>
__device__ void load_tiles(const TreeParams& p, TreeSmem<kFp8>& sm, Walk walk, const CUtensorMap* tm_q,
                           const CUtensorMap* tm_k, const CUtensorMap* tm_v, int w) {
  using S = Shape<kFp8>;
  const int lane = threadIdx.x & 31;
  const int ps = p.pv.page_size, pages = kKeys / ps;
  const int boxes = kFp8 ? pages : 2 * pages;
  const int mine = w + kLoaders * lane;  // this lane's box
  const int page = kFp8 ? mine : mine >> 1, half = kFp8 ? 0 : mine & 1;
  const uint32_t bytes = uint32_t((boxes - w + kLoaders - 1) / kLoaders) * uint32_t(ps) * 128u;
  const uint32_t place = uint32_t(half) * kHalfBytes + uint32_t(page * ps) * 128u;
  uint8_t* ring = kFp8 ? sm.raw[0] : sm.kv[0];
  constexpr int kStep = kFp8 ? kHalfBytes : kTileBytes;
  uint64_t* empty = kFp8 ? sm.raw_empty : sm.empty;
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
  int n = 0, nu = 0;  // tiles and pieces issued
  bool ok = true, more = walk.next(c);
  int t = more ? c.k0 : 0;
  int z_next = more ? locate(c, t) : 0;
  while (more && ok) {
    const int z = z_next, head = c.head;
    if (t == c.k0) {
      if (w == 0) {
        const int b = nu & 1;
        if (nu >= 2) ok = __all_sync(kAll, mbar_wait(&sm.q_empty[b], ((nu >> 1) - 1) & 1, p.pv.err, &sm.abort));
        if (ok && lane == 0) {
          mbar_arrive_expect_tx(&sm.q_full[b], p.q_tile_bytes);
          tc::tma_load_3d(sm.q[b], tm_q, 0, head * p.group, c.q0, &sm.q_full[b]);
          tc::tma_load_3d(sm.q[b] + kHalfBytes, tm_q, 64, head * p.group, c.q0, &sm.q_full[b]);
        }
        __syncwarp();
        if (!ok) break;
      }
      ++nu;
    }
    if (++t == c.k1) {
      more = walk.next(c);
      t = c.k0;
    }
    if (more) z_next = locate(c, t);  // lands while this tile waits for its place
    for (int v = 0; v < 2; ++v, ++n) {
      const int slot = n % S::kRing;
      if (n >= S::kRing) ok = __all_sync(kAll, mbar_wait(&empty[slot], (n / S::kRing - 1) & 1, p.pv.err, &sm.abort));
      if (!ok) break;
      if (lane == 0) mbar_arrive_expect_tx(&sm.full[slot], bytes);
      __syncwarp();
      if (mine < boxes) tc::tma_load_4d(ring + slot * kStep + place, v ? tm_v : tm_k, 64 * half, head, 0, z, &sm.full[slot]);
    }
  }
  // no copy is left landing in this CTA's shared memory
  if (w == 0)
    for (int k = max(0, nu - 2); k < nu; ++k) mbar_wait_bounded(&sm.q_full[k & 1], (k >> 1) & 1);
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

// e4m3: widening warp `w` of four takes 32 rows of every tile: eight lanes read one row of codes and write it as f16 in the
// products' layout (16-byte chunk c of a 64-dim half's row r at c ^ (r % 8)).  The lanes of the second half write
// their odd chunk first, so that a row's eight lanes fill different banks.  Rows behind the last key become zeros: a page's
// unused slots may hold NaN, which a weight of zero would not cancel.  Each piece's Q tile turns from bf16 to f16 in
// place (exact within f16's normal range).
__device__ void widen_tiles(const TreeParams& p, TreeSmem<true>& sm, Walk walk, int w) {
  using S = Shape<true>;
  const int lane = threadIdx.x & 31, chunk = lane & 7;
  const uint32_t half_off = uint32_t(chunk >> 2) * kHalfBytes;
  const bool swap = chunk >= 4;
  const int m = (2 * chunk) & 7;
  Piece c;
  int n = 0, nu = 0;
  bool ok = true;
  while (ok && walk.next(c)) {
    const int b = nu & 1;
    ok = __all_sync(kAll, mbar_wait(&sm.q_full[b], (nu >> 1) & 1, p.pv.err, &sm.abort));
    if (!ok) break;
    const uint32_t q = smem_u32(sm.q[b]) + uint32_t(w * (kTileBytes / 4) + lane * 16);
#pragma unroll 4
    for (int i = 0; i < kTileBytes / 4 / 512; ++i) {
      uint32_t x[4];
      asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(q + 512 * i) : "memory");
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = f2_to_f16x2(__uint_as_float(x[k] << 16), __uint_as_float(x[k] & 0xffff0000u));
      asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(q + 512 * i), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]) : "memory");
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.q_ready[b]);
    ++nu;
    for (int t = c.k0; t < c.k1 && ok; ++t) {
      const int lim = c.lkv - t * kKeys;
      for (int v = 0; v < 2; ++v, ++n) {
        const int from = n % S::kRaw, to = n % S::kTiles;
        ok = __all_sync(kAll, mbar_wait(&sm.full[from], (n / S::kRaw) & 1, p.pv.err, &sm.abort) &&
                                  (n < S::kTiles || mbar_wait(&sm.empty[to], (n / S::kTiles - 1) & 1, p.pv.err, &sm.abort)));
        if (!ok) break;
        const int r0 = 32 * w + (lane >> 3);
        const uint32_t src = smem_u32(sm.raw[from]) + uint32_t(r0 * 128 + 16 * chunk);
        const uint32_t dst = smem_u32(sm.kv[to]) + half_off + uint32_t(r0 * 128);
#pragma unroll
        for (int i0 = 0; i0 < 8; i0 += 4) {
          uint32_t x[4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(x[i][0]), "=r"(x[i][1]), "=r"(x[i][2]), "=r"(x[i][3])
                         : "r"(src + 512 * (i0 + i))
                         : "memory");
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = r0 + 4 * (i0 + i);
            if (r >= lim) x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0u;
            const uint32_t a0 = e4m3x2_to_f16x2(swap ? x[i][2] : x[i][0]), a1 = e4m3x2_to_f16x2((swap ? x[i][2] : x[i][0]) >> 16);
            const uint32_t a2 = e4m3x2_to_f16x2(swap ? x[i][3] : x[i][1]), a3 = e4m3x2_to_f16x2((swap ? x[i][3] : x[i][1]) >> 16);
            const uint32_t b0 = e4m3x2_to_f16x2(swap ? x[i][0] : x[i][2]), b1 = e4m3x2_to_f16x2((swap ? x[i][0] : x[i][2]) >> 16);
            const uint32_t b2 = e4m3x2_to_f16x2(swap ? x[i][1] : x[i][3]), b3 = e4m3x2_to_f16x2((swap ? x[i][1] : x[i][3]) >> 16);
            const uint32_t row = dst + 512 * (i0 + i);
            const int ca = (swap ? m + 1 : m) ^ (r & 7), cb = (swap ? m : m + 1) ^ (r & 7);
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(row + 16 * ca), "r"(a0), "r"(a1), "r"(a2), "r"(a3) : "memory");
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(row + 16 * cb), "r"(b0), "r"(b1), "r"(b2), "r"(b3) : "memory");
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sm.ready[to]);
          mbar_arrive(&sm.raw_empty[from]);
        }
      }
    }
  }
}

// ---- products ----------------------------------------------------------------------------------------
// One warp issues S, another O; an elected lane of a uniform warp (a branch on the lane number costs each product 50
// clocks and more).

template <bool kFp8>
__device__ void issue_scores(const TreeParams& p, TreeSmem<kFp8>& sm, Walk walk, uint32_t tmem) {
  using S = Shape<kFp8>;
  constexpr uint32_t idesc = kFp8 ? tc::idesc_f16_f32(kRows, kKeys, 0, 0) : tc::idesc_bf16_f32(kRows, kKeys, 0, 0);
  uint64_t* k_in = kFp8 ? sm.ready : sm.full;
  uint64_t* q_in = kFp8 ? sm.q_ready : sm.q_full;
  const bool leads = elect_one();
  Piece c;
  int tt = 0, nu = 0;
  while (walk.next(c)) {
    if (!__all_sync(kAll, mbar_wait(&q_in[nu & 1], (nu >> 1) & 1, p.pv.err, &sm.abort))) return;
    const uint32_t q = smem_u32(sm.q[nu & 1]);
    for (int t = c.k0; t < c.k1; ++t, ++tt) {
      const int n = 2 * tt, slot = n % S::kTiles, b = tt & 1;
      bool ok = mbar_wait(&k_in[slot], (n / S::kTiles) & 1, p.pv.err, &sm.abort);
      if (tt >= 2)  // the buffer's last P has been read
        ok = ok && mbar_wait(&sm.pv_done[0][b], ((tt >> 1) - 1) & 1, p.pv.err, &sm.abort) &&
             mbar_wait(&sm.pv_done[1][b], ((tt >> 1) - 1) & 1, p.pv.err, &sm.abort);
      if (!__all_sync(kAll, ok)) return;
      tc::fence_after_sync();
      if (leads) {
        const uint32_t k = smem_u32(sm.kv[slot]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t off = uint32_t(i >> 2) * kHalfBytes + uint32_t(i & 3) * 32;
          tc::mma_ss(tmem + uint32_t(b * kKeys), tc::smem_desc(q + off, 16, 1024, tc::kLayoutSw128),
                     tc::smem_desc(k + off, 16, 1024, tc::kLayoutSw128), idesc, i != 0 ? 1u : 0u);
        }
        tc::commit(&sm.s_full[b]);
        tc::commit(&sm.empty[slot]);
        if (t == c.k1 - 1) tc::commit(&sm.q_empty[nu & 1]);
      }
      __syncwarp();
    }
    ++nu;
  }
}

template <bool kFp8>
__device__ void issue_outputs(const TreeParams& p, TreeSmem<kFp8>& sm, Walk walk, uint32_t tmem) {
  using S = Shape<kFp8>;
  constexpr uint32_t idesc = kFp8 ? tc::idesc_f16_f32(kRows, kHeadDim, 0, 1) : tc::idesc_bf16_f32(kRows, kHeadDim, 0, 1);
  uint64_t* v_in = kFp8 ? sm.ready : sm.full;
  const bool leads = elect_one();
  const int lane = threadIdx.x & 31;
  Piece c;
  int tt = 0, nu = 0;
  while (walk.next(c)) {
    for (int t = c.k0; t < c.k1; ++t, ++tt) {
      const int n = 2 * tt + 1, slot = n % S::kTiles, b = tt & 1;
      if (!__all_sync(kAll, mbar_wait(&v_in[slot], (n / S::kTiles) & 1, p.pv.err, &sm.abort))) return;
      const int lim = c.lkv - t * kKeys;
      if (!kFp8 && lim < kKeys) {
        // the box of the last page brought the slots behind the last key, which may hold NaN: a weight of zero would not
        // cancel it (the rows behind that page came in as zeros)
        const int stop = min(kKeys, (max(lim, 0) + p.pv.page_size - 1) / p.pv.page_size * p.pv.page_size);
        for (int i = max(lim, 0) * 16 + lane; i < stop * 16; i += 32)
          *reinterpret_cast<uint4*>(sm.kv[slot] + ((i >> 3) & 1) * kHalfBytes + (i >> 4) * 128 + (i & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
        __syncwarp();
      }
      const uint32_t v = smem_u32(sm.kv[slot]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        bool ok = mbar_wait(&sm.p_full[h][b], (tt >> 1) & 1, p.pv.err, &sm.abort);
        // the piece's first product overwrites O once the last piece's has been read out
        if (t == c.k0 && h == 0 && nu > 0) ok = ok && mbar_wait(&sm.o_free, (nu - 1) & 1, p.pv.err, &sm.abort);
        if (!__all_sync(kAll, ok)) return;
        tc::fence_after_sync();
        if (leads) {
#pragma unroll
          for (int i = 0; i < kHalfKeys / 16; ++i)
            // V as B (keys x dims), MN-major: 16 keys are two 8-row groups, the second 64 dims the leading step
            tc::mma_ts(tmem + kColO + uint32_t(h * kHeadDim), tmem + uint32_t(b * kKeys + h * kHalfKeys + i * 8),
                       tc::smem_desc(v + uint32_t(h * kHalfKeys * 128 + i * 2048), kHalfBytes, 1024, tc::kLayoutSw128), idesc,
                       (t != c.k0 || i != 0) ? 1u : 0u);
          tc::commit(&sm.pv_done[h][b]);
          if (h == 1) tc::commit(&sm.empty[slot]);
        }
        __syncwarp();
      }
    }
    ++nu;
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

template <bool kMasked, int kCap, bool kF16>
__device__ __forceinline__ void softmax_half(const TreeParams& p, uint32_t t_s, uint32_t t_o, uint64_t seen, float& m, float& l,
                                             bool first, uint64_t* pv_done, int pv_parity, int32_t* err, int* abort, bool& alive) {
  uint32_t s[kHalfKeys];
  tc::tmem_ld32(t_s, *reinterpret_cast<uint32_t(*)[32]>(s));
  tc::tmem_ld32(t_s + 32, *reinterpret_cast<uint32_t(*)[32]>(s + 32));
  tc::tmem_wait_ld();
  float scale = p.scale_log2;
  if (kCap) {
    const float in = p.scale_log2 * p.inv_cap_log2;
#pragma unroll
    for (int j = 0; j < kHalfKeys; ++j) {
      const float y = __uint_as_float(s[j]) * in;
      float th = tanh_exp2(y);
      if (kCap == 2 && y * y < kNearReach) th = y * tanh_near_factor(make_float2(y * y, 0.f)).x;
      s[j] = __float_as_uint(p.cap_log2 * th);
    }
    scale = 1.f;
  }
  float mx[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) mx[j] = -INFINITY;
#pragma unroll
  for (int j = 0; j < kHalfKeys; ++j) {
    if (kMasked) s[j] = (uint32_t(seen >> (j & 32)) >> (j & 31)) & 1u ? s[j] : __float_as_uint(-INFINITY);
    mx[j & 7] = fmaxf(mx[j & 7], __uint_as_float(s[j]));
  }
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
    alive = alive && __all_sync(kAll, mbar_wait(pv_done, pv_parity, err, abort));
    tc::fence_after_sync();
#pragma unroll
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
__device__ void softmax_keys(const TreeParams& p, TreeSmem<kFp8>& sm, Walk walk, uint32_t tmem, int h) {
  const int row = threadIdx.x & (kRows - 1), lane = threadIdx.x & 31;
  const uint32_t mine = tmem + (uint32_t(row & ~31) << 16);
  const uint32_t t_o = mine + kColO + uint32_t(h * kHeadDim);
  const int token = row / p.group;
  Piece c;
  int tt = 0, nu = 0;
  bool alive = true;
  while (walk.next(c)) {
    const bool busy = (row & ~31) < c.nq * p.group;  // the warp has rows of the piece
    const uint32_t* mask = p.mask + (long long)(c.q0 + min(token, c.nq - 1)) * p.mask_words;
    const int off = c.lkv - c.lq;
    float m = -INFINITY, l = 0.f;
    for (int t = c.k0; t < c.k1; ++t, ++tt) {
      const int b = tt & 1;
      const int base = t * kKeys + h * kHalfKeys;
      const uint64_t seen = busy ? seen_keys(mask, p.mask_words, base, off, c.lq) : 0;
      alive = alive && __all_sync(kAll, mbar_wait(&sm.s_full[b], (tt >> 1) & 1, p.pv.err, &sm.abort));
      if (alive && busy) {
        tc::fence_after_sync();
        const uint32_t t_s = mine + uint32_t(b * kKeys + h * kHalfKeys);
        uint64_t* before = &sm.pv_done[h][b ^ 1];  // the product that wrote O last
        const int parity = ((tt - 1) >> 1) & 1;
        if (__all_sync(kAll, seen == ~0ull))
          softmax_half<false, kCap, kFp8>(p, t_s, t_o, seen, m, l, t == c.k0, before, parity, p.pv.err, &sm.abort, alive);
        else
          softmax_half<true, kCap, kFp8>(p, t_s, t_o, seen, m, l, t == c.k0, before, parity, p.pv.err, &sm.abort, alive);
        tc::fence_before_sync();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.p_full[h][b]);
    }
    if (nu >= 1) alive = alive && __all_sync(kAll, mbar_wait(&sm.stat_empty, (nu - 1) & 1, p.pv.err, &sm.abort));
    sm.stat_m[h][row] = m;
    sm.stat_l[h][row] = l;
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.stat_full);
    ++nu;
  }
}

__device__ __forceinline__ void tmem_ld16(uint32_t at, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(at));
}

// The two halves of a finished piece, joined: to the output, or as a state to the piece's slot.
template <bool kFp8>
__device__ void join_halves(const TreeParams& p, TreeSmem<kFp8>& sm, Walk walk, uint32_t tmem) {
  const int row = threadIdx.x & (kRows - 1), lane = threadIdx.x & 31;
  const uint32_t mine = tmem + (uint32_t(row & ~31) << 16) + kColO;
  Piece c;
  int tt = 0, nu = 0;
  bool alive = true;
  while (walk.next(c)) {
    alive = alive && __all_sync(kAll, mbar_wait(&sm.stat_full, nu & 1, p.pv.err, &sm.abort));
    const float m0 = sm.stat_m[0][row], m1 = sm.stat_m[1][row], l0 = sm.stat_l[0][row], l1 = sm.stat_l[1][row];
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.stat_empty);
    tt += c.k1 - c.k0;
    const int last = tt - 1;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      alive = alive && __all_sync(kAll, mbar_wait(&sm.pv_done[h][last & 1], (last >> 1) & 1, p.pv.err, &sm.abort));
    tc::fence_after_sync();
    const float m = fmaxf(m0, m1);
    float w0 = 0.f, w1 = 0.f, lse2 = -INFINITY;
    if (m != -INFINITY) {
      w0 = fast_exp2(m0 - m);
      w1 = fast_exp2(m1 - m);
      const float l = w0 * l0 + w1 * l1;
      lse2 = m + fast_log2(l);
      const float inv = p.v_scale / l;
      w0 *= inv;
      w1 *= inv;
    }
    const int rows = c.nq * p.group;
    const bool write = row < rows;
    const long long orow = (long long)(c.q0 + row / p.group) * p.hqo + c.head * p.group + row % p.group;
    const long long srow = (long long)c.slot * kRows + row;
    if ((row & ~31) < rows) {
#pragma unroll 1
      for (int k = 0; k < kHeadDim; k += 16) {
        uint32_t a[16], b[16];
        tmem_ld16(mine + k, a);
        tmem_ld16(mine + kHeadDim + k, b);
        tc::tmem_wait_ld();
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {  // a half without a seen key has nothing to add, not even 0 x NaN
          const float x = w0 != 0.f ? __uint_as_float(a[j]) * w0 : 0.f;
          v[j] = w1 != 0.f ? fmaf(__uint_as_float(b[j]), w1, x) : x;
        }
        if (!write) continue;
        if (c.slot < 0) {
          uint4* to = reinterpret_cast<uint4*>(p.o + orow * kHeadDim + k);
#pragma unroll
          for (int j = 0; j < 2; ++j)
            to[j] = make_uint4(f2_to_bf16x2(v[8 * j], v[8 * j + 1]), f2_to_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                               f2_to_bf16x2(v[8 * j + 4], v[8 * j + 5]), f2_to_bf16x2(v[8 * j + 6], v[8 * j + 7]));
        } else {
          float4* to = reinterpret_cast<float4*>(p.part_o + srow * kHeadDim + k);
#pragma unroll
          for (int j = 0; j < 4; ++j) to[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        }
      }
    }
    tc::fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.o_free);
    if (write) {
      if (c.slot < 0)
        p.lse[orow] = lse2 * kLn2;
      else
        p.part_lse[srow] = lse2;
    }
    ++nu;
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
      mbar_init(&sm.q_empty[b], 1);
      mbar_init(&sm.q_ready[b], 4);
      mbar_init(&sm.s_full[b], 1);
      for (int h = 0; h < 2; ++h) {
        mbar_init(&sm.p_full[h][b], 4);
        mbar_init(&sm.pv_done[h][b], 1);
      }
    }
    for (int i = 0; i < S::kRing; ++i) mbar_init(&sm.full[i], kLoaders);
    for (int i = 0; i < S::kRaw; ++i) mbar_init(&sm.raw_empty[i], 4);
    for (int i = 0; i < S::kTiles; ++i) {
      mbar_init(&sm.ready[i], 4);
      mbar_init(&sm.empty[i], 1);
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
  wait_prior_grid();
  const uint32_t tmem = sm.tmem_base;
  const GeoHead plan = load_head(p.pv.geo);
  const Line line(plan.tree, int(gridDim.x));
  if ((tmem & 0xFFFFu) + kTmemCols > 512u || (smem_u32(smem_raw) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicOr(p.pv.err, FI_DEVERR_TMEM);
  } else if (int(blockIdx.x) < line.ctas) {
    Walk walk;
    walk.init(p, plan, line, int(blockIdx.x));
    if (warp < 8) {
      tc::regs_increase<S::kSoftmaxRegs>();
      softmax_keys<kFp8, kCap>(p, sm, walk, tmem, warp >> 2);
    } else if (warp < 12) {
      if constexpr (S::kJoinRegs < S::kLaunchRegs) tc::regs_decrease<S::kJoinRegs>();
      join_halves<kFp8>(p, sm, walk, tmem);
    } else if (warp < 16) {
      tc::regs_decrease<S::kLoadRegs>();
      load_tiles<kFp8>(p, sm, walk, &tm_q, &tm_k, &tm_v, warp - 12);
    } else if (warp < 20) {
      tc::regs_decrease<S::kIssueRegs>();
      if (warp == 16)
        issue_scores<kFp8>(p, sm, walk, tmem);
      else if (warp == 17)
        issue_outputs<kFp8>(p, sm, walk, tmem);
    } else if constexpr (kFp8) {
      tc::regs_decrease<S::kWidenRegs>();
      widen_tiles(p, sm, walk, warp - 20);
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
// kJoinCtas CTAs for each place where the line was cut: if it is the first cut of a unit, they join the unit's states in
// the pieces' order, a warp a row, four dims a lane.  What a row has to read, n states of 516 bytes, lies in L2.
constexpr int kJoinThreads = 256;
constexpr int kJoinCtas = 4;
constexpr int kJoinAhead = 8;

__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const __grid_constant__ TreeParams p, int grid) {
  wait_prior_grid();
  const GeoHead plan = load_head(p.pv.geo);
  const Line line(plan.tree, grid);
  const int cut = int(blockIdx.x) / kJoinCtas + 1, part = int(blockIdx.x) % kJoinCtas;
  if (cut >= line.ctas) return;
  const int lane = threadIdx.x & 31;
  const int x = cut * line.per;
  Geo g = load_geo(p.pv.geo, find_request(p.pv.geo, plan.batch, &Geo::tree0, x));
  const int tiles = max(1, (g.lkv + kKeys - 1) / kKeys), row_tiles = (g.lq + p.tile_tokens - 1) / p.tile_tokens;
  const int unit = (x - g.tree0) / tiles, a = g.tree0 + unit * tiles;
  if (a == x || a / line.per != cut - 1) return;  // nothing is cut here, or it was cut before
  const int n = (a + tiles - 1) / line.per - (cut - 1) + 1;
  const long long first = 2ll * (cut - 1);
  const int tile = unit % row_tiles, head = unit / row_tiles;
  const int q0 = g.q0 + tile * p.tile_tokens, rows = min(p.tile_tokens, g.lq - tile * p.tile_tokens) * p.group;
  for (int row = part * (kJoinThreads / 32) + (threadIdx.x >> 5); row < rows; row += kJoinCtas * (kJoinThreads / 32)) {
    const float* lses = p.part_lse + first * kRows + row;
    float m = -INFINITY;
    for (int k = lane; k < n; k += 32) m = fmaxf(m, __ldcg(lses + (long long)k * kRows));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
    const float m_use = m == -INFINITY ? 0.f : m;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
    const float4* src = reinterpret_cast<const float4*>(p.part_o + (first * kRows + row) * kHeadDim) + lane;
    for (int k0 = 0; k0 < n; k0 += 32) {
      const float w = k0 + lane < n ? fast_exp2(__ldcg(lses + (long long)(k0 + lane) * kRows) - m_use) : 0.f;
      sum += w;
      const int some = min(32, n - k0);
      for (int j = 0; j < some; j += kJoinAhead) {
        float4 v[kJoinAhead];
#pragma unroll
        for (int k = 0; k < kJoinAhead; ++k)
          v[k] = j + k < some ? __ldcg(src + (long long)(k0 + j + k) * (kRows * kHeadDim / 4)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kJoinAhead; ++k) {
          const float wk = __shfl_sync(kAll, w, (j + k) & 31);
          if (wk == 0.f) continue;
          acc.x = fmaf(wk, v[k].x, acc.x);
          acc.y = fmaf(wk, v[k].y, acc.y);
          acc.z = fmaf(wk, v[k].z, acc.z);
          acc.w = fmaf(wk, v[k].w, acc.w);
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    const float inv = m == -INFINITY ? 0.f : 1.f / sum;
    const long long orow = (long long)(q0 + row / p.group) * p.hqo + head * p.group + row % p.group;
    *reinterpret_cast<uint2*>(p.o + orow * kHeadDim + 4 * lane) =
        make_uint2(f2_to_bf16x2(acc.x * inv, acc.y * inv), f2_to_bf16x2(acc.z * inv, acc.w * inv));
    if (lane == 0) p.lse[orow] = m == -INFINITY ? -INFINITY : (m + fast_log2(sum)) * kLn2;
  }
}

// ---- the accepted path ---------------------------------------------------------------------------------
// A warp a (request, KV head): the rows of up to 16 accepted tokens are read, K and V, before the first of them is
// written; path entries ascend, so a later entry's row is never one that an earlier entry has overwritten.  The bytes
// are few (a path of six tokens of 8 heads: 48 KB a request); what counts is the chain plan, path, page id, row.
constexpr int kCommitRows = 16;

template <bool kFp8>
__global__ void __launch_bounds__(128) commit_kernel(const __grid_constant__ CommitParams p) {
  constexpr int kElem = kFp8 ? 1 : 2, kLanes = kHeadDim * kElem / 16;  // lanes of a row
  constexpr int kSide = 32 / kLanes, kSteps = kCommitRows / kSide;     // rows at a time
  wait_prior_grid();
  const PageView& pv = p.pv;
  const int batch = load_head(pv.geo).batch;
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

// Pages of either layout as (dim, KV head, token in page, page); a box is one page and head, 64 dims of bf16
// (128B-swizzled) or 128 codes.
bool page_map(CUtensorMap* m, const void* base, const PageView& pv, bool fp8) {
  const cuuint64_t e = fp8 ? 1 : 2;
  const cuuint64_t dims[4] = {cuuint64_t(kHeadDim), cuuint64_t(pv.hkv), cuuint64_t(pv.page_size), cuuint64_t(pv.num_pages)};
  const cuuint64_t strides[3] = {pv.head_stride * e, pv.tok_stride * e, pv.page_stride * e};
  const cuuint32_t box[4] = {fp8 ? 128u : 64u, 1u, cuuint32_t(pv.page_size), 1u}, step[4] = {1u, 1u, 1u, 1u};
  return encoder()(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims,
                   strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, fp8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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
