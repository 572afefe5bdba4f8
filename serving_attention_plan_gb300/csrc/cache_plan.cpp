// Host side of the cache operators: request geometry, page conditions, rotary frequencies.
#include <algorithm>
#include <cmath>
#include <exception>
#include <vector>

#include "../../include/fi.h"
#include "cache_ops.h"
#include "tree_ops.h"

namespace fi {

GeoTotals fill_geo(const int32_t* qo_indptr, const int32_t* kv_indptr, const int32_t* last_page_len, int batch,
                   int page_size, Geo* out) {
  GeoTotals t;
  int64_t tiles = 0;
  for (int i = 0; i <= batch; ++i) {
    Geo g{};
    g.q0 = qo_indptr[i];
    g.kv0 = kv_indptr[i];
    g.blk0 = int32_t(t.blocks);
    g.tile0 = int32_t(tiles);
    if (i < batch) {
      const int32_t pages = kv_indptr[i + 1] - kv_indptr[i];
      // at most 2^30, as the planner accepts
      const int64_t keys = pages > 0 ? int64_t(pages - 1) * page_size + last_page_len[i] : 0;
      g.lq = qo_indptr[i + 1] - qo_indptr[i];
      g.lkv = int32_t(keys);
      t.blocks += (keys + kBlkKeys - 1) / kBlkKeys;
      tiles += (keys + kTileKeys - 1) / kTileKeys;
      t.max_lkv = std::max(t.max_lkv, g.lkv);
    }
    out[i] = g;
  }
  t.ok = t.blocks <= INT32_MAX;
  return t;
}

void split_weights(Geo* geo, int batch, int hkv, int group, int row_limit, bool causal, int window, GeoTotals* totals) {
  int64_t work = 0, blocks = 0;
  for (int i = 0; i <= batch; ++i) {
    geo[i].work0 = int32_t(work);
    geo[i].blk0 = int32_t(blocks);
    if (i == batch) break;
    if (int64_t(geo[i].lq) * group <= row_limit) {
      blocks += (int64_t(geo[i].lkv) + kBlkKeys - 1) / kBlkKeys;
      continue;
    }
    int64_t head = 0;
    for (int kt = 0; int64_t(kt) * kTileKeys < geo[i].lkv; ++kt) {
      int t0, tokens, cost;
      weight_item(geo[i].lq, geo[i].lkv, kt, causal, window, kWeightTileRows / group, &t0, &tokens, &cost);
      head += cost;
    }
    work += head * hkv;
    if (work > INT32_MAX) {  // not with the tensor cores: all requests as they were
      blocks = 0;
      for (int k = 0; k <= batch; ++k) {
        geo[k].work0 = 0;
        geo[k].blk0 = int32_t(blocks);
        if (k < batch) blocks += (int64_t(geo[k].lkv) + kBlkKeys - 1) / kBlkKeys;
      }
      return;
    }
  }
  totals->blocks = blocks;
  totals->work = work;
}

bool fill_tree(Geo* geo, int batch, int hkv, int group, int ctas, int32_t* total, int32_t* starts) {
  const int tokens = 2 * (kTreeRows / group);  // of a unit: two row tiles
  int64_t tiles = 0;
  for (int i = 0; i <= batch; ++i) {
    geo[i].tree0 = int32_t(tiles);
    if (i == batch) break;
    const int64_t keys = std::max<int64_t>(1, (int64_t(geo[i].lkv) + kTreeKeys - 1) / kTreeKeys);
    tiles += int64_t(hkv) * ((int64_t(geo[i].lq) + tokens - 1) / tokens) * keys;
    if (tiles > INT32_MAX / 2) return false;  // a CTA's end of the line stays in 32 bits
  }
  *total = int32_t(tiles);
  const int64_t per = std::max<int64_t>(kTreeLeastTiles, (tiles + ctas - 1) / ctas);
  for (int c = 0, r = 0; c < ctas; ++c) {
    while (r + 1 < batch && geo[r + 1].tree0 <= c * per) ++r;
    starts[c] = r;
  }
  return true;
}

int check_pages_once(const int32_t* a, int64_t na, const int32_t* b, int64_t nb, int32_t max_page) {
  if (na + nb == 0) return FI_OK;  // max_page is -1
  try {
    std::vector<uint64_t> seen((size_t(max_page) >> 6) + 1, 0);
    uint64_t twice = 0;  // no branch in the loop
    auto scan = [&](const int32_t* idx, int64_t n) {
      for (int64_t k = 0; k < n; ++k) {
        uint64_t& w = seen[size_t(idx[k]) >> 6];
        const uint64_t bit = uint64_t(1) << (idx[k] & 63);
        twice |= w & bit;
        w |= bit;
      }
    };
    scan(a, na);
    scan(b, nb);
    return twice == 0 ? FI_OK : FI_ERR_UNSUPPORTED;
  } catch (const std::exception&) {
    return FI_ERR_CAPACITY;
  }
}

int check_tails_once(const Geo* geo, const int32_t* kv_indices, int batch, int page_size, const int32_t* shared,
                     int64_t n_shared) {
  try {
    std::vector<int32_t> pages;
    for (int i = 0; i < batch; ++i) {
      const Geo& g = geo[i];
      if (g.lq == 0 || g.lkv == 0) continue;
      const int first = std::max(0, g.lkv - g.lq) / page_size, last = (g.lkv - 1) / page_size;
      pages.insert(pages.end(), kv_indices + g.kv0 + first, kv_indices + g.kv0 + last + 1);
    }
    std::sort(pages.begin(), pages.end());
    bool once = std::adjacent_find(pages.begin(), pages.end()) == pages.end();
    for (int64_t k = 0; k < n_shared && once; ++k) once = !std::binary_search(pages.begin(), pages.end(), shared[k]);
    return once ? FI_OK : FI_ERR_UNSUPPORTED;
  } catch (const std::exception&) {
    return FI_ERR_CAPACITY;
  }
}

uint64_t turns_fraction(double inv_freq) {
  double turns = inv_freq / 6.283185307179586476925286766559;
  turns -= std::floor(turns);
  const double scaled = std::ldexp(turns, 64);
  return scaled >= 18446744073709551616.0 ? 0 : static_cast<uint64_t>(scaled);
}

}  // namespace fi
