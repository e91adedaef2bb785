// Host half of a latent decode step (paged_decode_plan with KV_PLAN_LATENT).
//
// Work is cut for pairs of CTAs (decode_latent.cu): an item is up to 128 query
// rows (branches x heads of a shared segment, or one branch's heads) over a
// range of logical blocks.  Every pair gets a list of items of about the same
// cost: the units' blocks are dealt out in order, and a unit that does not fit
// the rest of a pair's share goes on in the next pair's, cut on a 128-token
// tile.  The cost of an item is its tiles plus a fixed part (the query load,
// the first tile's latency, the epilogue), so that a step of many short items
// is balanced too, and no piece is cut shorter than two tiles.
//
// Items of at most 16 rows run on one SM each (decode_latent_few.cu), in lists of
// their own; the other items' lists come first in the plan.  The two kernels run
// beside each other, each on the SMs that its share of the work is worth.  Where
// there is little work of few rows all of it is the pairs'.
//
// An item whose branches' rows all lie in one item each writes their output; the
// other branches' partial results are merged, all heads of a branch one way.

#include <algorithm>
#include <cstring>
#include <numeric>
#include <utility>

#include "internal.h"

namespace pkv {
namespace {

struct LatentUnit {
  int32_t branch0, row0, nrows, blk_begin, blk_end, masked;
};

constexpr int kTileBlocks = 8;  // blocks of a 128-token tile
constexpr int kMinTiles = 2;    // the shortest piece of a unit (few rows: 1)
// Costs in half tiles (0.85 us): a tile, and an item's fixed part -- measured on
// steps of long and of short items: about 3.5 us, and 3 to 5 us more for 128 rows
// of partial results.
constexpr int kTileCost = 2;
// For few rows, in tiles' worth of an SM's time (3.3 us a 128-token tile, where
// HBM brings every SM its share): about 3 us.
int32_t item_cost(int32_t nrows, bool few) { return few ? 2 : 4 + nrows / 32; }

struct Piece {
  int32_t unit, lo, hi;  // blocks
};

int32_t tiles(int32_t blocks) { return (blocks + kTileBlocks - 1) / kTileBlocks; }

// Deal the units `which` out to `bins` lists (few: of items of few rows) of at most
// `share` cost each; returns whether they fit.
bool deal(const std::vector<LatentUnit>& units, const std::vector<int32_t>& which,
          int64_t share, int32_t bins, bool few, std::vector<Piece>* out,
          std::vector<int32_t>* ptr) {
  out->clear();
  ptr->assign(1, 0);
  const int32_t least = few ? 1 : kMinTiles;
  int64_t used = 0;  // cost of the list being filled
  for (int32_t u : which) {
    int32_t lo = units[u].blk_begin;
    while (lo < units[u].blk_end) {
      const int32_t left = tiles(units[u].blk_end - lo);
      const int32_t fixed = item_cost(units[u].nrows, few);
      int64_t room = (share - used - fixed) / kTileCost;  // tiles
      if (used > 0 && room < std::min(left, least)) {
        ptr->push_back((int32_t)out->size());
        if ((int32_t)ptr->size() > bins) return false;
        used = 0;
        room = (share - fixed) / kTileCost;
      }
      room = std::max<int64_t>(room, least);
      // The rest of the unit is not left shorter than the shortest piece.
      int32_t take = left;
      if (left > room) {
        take = (int32_t)room;
        if (left - take < least) take = left - least;
        if (take < least) take = left;
      }
      const int32_t hi =
          std::min(units[u].blk_end, lo + take * kTileBlocks);
      out->push_back({u, lo, hi});
      used += (int64_t)take * kTileCost + fixed;
      lo = hi;
    }
  }
  ptr->push_back((int32_t)out->size());
  return (int32_t)ptr->size() - 1 <= bins;
}

}  // namespace

kv_status latent_plan(int32_t nb, int32_t Hq, int32_t max_blocks,
                      const int32_t* nblk, const int32_t* groups,
                      int32_t n_groups, const int32_t* shared_end,
                      int32_t num_sms, int32_t flags, int32_t* plan,
                      int64_t plan_cap, kv_decode_plan_info* info) {
  (void)max_blocks;
  if ((int64_t)nb * Hq > INT32_MAX / 2)
    return fail(KV_ERR_INVALID_ARG, "nb x Hq too large");
  std::vector<LatentUnit> units;
  auto add = [&](int32_t b0, int64_t rows, int32_t lo, int32_t hi, int32_t masked) {
    for (int64_t r = 0; r < rows; r += kTileRows)
      units.push_back({b0, (int32_t)r,
                       (int32_t)std::min<int64_t>(kTileRows, rows - r), lo, hi,
                       masked});
  };
  std::vector<int32_t> n_units(nb, 0);
  for (int32_t i = 0; i < n_groups; ++i) {
    const int32_t* s = groups + 4 * (int64_t)i;
    add(s[0], (int64_t)s[1] * Hq, s[2], s[2] + s[3], 0);
    for (int32_t b = s[0]; b < s[0] + s[1]; ++b) ++n_units[b];
  }
  for (int32_t b = 0; b < nb; ++b)
    if (shared_end[b] < nblk[b]) {
      add(b, Hq, shared_end[b], nblk[b], 1);
      ++n_units[b];
    }
  // Longest first: the short ones fill the shares' ends.
  std::stable_sort(units.begin(), units.end(),
                   [](const LatentUnit& x, const LatentUnit& y) {
                     return x.blk_end - x.blk_begin > y.blk_end - y.blk_begin;
                   });
  const int32_t pairs_max = std::max(1, num_sms / 2);
  std::vector<Piece> pieces;
  std::vector<int32_t> ptr[2];  // the pairs' lists, the SMs' lists of few rows
  int64_t chunk = 0;
  std::vector<int32_t> kind[2];
  for (int32_t u = 0; u < (int32_t)units.size(); ++u)
    kind[units[u].nrows <= kLatentFewRows].push_back(u);
  auto cost_of = [&](const std::vector<int32_t>& which, bool few) {
    int64_t c = 0;
    for (int32_t u : which)
      c += (int64_t)tiles(units[u].blk_end - units[u].blk_begin) * kTileCost +
           item_cost(units[u].nrows, few);
    return c;
  };
  int64_t total_cost[2] = {cost_of(kind[0], false), cost_of(kind[1], true)};
  int32_t lists_max[2] = {pairs_max, 2 * pairs_max};
  if (!kind[0].empty() && !kind[1].empty()) {
    // Times, spread over all pairs: 0.7 us a pair and 0.94 us an SM for a unit of
    // cost.  The second kernel starts some 2 us after the first, so that a step
    // whose few rows the pairs would not take much longer for runs in the pairs'
    // kernel alone (17 branches of 16 heads and 100 tokens on a segment of 256 24.6
    // us instead of 26.6; 16 branches of 32752 tokens on a segment of 16 run in both,
    // 108.7 us instead of 122.5).  Of 130 steps with 4 to 140
    // branches measured in both ways a limit of 2.5 us picks one that is 0.6%
    // slower than the faster on average; 1.5 and 4.5 us 1.2% and 0.8%, the pairs
    // alone 5.8%, both always 3.9%.
    const double us = 1.0 / pairs_max;
    const double many = 0.7 * us * total_cost[0], few = 0.47 * us * total_cost[1];
    const double alone = many + 0.7 * us * cost_of(kind[1], false);
    if (alone - (many + few) <= 2.5) {
      kind[0].resize(units.size());
      std::iota(kind[0].begin(), kind[0].end(), 0);
      kind[1].clear();
      total_cost[0] = cost_of(kind[0], false);
    } else {
      // SMs in proportion (8 roots x 64 branches: 108 us; with 1.1 us an SM 113,
      // with 0.8 113; one kind after the other on all SMs 123).
      lists_max[0] = std::max(
          1, std::min(pairs_max - 1, (int32_t)(pairs_max * many / (many + few) + 0.5)));
      lists_max[1] = std::max(1, 2 * (pairs_max - lists_max[0]));
    }
  }
  std::vector<Piece> dealt[2];
  std::vector<int32_t> cuts[2];
  for (int few = 1; few >= 0; --few) {
    cuts[few].assign(1, 0);
    if (kind[few].empty()) continue;
    const int32_t bins = lists_max[few];
    int64_t share = std::max<int64_t>((total_cost[few] + bins - 1) / bins,
                                      kTileCost * (few ? 1 : kMinTiles));
    while (!deal(units, kind[few], share, bins, few, &dealt[few], &cuts[few]))
      share += std::max<int64_t>(1, share / 50);
    chunk = std::max(chunk, share);
  }
  for (int few = 0; few < 2; ++few) {
    const int32_t at = (int32_t)pieces.size();
    pieces.insert(pieces.end(), dealt[few].begin(), dealt[few].end());
    for (int32_t c : cuts[few]) ptr[few].push_back(at + c);
  }
  const int32_t n_few = (int32_t)dealt[1].size();
  const int32_t n_pairs = (int32_t)ptr[0].size() - 1;
  const int32_t n_lists = (int32_t)ptr[1].size() - 1;

  // Pieces of each unit; a branch is finished by its items when it lies in one
  // unit (per row tile) of one piece, and so do the branches beside it there.
  std::vector<int32_t> n_pieces(units.size(), 0);
  for (const Piece& p : pieces) ++n_pieces[p.unit];
  std::vector<char> single(nb, 1);
  auto branches_of = [&](const LatentUnit& x) {  // [first, second)
    return std::pair<int32_t, int32_t>(
        x.branch0 + x.row0 / Hq, x.branch0 + (x.row0 + x.nrows - 1) / Hq + 1);
  };
  for (size_t u = 0; u < units.size(); ++u) {
    const auto [b0, b1] = branches_of(units[u]);
    for (int32_t b = b0; b < b1; ++b)
      if (n_units[b] != 1 || n_pieces[u] != 1) single[b] = 0;
  }
  // A unit finishes all of its rows or none, so a branch that shares a unit with a
  // merged one is merged too; one whose heads lie in two units of a segment (Hq does
  // not divide 128) hands that on to the next unit.  A segment's units are next to
  // one another in row order: a pass up and a pass down reach the ends of a chain.
  std::vector<char> direct(units.size(), 1);
  auto settle = [&](size_t u) {
    const auto [b0, b1] = branches_of(units[u]);
    for (int32_t b = b0; b < b1; ++b)
      if (!single[b]) direct[u] = 0;
    if (!direct[u]) std::fill(single.begin() + b0, single.begin() + b1, 0);
  };
  for (size_t u = 0; u < units.size(); ++u) settle(u);
  for (size_t u = units.size(); u-- > 0;) settle(u);
  struct Tagged { int32_t branch; MergeEntry e; };
  std::vector<Tagged> merge;
  std::vector<WorkItem> items;
  items.reserve(pieces.size());
  int64_t prow = 0;
  for (const Piece& p : pieces) {
    const LatentUnit& u = units[p.unit];
    const int32_t row1 = u.row0 + u.nrows;
    const bool done = direct[p.unit] != 0;
    // `g` (there is one kv-head) says whether the item writes the output.
    items.push_back({u.branch0, done ? 1 : 0, u.row0, u.nrows, p.lo, p.hi,
                     done ? 0 : (int32_t)prow, u.masked});
    if (done) continue;
    for (int32_t b = u.row0 / Hq; b * (int64_t)Hq < row1; ++b) {
      const int32_t a = std::max(u.row0, b * Hq);
      const int32_t e = std::min<int64_t>(row1, (int64_t)b * Hq + Hq);
      merge.push_back({u.branch0 + b,
                       {(int32_t)(prow + (a - u.row0)), 0,  // one kv-head: no stride
                        a - b * Hq, e - b * Hq}});
    }
    prow += u.nrows;
    if (prow > INT32_MAX / 2)
      return fail(KV_ERR_INVALID_ARG, "step too large for one plan");
  }
  // Branches with anything to merge.
  std::vector<int32_t> merged;
  {
    std::vector<char> any(nb, 0);
    for (const Tagged& t : merge) any[t.branch] = 1;
    for (int32_t b = 0; b < nb; ++b)
      if (any[b]) merged.push_back(b);
  }
  const int64_t n_csr = (int64_t)merge.size();
  const int64_t off_item = kPlanHeaderInts;
  const int64_t off_pair = off_item + 8 * (int64_t)items.size();
  const int64_t off_merge = off_pair + n_pairs + 1 + n_lists + 1;
  const int64_t off_ptr = off_merge + (int64_t)merged.size();
  const int64_t off_ent = off_ptr + nb + 1;
  const int64_t total = off_ent + 4 * n_csr;
  if (total > INT32_MAX) return fail(KV_ERR_INVALID_ARG, "plan too large");
  std::memset(info, 0, sizeof *info);
  info->plan_ints = total;
  info->workspace_bytes = (int64_t)ws_total(prow, KV_LATENT_RANK);
  info->partial_rows = prow;
  info->n_tile_items = (int32_t)items.size();
  info->n_tile_wide_items = n_pairs;
  info->n_row_items = n_few;
  info->n_row_warp_items = n_lists;
  info->n_merge_rows = (int32_t)merged.size();
  info->chunk_blocks =
      (int32_t)std::min<int64_t>(INT32_MAX, chunk / kTileCost * kTileBlocks);
  info->flags = flags;
  info->latent_rows = nb * Hq;
  if (!plan) return KV_OK;
  if (plan_cap < total)
    return fail(KV_ERR_INVALID_ARG, "plan_cap %lld < %lld", (long long)plan_cap,
                (long long)total);
  int32_t* h = plan;
  std::fill(h, h + kPlanHeaderInts, 0);
  h[H_MAGIC] = kLatentPlanMagic;
  h[H_NB] = nb;
  h[H_HQ] = Hq;
  h[H_HKV] = 1;
  h[H_D] = KV_LATENT_RANK;
  h[H_N_TILE_ITEMS] = (int32_t)items.size();
  h[H_N_CSR] = (int32_t)n_csr;
  h[H_OFF_TILE_ITEMS] = (int32_t)off_item;
  h[H_OFF_CSR_PTR] = (int32_t)off_ptr;
  h[H_OFF_CSR_ENT] = (int32_t)off_ent;
  h[H_PARTIAL_ROWS] = (int32_t)prow;
  h[H_CHUNK] = info->chunk_blocks;
  h[H_FLAGS] = flags;
  h[H_TOTAL] = (int32_t)total;
  std::memcpy(h + off_item, items.data(), items.size() * sizeof(WorkItem));
  std::copy(ptr[1].begin(), ptr[1].end(),
            std::copy(ptr[0].begin(), ptr[0].end(), h + off_pair));
  std::copy(merged.begin(), merged.end(), h + off_merge);
  int32_t* cp = h + off_ptr;
  int32_t* ent = h + off_ent;
  std::fill(cp, cp + nb + 1, 0);
  for (const Tagged& t : merge) ++cp[t.branch + 1];
  for (int32_t b = 0; b < nb; ++b) cp[b + 1] += cp[b];
  std::vector<int32_t> at(cp, cp + nb);
  for (const Tagged& t : merge)
    std::memcpy(ent + 4 * (int64_t)at[t.branch]++, &t.e, sizeof(MergeEntry));
  return KV_OK;
}

}  // namespace pkv
