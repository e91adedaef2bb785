// Host half of chunk attention (paged_chunk_plan): tiles of query tokens, cut
// along the keys where there are too few of them for the GPU.
//
// A tile is up to 2 floor(128 / G) tokens of one branch with the G query heads
// of a kv-head: floor(128 / G) tokens x G heads on each CTA of a pair, or on a single
// CTA where it has no more.
//
// Plan (int32): header; for e4m3 pools the distinct blocks in order of first use;
// the branches' tables (physical blocks, or indices into the distinct ones); one
// descriptor of 8 per work item of a kv-head (tiles for pairs first, in each kind
// longest key ranges first); one of 4 per tile whose key range is cut.

#include <algorithm>
#include <cstring>
#include <functional>
#include <new>
#include <queue>
#include <utility>

#include "internal.h"

using pkv::fail;

namespace {

constexpr int kKeys = pkv::kChunkKeys;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Tile {
  int32_t row0, ntok, pos0, table;
  int32_t keys() const { return (pos0 + ntok - 1) / kKeys + 1; }  // key tiles
};

// When the persistent CTAs would be done, in pair tiles (a key tile of an item on a
// pair of SMs, 0.58 us), with the items' order the kernels take them in.  Measured:
// a single CTA takes a key tile in 0.55 of that, an item costs either about kItem on
// top (its first loads, the last products, the joining of the rows), a cut kPartial
// more (the partial rows out, and in again), the merge kMerge once.
struct Cost {
  static constexpr double kSingle = 0.55, kItem = 5, kPartial = 1.5, kMerge = 5;
  int32_t Hkv, ctok, pairs;

  // Tiles before `from` (of the sorted list) uncut, the others in pieces of at most
  // `cut`.
  double finish(const std::vector<Tile>& tiles, size_t from, int32_t cut) const {
    // Durations of each kind, with how many items there are of each.
    std::vector<std::pair<double, int64_t>> wide, narrow;
    bool any_cut = false;
    for (size_t i = 0; i < tiles.size(); ++i) {
      const int32_t keys = tiles[i].keys();
      const int64_t pieces = i < from ? 1 : ceil_div(keys, cut);
      any_cut |= pieces > 1;
      const bool w = tiles[i].ntok > ctok;
      const double each = (double)keys / pieces * (w ? 1. : kSingle) + kItem +
                          (pieces > 1 ? kPartial : 0.);
      (w ? wide : narrow).push_back({each, pieces * Hkv});
    }
    auto longer = [](auto& x, auto& y) { return x.first > y.first; };
    std::sort(wide.begin(), wide.end(), longer);
    std::sort(narrow.begin(), narrow.end(), longer);
    // Pairs, then the SMs of each as it is done.
    using Heap = std::priority_queue<double, std::vector<double>, std::greater<double>>;
    Heap on_pairs(std::greater<double>(), std::vector<double>(pairs, 0.));
    double end = 0;
    auto run = [&](Heap& heap, const auto& items) {
      for (const auto& x : items)
        for (int64_t k = 0; k < x.second; ++k) {
          const double t = heap.top() + x.first;
          heap.pop();
          heap.push(t);
          end = std::max(end, t);
        }
    };
    run(on_pairs, wide);
    Heap on_sms;
    for (; !on_pairs.empty(); on_pairs.pop()) {
      on_sms.push(on_pairs.top());
      on_sms.push(on_pairs.top());
    }
    run(on_sms, narrow);
    return end + (any_cut ? kMerge : 0.);
  }
};

// Where the keys of tiles (sorted, most keys first) are cut: from which tile on, and
// into pieces of how many key tiles at most.  Uncut, all in pieces, or only those that
// come after the last whole round of the pairs, whichever is done first.  Steps of
// more than eight rounds of items even out by themselves.
void pick_cut(const std::vector<Tile>& tiles, int32_t Hkv, int32_t ctok, int32_t pairs,
              size_t* from, int32_t* cut) {
  *from = tiles.size();
  *cut = 1;
  if (tiles.empty() || (int64_t)tiles.size() * Hkv > 8ll * pairs) return;
  const Cost cost{Hkv, ctok, pairs};
  const int32_t longest = tiles.front().keys();
  double least = cost.finish(tiles, tiles.size(), 1) * 0.97;  // cuts have to pay
  auto attempt = [&](size_t f, int32_t c) {
    const double t = cost.finish(tiles, f, c);
    if (t < least) {
      least = t;
      *from = f;
      *cut = c;
    }
  };
  const size_t round = std::max<int64_t>(pairs / Hkv, 1);
  const size_t rest = tiles.size() / round * round;  // tiles of whole rounds
  for (int32_t c = longest * 3 / 4; c >= 2; c = c * 3 / 4) {
    attempt(0, c);
    if (rest > 0 && rest < tiles.size()) attempt(rest, c);
    if (rest > round) attempt(rest - round, c);
  }
}

kv_status chunk_plan(int32_t nb, int32_t Hq, int32_t Hkv, int32_t d,
                     int64_t num_blocks, int32_t max_blocks, const int32_t* tables,
                     const int32_t* seq_lens, const int32_t* q_lens,
                     int32_t num_sms, int32_t flags, int32_t* plan,
                     int64_t plan_cap, kv_decode_plan_info* info) {
  if (!info || !tables || !seq_lens || !q_lens)
    return fail(KV_ERR_INVALID_ARG, "null argument");
  if (kv_status s = pkv::chunk_heads_ok(Hq, Hkv, d)) return s;
  if (nb < 1 || max_blocks < 1)
    return fail(KV_ERR_INVALID_ARG, "bad nb/max_blocks (%d/%d)", nb, max_blocks);
  if (num_blocks < 1 || num_blocks > (int64_t)INT32_MAX / 16 / Hkv)
    return fail(KV_ERR_INVALID_ARG, "num_blocks out of range");
  if (flags & ~KV_PLAN_KV_E4M3)
    return fail(KV_ERR_INVALID_ARG, "unknown plan flags 0x%x", flags);
  const bool e4m3 = flags & KV_PLAN_KV_E4M3;
  if (num_sms <= 0) num_sms = 152;
  const int32_t pairs = std::clamp(num_sms / 2, 1, 4096);
  const int32_t G = Hq / Hkv, step = 2 * (pkv::kChunkRows / G);

  std::vector<int32_t> uniq, slots;
  std::vector<Tile> whole;
  std::vector<int32_t> slot_of(e4m3 ? num_blocks : 0, -1);
  int64_t row = 0;
  for (int32_t b = 0; b < nb; ++b) {
    const int32_t L = seq_lens[b], n = q_lens[b];
    if (n < 0 || L < n || (int64_t)L > (int64_t)max_blocks * 16)
      return fail(KV_ERR_INVALID_ARG, "branch %d: q_lens %d, seq_lens %d, at most "
                                      "%lld tokens", b, n, L,
                  (long long)max_blocks * 16);
    if (n == 0) continue;
    if (row + n > INT32_MAX / 2)
      return fail(KV_ERR_INVALID_ARG, "too many query rows");
    const int64_t off = (int64_t)slots.size();
    const int32_t nblk = (int32_t)(((int64_t)L + 15) / 16);
    if (off + nblk > INT32_MAX / 4)
      return fail(KV_ERR_INVALID_ARG, "tables too large for one plan");
    for (int32_t k = 0; k < nblk; ++k) {
      const int32_t phys = tables[(int64_t)b * max_blocks + k];
      if (phys < 0 || phys >= num_blocks)
        return fail(KV_ERR_INVALID_ARG, "branch %d: block %d is %d, outside the "
                                        "pool", b, k, phys);
      if (e4m3 && slot_of[phys] < 0) {
        slot_of[phys] = (int32_t)uniq.size();
        uniq.push_back(phys);
      }
      slots.push_back(e4m3 ? slot_of[phys] : phys);
    }
    for (int32_t r = 0; r < n; r += step)
      whole.push_back({(int32_t)(row + r), std::min(step, n - r), L - n + r,
                       (int32_t)off});
    row += n;
  }
  std::stable_sort(whole.begin(), whole.end(),
                   [](const Tile& x, const Tile& y) { return x.keys() > y.keys(); });
  size_t cut_from;
  int32_t cut, most = 0;
  pick_cut(whole, Hkv, step / 2, pairs, &cut_from, &cut);
  std::vector<pkv::ChunkItem> items;
  std::vector<pkv::ChunkMerge> merges;
  int64_t partial = 0;
  for (size_t k = 0; k < whole.size(); ++k) {
    const Tile& t = whole[k];
    const int32_t keys = t.keys();
    const int32_t pieces = k < cut_from ? 1 : (int32_t)ceil_div(keys, cut);
    most = std::max(most, (keys - 1) / pieces + 1);
    const int64_t rows = (int64_t)t.ntok * Hq;  // of a piece
    if (pieces > 1)
      merges.push_back({t.row0, t.ntok, (int32_t)partial, pieces});
    for (int32_t i = 0; i < pieces; ++i) {
      items.push_back({t.row0, t.ntok, t.pos0, t.table,
                       (int32_t)((int64_t)keys * i / pieces),
                       (int32_t)((int64_t)keys * (i + 1) / pieces),
                       pieces > 1 ? (int32_t)partial : -1, 0});
      if (pieces > 1) partial += rows;
      if (partial > INT32_MAX / 4)
        return fail(KV_ERR_INVALID_ARG, "step too large for one plan");
    }
  }
  // Tiles for pairs, then those of no more than a CTA's tokens; longest first: the
  // persistent CTAs take the items in this order, so that the last ones to start are
  // short.
  const int32_t ctok = step / 2;
  std::stable_sort(items.begin(), items.end(),
                   [ctok](const pkv::ChunkItem& x, const pkv::ChunkItem& y) {
                     const bool wx = x.ntok > ctok, wy = y.ntok > ctok;
                     if (wx != wy) return wx;
                     return x.key_end - x.key_begin > y.key_end - y.key_begin;
                   });
  const auto n_wide = std::count_if(
      items.begin(), items.end(),
      [ctok](const pkv::ChunkItem& x) { return x.ntok > ctok; });
  const int64_t U = (int64_t)uniq.size();
  if ((int64_t)items.size() * Hkv > INT32_MAX / 2 || U * Hkv > INT32_MAX / 16)
    return fail(KV_ERR_INVALID_ARG, "step too large for one plan");
  const int64_t off_slots = pkv::kPlanHeaderInts + U;
  const int64_t off_items = off_slots + (int64_t)slots.size();
  const int64_t off_merges = off_items + 8 * (int64_t)items.size();
  const int64_t total = off_merges + 4 * (int64_t)merges.size();
  if (total > INT32_MAX) return fail(KV_ERR_INVALID_ARG, "plan too large");
  std::memset(info, 0, sizeof *info);
  info->plan_ints = total;
  info->partial_rows = partial;
  info->workspace_bytes = (int64_t)pkv::chunk_workspace(partial, U, Hkv, d);
  info->n_row_items = (int32_t)U;
  info->n_tile_items = (int32_t)items.size();
  info->n_merge_rows = (int32_t)row;
  info->chunk_blocks = most * (kKeys / 16);
  info->n_tile_wide_items = (int32_t)n_wide;
  info->n_row_warp_items = (int32_t)merges.size();
  info->flags = pkv::kChunkPlan | flags;
  info->latent_rows = pkv::chunk_mark(Hq, Hkv, d);
  if (!plan) return KV_OK;
  if (plan_cap < total)
    return fail(KV_ERR_INVALID_ARG, "plan_cap %lld < %lld", (long long)plan_cap,
                (long long)total);
  std::fill(plan, plan + pkv::kPlanHeaderInts, 0);
  plan[pkv::H_MAGIC] = pkv::kChunkPlanMagic;
  plan[pkv::H_NB] = nb;
  plan[pkv::H_HQ] = Hq;
  plan[pkv::H_HKV] = Hkv;
  plan[pkv::H_D] = d;
  plan[pkv::H_N_ROW_ITEMS] = (int32_t)U;
  plan[pkv::H_N_TILE_ITEMS] = (int32_t)items.size();
  plan[pkv::H_OFF_TILE_ITEMS] = (int32_t)off_items;
  plan[pkv::H_PARTIAL_ROWS] = (int32_t)partial;
  plan[pkv::H_CHUNK] = info->chunk_blocks;
  plan[pkv::H_FLAGS] = info->flags;
  plan[pkv::H_TOTAL] = (int32_t)total;
  std::copy(uniq.begin(), uniq.end(), plan + pkv::kPlanHeaderInts);
  std::copy(slots.begin(), slots.end(), plan + off_slots);
  if (!items.empty())
    std::memcpy(plan + off_items, items.data(), items.size() * sizeof items[0]);
  if (!merges.empty())
    std::memcpy(plan + off_merges, merges.data(), merges.size() * sizeof merges[0]);
  return KV_OK;
}

}  // namespace

namespace pkv {

kv_status chunk_heads_ok(int32_t Hq, int32_t Hkv, int32_t d) {
  if (Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Hq > 32767 || Hkv > 2047)
    return fail(KV_ERR_INVALID_ARG, "bad Hq/Hkv (%d/%d)", Hq, Hkv);
  if (Hq / Hkv > kChunkRows)
    return fail(KV_ERR_INVALID_ARG, "more than %d query heads a kv-head", kChunkRows);
  if (d != 64 && d != 128) return fail(KV_ERR_INVALID_ARG, "head_dim must be 64 or 128");
  return KV_OK;
}

}  // namespace pkv

extern "C" kv_status paged_chunk_plan(
    int32_t nb, int32_t Hq, int32_t Hkv, int32_t head_dim, int64_t num_blocks,
    int32_t max_blocks, const int32_t* tables, const int32_t* seq_lens,
    const int32_t* q_lens, int32_t num_sms, int32_t flags, int32_t* plan,
    int64_t plan_cap, kv_decode_plan_info* info) {
  pkv::clear_error();
  try {
    return chunk_plan(nb, Hq, Hkv, head_dim, num_blocks, max_blocks, tables,
                      seq_lens, q_lens, num_sms, flags, plan, plan_cap, info);
  } catch (const std::bad_alloc&) {
    return fail(KV_ERR_OOM, "no host memory for the plan");
  }
}
