// Host half of a latent prefill (paged_latent_prefill_plan): which physical
// blocks the step's branches hold, each expanded once however many branches
// share it, and the tiles of query rows.
//
// Plan (int32): header, the distinct blocks in order of first use with their
// count of valid tokens, the branches' tables as indices into them, and one
// descriptor per tile of up to 256 query rows, longest key ranges first.

#include <algorithm>
#include <cstring>
#include <new>

#include "internal.h"

using pkv::fail;

namespace {

kv_status prefill_plan(int32_t nb, int32_t Hq, int64_t num_blocks,
                       int32_t max_blocks, const int32_t* tables,
                       const int32_t* seq_lens, const int32_t* q_lens,
                       int32_t* plan, int64_t plan_cap,
                       kv_decode_plan_info* info) {
  if (!info || !tables || !seq_lens || !q_lens)
    return fail(KV_ERR_INVALID_ARG, "null argument");
  if (nb < 1 || Hq < 1 || Hq > 65535 || max_blocks < 1)
    return fail(KV_ERR_INVALID_ARG, "bad nb/Hq/max_blocks (%d/%d/%d)", nb, Hq,
                max_blocks);
  if (num_blocks < 1 || num_blocks > (int64_t)INT32_MAX / 16)
    return fail(KV_ERR_INVALID_ARG, "num_blocks out of range");
  std::vector<int32_t> uniq, valid, slots;
  std::vector<pkv::PrefillTile> tiles;
  std::vector<int32_t> slot_of(num_blocks, -1);
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
    const int32_t nblk = (L + 15) / 16;
    if (off + nblk > INT32_MAX / 2)
      return fail(KV_ERR_INVALID_ARG, "tables too large for one plan");
    for (int32_t k = 0; k < nblk; ++k) {
      const int32_t phys = tables[(int64_t)b * max_blocks + k];
      if (phys < 0 || phys >= num_blocks)
        return fail(KV_ERR_INVALID_ARG, "branch %d: block %d is %d, outside the "
                                        "pool", b, k, phys);
      if (slot_of[phys] < 0) {
        slot_of[phys] = (int32_t)uniq.size();
        uniq.push_back(phys);
        valid.push_back(0);
      }
      const int32_t s = slot_of[phys];
      valid[s] = std::max(valid[s], std::min(16, L - k * 16));
      slots.push_back(s);
    }
    for (int32_t r = 0; r < n; r += pkv::kPrefillRows)
      tiles.push_back({(int32_t)(row + r), std::min(pkv::kPrefillRows, n - r),
                       L - n + r, (int32_t)off});
    row += n;
  }
  // Longest first: the persistent pairs take the tiles of a group of heads in this
  // order, so that the last ones to start are short.
  std::stable_sort(tiles.begin(), tiles.end(),
                   [](const pkv::PrefillTile& x, const pkv::PrefillTile& y) {
                     return x.pos0 + x.nrows > y.pos0 + y.nrows;
                   });
  const int64_t U = (int64_t)uniq.size();
  if (U * Hq > INT32_MAX / 2 || (int64_t)tiles.size() * Hq > INT32_MAX / 2)
    return fail(KV_ERR_INVALID_ARG, "step too large for one plan");
  const int64_t off_valid = pkv::kPlanHeaderInts + U;
  const int64_t off_slots = off_valid + U;
  const int64_t off_tiles = off_slots + (int64_t)slots.size();
  const int64_t total = off_tiles + 4 * (int64_t)tiles.size();
  if (total > INT32_MAX) return fail(KV_ERR_INVALID_ARG, "plan too large");
  std::memset(info, 0, sizeof *info);
  info->plan_ints = total;
  info->partial_rows = (int64_t)slots.size();
  info->workspace_bytes = (int64_t)pkv::prefill_workspace(U, Hq);
  info->n_row_items = (int32_t)U;
  info->n_tile_items = (int32_t)tiles.size();
  info->n_merge_rows = (int32_t)row;
  info->flags = pkv::kPrefillPlan;
  if (!plan) return KV_OK;
  if (plan_cap < total)
    return fail(KV_ERR_INVALID_ARG, "plan_cap %lld < %lld", (long long)plan_cap,
                (long long)total);
  std::fill(plan, plan + pkv::kPlanHeaderInts, 0);
  plan[pkv::H_MAGIC] = pkv::kPrefillPlanMagic;
  plan[pkv::H_NB] = nb;
  plan[pkv::H_HQ] = Hq;
  plan[pkv::H_D] = KV_LATENT_RANK;
  plan[pkv::H_N_ROW_ITEMS] = (int32_t)U;
  plan[pkv::H_N_TILE_ITEMS] = (int32_t)tiles.size();
  plan[pkv::H_TOTAL] = (int32_t)total;
  std::copy(uniq.begin(), uniq.end(), plan + pkv::kPlanHeaderInts);
  std::copy(valid.begin(), valid.end(), plan + off_valid);
  std::copy(slots.begin(), slots.end(), plan + off_slots);
  std::memcpy(plan + off_tiles, tiles.data(), tiles.size() * sizeof(pkv::PrefillTile));
  return KV_OK;
}

}  // namespace

extern "C" kv_status paged_latent_prefill_plan(
    int32_t nb, int32_t Hq, int64_t num_blocks, int32_t max_blocks,
    const int32_t* tables, const int32_t* seq_lens, const int32_t* q_lens,
    int32_t num_sms, int32_t* plan, int64_t plan_cap,
    kv_decode_plan_info* info) {
  pkv::clear_error();
  (void)num_sms;
  try {
    return prefill_plan(nb, Hq, num_blocks, max_blocks, tables, seq_lens, q_lens,
                        plan, plan_cap, info);
  } catch (const std::bad_alloc&) {
    return fail(KV_ERR_OOM, "no host memory for the plan");
  }
}
