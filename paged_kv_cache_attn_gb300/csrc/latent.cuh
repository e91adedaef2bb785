// What the two latent decode kernels share: a step's arguments and the walk over
// a pair's work items.
#pragma once

#include "cluster.cuh"

namespace pkv {
namespace lat {

constexpr int kRank = KV_LATENT_RANK;
constexpr int kFewRows = kLatentFewRows;

struct Params {
  const int32_t* tables;
  const int32_t* seq_lens;
  const WorkItem* items;
  const int32_t* pair_ptr;
  const int32_t* few_ptr;  // lists of items of few rows
  float2* ml;
  float* o;
  __nv_bfloat16* out;
  DeviceStatus* status;
  int nb, Hq, max_blocks, n_items, n_pairs, n_few_lists;
  int64_t num_blocks, partial_rows;
  float scale_log2;
  bool trigger;  // the kernel for few rows follows and may start beside this one
};

__device__ __forceinline__ bool item_fits(const WorkItem& it, const Params& p) {
  const int64_t last = (int64_t)it.row0 + it.nrows - 1;
  return it.nrows >= 1 && it.nrows <= 128 && it.row0 >= 0 && it.branch0 >= 0 &&
         it.branch0 + last / p.Hq < p.nb && it.blk_begin >= 0 &&
         it.blk_begin < it.blk_end && it.blk_end <= p.max_blocks &&
         (it.g != 0 || (it.prow_base >= 0 &&
                        (int64_t)it.prow_base + it.nrows <= p.partial_rows));
}

// The items of this pair, the same for every role of both CTAs, read one
// ahead.  Malformed ones are skipped by all (and recorded by one warp, see
// report_bad).
// (A list is a pair's, or an SM's of items of at most kFewRows rows.)
template <bool kFew>
struct ItemLoop {
  const Params& p;
  int i, end;
  WorkItem ahead;
  __device__ ItemLoop(const Params& pp, int list) : p(pp) {
    const int32_t* ptr = kFew ? p.few_ptr : p.pair_ptr;
    i = ptr[list];
    end = ptr[list + 1];
    if (i < 0 || end > p.n_items || i > end) i = end = 0;
    if (i < end) ahead = p.items[i];
  }
  __device__ bool next(WorkItem& it) {
    while (i < end) {
      it = ahead;
      if (++i < end) ahead = p.items[i];
      if (item_fits(it, p) && (!kFew || it.nrows <= kFewRows)) return true;
    }
    return false;
  }
};

template <bool kFew>
__device__ __forceinline__ void report_bad(const Params& p, int pair) {
  const int32_t* ptr = kFew ? p.few_ptr : p.pair_ptr;
  const int a = ptr[pair], b = ptr[pair + 1];
  if (a < 0 || b > p.n_items || a > b) {
    record_status(p.status, KV_ERR_DEVICE, -1 - pair);
    return;
  }
  for (int i = a; i < b; ++i)
    if (!item_fits(p.items[i], p) || (kFew && p.items[i].nrows > kFewRows))
      record_status(p.status, KV_ERR_DEVICE, -1 - i);
}

// The physical block of `blk` of the item, or -1 (past the range, or not a
// block of the pool).
__device__ __forceinline__ int block_of(const Params& p, const WorkItem& it,
                                        int blk, bool& bad) {
  bad = false;
  if (blk >= it.blk_end) return -1;
  const int phys = p.tables[(int64_t)it.branch0 * p.max_blocks + blk];
  if (phys >= 0 && (int64_t)phys < p.num_blocks) return phys;
  bad = true;
  return -1;
}


}  // namespace lat

// The kernel for items of at most kLatentFewRows rows (decode_latent_few.cu).
// beside: it was preceded by the pairs' kernel, which let it start early.
cudaError_t launch_latent_few(const CUtensorMap& tmC, const CUtensorMap& tmR,
                              const CUtensorMap& tmQ, const lat::Params& p,
                              bool beside, cudaStream_t st);

}  // namespace pkv
