// Decode attention over a latent pool, absorbed form (paged_latent_decode_attn).
//
// For every query row (a branch and a head), with c_t the latent (512) and r_t
// the position key (64) of token t:
//   s_t = q . [c_t ; r_t],  out = sum_t softmax_t(scale s_t) c_t.
// All heads share the tokens, so 128 rows (the heads of a branch, or the
// branches x heads of a shared segment) are one tile: 2 x 1088 flops a row and
// token against 1152 bytes a token, 242 flops a byte at 128 rows -- dense
// enough for the tensor cores to be the bound of shared segments and of 128
// heads, with HBM the bound of fewer rows.
//
// Neither operand set fits one SM: O is 128 x 512 fp32, the whole tensor
// memory, which leaves no room for scores, and Q is another 147 KB.  So two
// SMs share an item as producer and consumer, a cluster of two CTAs:
//
//   score CTA (rank 0):  S = Q K^T.  TMEM: Q's latent part as the A operand
//     (256 columns, bf16 pairs) and two S buffers (2 x 128 fp32 columns); the
//     position part of Q in shared memory.  K streams through a ring of
//     128-token x 128-dimension stages.  256 softmax threads (two per row, 64
//     columns each, maxima exchanged through shared memory) turn S into P
//     (bf16, base 2, lazy maximum) in two staging tiles of 64 tokens, which
//     bulk copies carry into the other CTA's shared memory.
//   output CTA (rank 1): O += P V, TMEM: O (512 columns).  V streams through a
//     ring of 16-token blocks (512 dimensions); P arrives in a ring of four
//     64-token tiles.  256 threads rescale O when a maximum has moved, and
//     write the result.
//
// No product is computed twice, and the tensor work is nearly even: per 128
// tokens 36 MMAs of N = 128 (65 cycles each, measured) against 16 of N = 256
// (128 cycles).  P flows one way, so the latency between the SMs is hidden by
// the rings.  The pairs are persistent: each works through its list of items
// (plan_latent.cpp), and loads run ahead across items.
//
// Measured alternatives of the tile shape (cycles per MMA with K = 16): N = 64
// 56, N = 128 65 (A in TMEM) or 69 (A in shared memory), N = 256 128.
//
// Slots past a branch's length may hold anything: their scores are replaced
// by -inf before the maximum, and their rows of V are zeroed in shared memory
// (0 x NaN would not be 0).  Blocks past an item's range are not loaded.
//
// Every wait is bounded; a wait that ran out is recorded, ends the loop of its
// role, and the other roles run into their own bounds.  Before the CTAs leave,
// copies in flight have landed and tensor memory is freed.

#include <cmath>
#include <cstring>

#include "cluster.cuh"
#include "tensor_map.h"

namespace pkv {
namespace lat {

using tc::bar_and;
using tc::bar_or;
using tc::cluster_rank;
using tc::cluster_sync;
using tc::copy_to_cta;
using tc::fence_after_sync;
using tc::fence_before_sync;
using tc::idesc;
using tc::map_rank;
using tc::mbar_wait_cluster;
using tc::remote_arrive;
using tc::sdesc;
using tc::tma_load_5d_at;
using tc::tmem_ld32;
using tc::tmem_st32;
using tc::tmem_wait_ld;
using tc::tmem_wait_st;
using tc::umma_commit;
using tc::umma_commit_to;
using tc::umma_ss;
using tc::umma_ts;

constexpr int kRank = KV_LATENT_RANK;
constexpr int kRope = KV_LATENT_ROPE;
constexpr int kQDim = kRank + kRope;
constexpr int kT = 128;            // tokens of a score tile
constexpr int kTB = kT / 16;       // its blocks
constexpr int kG = 64;             // tokens of a P tile
constexpr int kGB = kG / 16;

// Score CTA's shared memory.
constexpr int kQr = 128 * 128;               // position part of Q
constexpr int kKStage = kT * 256;            // 128 tokens x 128 dimensions
constexpr int kNK = 4;
constexpr int kRStage = kT * 128;            // position keys of a tile
constexpr int kNR = 2;
constexpr int kP = 128 * 128;                // 128 rows x 64 tokens of P
// What goes with a P tile: 128 rescale factors and a flag word.
constexpr int kHdr = 528, kHdrStride = 640;
constexpr int kOffK = kQr;
constexpr int kOffR = kOffK + kNK * kKStage;
constexpr int kOffStage = kOffR + kNR * kRStage;
constexpr int kOffStageHdr = kOffStage + 2 * kP;
constexpr int kOffStageFin = kOffStageHdr + 2 * kHdrStride;
constexpr int kScoreSmem = kOffStageFin + 2 * 512;
// Output CTA's shared memory.
constexpr int kVBlk = 16 * kRank * 2;        // one block
constexpr int kNV = 9;
constexpr int kNP = 4;
constexpr int kOffP = kNV * kVBlk;
constexpr int kOffHdr = kOffP + kNP * kP;
constexpr int kOffFin = kOffHdr + kNP * kHdrStride;
constexpr int kOutSmem = kOffFin + 2 * 512;
constexpr int kSmem =
    (kScoreSmem > kOutSmem ? kScoreSmem : kOutSmem) + 1024;

constexpr int kThreads = 12 * 32;
constexpr int kRowThreads = 256;             // warps 0-7
constexpr int kMmaWarp = 8;                  // warps 9-11 load (11: see below)
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 256;              // score CTA: Q 0..255, S 256..511
constexpr float kRescale = 8.f;              // lazy-max threshold (log2 units)

struct Params {
  const __nv_bfloat16* q;
  const int32_t* tables;
  const int32_t* seq_lens;
  const WorkItem* items;
  const int32_t* pair_ptr;
  float2* ml;
  float* o;
  __nv_bfloat16* out;
  DeviceStatus* status;
  int nb, Hq, max_blocks, n_items, n_pairs;
  int64_t num_blocks, partial_rows;
  float scale_log2;
};

// At the same place in both CTAs.
struct Bars {
  // score CTA
  uint64_t k_full[kNK], k_empty[kNK], r_full[kNR], r_empty[kNR];
  uint64_t q_full, s_full[2], s_empty[2];
  uint64_t p_ack[2];       // a staged P tile has landed on the other side
  uint64_t p_empty[kNP];   // the other side has consumed P slot i
  uint64_t fin_empty[2];
  // output CTA
  uint64_t v_full[kNV], v_empty[kNV], v_fix[kNV], p_full[kNP], fin_full[2];
  uint64_t event, o_ok;
  uint64_t drain;
};

__device__ __forceinline__ bool item_fits(const WorkItem& it, const Params& p) {
  const int64_t last = (int64_t)it.row0 + it.nrows - 1;
  return it.nrows >= 1 && it.nrows <= 128 && it.row0 >= 0 && it.branch0 >= 0 &&
         it.branch0 + last / p.Hq < p.nb && it.blk_begin >= 0 &&
         it.blk_begin < it.blk_end && it.blk_end <= p.max_blocks &&
         (it.g != 0 || (it.prow_base >= 0 &&
                        (int64_t)it.prow_base + it.nrows <= p.partial_rows));
}

// The items of this pair, the same for every role of both CTAs.  A malformed
// item or list is recorded by one thread and skipped by all.
struct ItemLoop {
  const Params& p;
  int i, end;
  __device__ ItemLoop(const Params& pp, int pair) : p(pp) {
    i = p.pair_ptr[pair];
    end = p.pair_ptr[pair + 1];
    if (i < 0 || end > p.n_items || i > end) i = end = 0;
  }
  __device__ bool next(WorkItem& it) {
    while (i < end) {
      it = p.items[i++];
      if (item_fits(it, p)) return true;
    }
    return false;
  }
};

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

__device__ __forceinline__ int n_tiles(const WorkItem& it) {
  return (it.blk_end - it.blk_begin + kTB - 1) / kTB;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    latent_decode_kernel(const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV,
                         const __grid_constant__ CUtensorMap tmR,
                         const Params p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) Bars bars;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  __shared__ int event_sh;                // slot of a rescale, or -1: item done
  __shared__ float max_sh[2][2][128];     // [tile parity][half][row]
  __shared__ float sum_sh[128];

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool scores = rank == 0;
  const int pair = blockIdx.x >> 1;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* base_ptr = smem_raw + (base - smem_u32(smem_raw));
  volatile int* aborted = &abort_sh;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kNK; ++s) {
      mbar_init(smem_u32(&bars.k_full[s]), 2);   // two producer warps
      mbar_init(smem_u32(&bars.k_empty[s]), 1);
    }
    for (int s = 0; s < kNR; ++s) {
      mbar_init(smem_u32(&bars.r_full[s]), 1);
      mbar_init(smem_u32(&bars.r_empty[s]), 1);
    }
    mbar_init(smem_u32(&bars.q_full), 8);        // the row warps
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&bars.s_full[b]), 1);
      mbar_init(smem_u32(&bars.s_empty[b]), 8);
      mbar_init(smem_u32(&bars.p_ack[b]), 1);
      mbar_init(smem_u32(&bars.fin_empty[b]), 8);  // the other side's row warps
      mbar_init(smem_u32(&bars.fin_full[b]), 1);
    }
    for (int s = 0; s < kNP; ++s) {
      mbar_init(smem_u32(&bars.p_empty[s]), 1);
      mbar_init(smem_u32(&bars.p_full[s]), 1);
    }
    for (int s = 0; s < kNV; ++s) {
      mbar_init(smem_u32(&bars.v_full[s]), 1);
      mbar_init(smem_u32(&bars.v_empty[s]), 1);
      mbar_init(smem_u32(&bars.v_fix[s]), 1);    // masked rows zeroed
    }
    mbar_init(smem_u32(&bars.event), 2);         // the MMA thread and its commit
    mbar_init(smem_u32(&bars.o_ok), 8);
    mbar_init(smem_u32(&bars.drain), 1);
    abort_sh = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    tma_prefetch_desc(&tmR);
    if (rank == 0) {
      // Malformed entries of this pair's list.
      const int a = p.pair_ptr[pair], b = p.pair_ptr[pair + 1];
      if (a < 0 || b > p.n_items || a > b) {
        record_status(p.status, KV_ERR_DEVICE, -1 - pair);
      } else {
        for (int i = a; i < b; ++i)
          if (!item_fits(p.items[i], p))
            record_status(p.status, KV_ERR_DEVICE, -1 - i);
      }
    }
  }
  if (warp == kMmaWarp) {
    asm volatile(
        "tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::
            "r"(smem_u32(&tmem_base_sh)),
        "r"(kTmemCols)
        : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::
                     : "memory");
  }
  fence_before_sync();
  __syncthreads();
  cluster_sync();  // the other CTA's barriers are ready too
  fence_after_sync();
  const uint32_t tmem = tmem_base_sh;
  ItemLoop loop(p, pair);
  WorkItem it;
  auto timed_out = [&](int site) {
    if (!*aborted) record_status(p.status, KV_ERR_TIMEOUT, site);
    atomicExch(&abort_sh, 1);
  };

  if (scores && warp < 8) {
    // ---- score CTA, rows: thread = (row r, half of a tile's columns) --------
    const int wg = warp >> 2;
    const int r = threadIdx.x & 127;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t stage = base + kOffStage + wg * kP;
    const uint32_t prow = stage + (r >> 3) * 1024 + (r & 7) * 128;
    float* hdr = reinterpret_cast<float*>(base_ptr + kOffStageHdr + wg * kHdrStride);
    const uint32_t peer_p = map_rank(base + kOffP, 1);
    const uint32_t peer_hdr = map_rank(base + kOffHdr, 1);
    const uint32_t peer_fin = map_rank(base + kOffFin, 1);
    uint32_t tc_n = 0;   // tiles so far
    uint32_t g_n = 0;    // P tiles sent so far, by both halves
    uint32_t mine = 0;   // ... by this half
    uint32_t fin_n = 0;  // items whose sums were sent
    bool ok = true;
    while (ok && loop.next(it)) {
      // Q of this row: latent part to TMEM (half of the columns each), the
      // position part to shared memory.  The previous item's products are
      // done (its last S has been read).
      {
        const uint4* src = r < it.nrows
            ? reinterpret_cast<const uint4*>(
                  p.q + ((int64_t)it.branch0 * p.Hq + it.row0 + r) * kQDim)
            : nullptr;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          uint32_t v[32];
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const uint4 x = src ? __ldg(src + wg * 32 + h * 8 + c)
                                : make_uint4(0, 0, 0, 0);
            v[4 * c] = x.x;
            v[4 * c + 1] = x.y;
            v[4 * c + 2] = x.z;
            v[4 * c + 3] = x.w;
          }
          tmem_st32(lane_base + wg * 128 + h * 32, v);
        }
        if (wg == 0) {
          const uint32_t qrow = base + (r >> 3) * 1024 + (r & 7) * 128;
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const uint4 x = src ? __ldg(src + 64 + c) : make_uint4(0, 0, 0, 0);
            tc::st_shared_v4(qrow + ((c ^ (r & 7)) << 4), x.x, x.y, x.z, x.w);
          }
          fence_proxy_async_smem();
        }
        tmem_wait_st();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars.q_full));
      }
      const int seq_len = it.masked ? p.seq_lens[it.branch0] : 0x7fffffff;
      const int nt = n_tiles(it);
      float m_used = -INFINITY, l = 0.f;
      for (int j = 0; j < nt; ++j, ++tc_n) {
        const int b = tc_n & 1;
        const int blk0 = it.blk_begin + j * kTB;
        const int left = (it.blk_end - blk0) * 16;  // tokens of the range
        int valid = min(min(kT, left), max(seq_len - blk0 * 16, 0)) - wg * kG;
        valid = min(valid, kG);
        float s[kG];
        bool w = mbar_wait(smem_u32(&bars.s_full[b]), (tc_n >> 1) & 1);
        w = __all_sync(0xffffffffu, w);
        float mx = -INFINITY;
        if (w) {
          fence_after_sync();
          uint32_t u[32];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            tmem_ld32(lane_base + kColS + b * kT + wg * kG + h * 32, u);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) s[h * 32 + i] = __uint_as_float(u[i]);
          }
          fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bars.s_empty[b]));
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          if (valid == kG) {
#pragma unroll
            for (int i = 0; i < kG; ++i) m4[i & 3] = fmaxf(m4[i & 3], s[i]);
          } else {
#pragma unroll
            for (int i = 0; i < kG; ++i) {
              s[i] = i < valid ? s[i] : -INFINITY;
              m4[i & 3] = fmaxf(m4[i & 3], s[i]);
            }
          }
          mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        } else {
          timed_out(30);
        }
        max_sh[b][wg][r] = mx;
        // Every row thread agrees whether to go on.
        ok = bar_and(1, kRowThreads, w && !*aborted);
        if (!ok) break;
        const float m_tile = fmaxf(mx, max_sh[b][wg ^ 1][r]) * p.scale_log2;
        const bool need = m_tile > m_used + kRescale;
        const float m_new = need ? m_tile : m_used;
        const float alpha = need ? ex2(m_used - m_new) : 1.f;
        m_used = m_new;
        l *= alpha;
        const bool two = left > kG;  // the tile has a second P tile
        if (wg == 0 || two) {
          const uint32_t g = g_n + wg;
          if (mine > 0 &&
              !mbar_wait_cluster(smem_u32(&bars.p_ack[wg]), (mine - 1) & 1))
            timed_out(31);
          const float neg_m = m_new == -INFINITY ? 0.f : -m_new;
          float sum4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            uint32_t pk[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float p0 = ex2(fmaf(s[c * 8 + 2 * i], p.scale_log2, neg_m));
              const float p1 =
                  ex2(fmaf(s[c * 8 + 2 * i + 1], p.scale_log2, neg_m));
              sum4[i] += p0 + p1;
              pk[i] = pack_bf16(p0, p1);
            }
            tc::st_shared_v4(prow + ((c ^ (r & 7)) << 4), pk[0], pk[1], pk[2],
                             pk[3]);
          }
          l += (sum4[0] + sum4[1]) + (sum4[2] + sum4[3]);
          hdr[r] = alpha;
          fence_proxy_async_smem();
          const bool moved = bar_or(2 + wg, 128, need && j > 0);
          if (r == 0) {
            // Only the tile's first P tile carries the factors: O is rescaled
            // once, before any of the tile's products.
            reinterpret_cast<uint32_t*>(hdr)[128] = moved && wg == 0 ? 1u : 0u;
            fence_proxy_async_smem();
            const uint32_t slot = g % kNP;
            if (g >= kNP &&
                !mbar_wait_cluster(smem_u32(&bars.p_empty[slot]),
                                   (g / kNP - 1) & 1))
              timed_out(32);
            if (!*aborted) {
              const uint32_t bar = map_rank(smem_u32(&bars.p_full[slot]), 1);
              copy_to_cta(peer_p + slot * kP, stage, kP, bar);
              copy_to_cta(peer_hdr + slot * kHdrStride, smem_u32(hdr), kHdr, bar);
            }
          }
          ++mine;
        }
        g_n += two ? 2 : 1;
      }
      if (!ok) break;
      // The row's sum over both halves.
      if (wg == 1) sum_sh[r] = l;
      ok = bar_and(1, kRowThreads, !*aborted);
      if (!ok) break;
      if (wg == 0) {
        l += sum_sh[r];
        if (it.g == 0) {
          if (r < it.nrows) p.ml[it.prow_base + r] = make_float2(m_used, l);
        } else {
          const int f = fin_n & 1;
          if (fin_n >= 2 &&
              !mbar_wait_cluster(smem_u32(&bars.fin_empty[f]), (fin_n / 2 - 1) & 1))
            timed_out(33);
          reinterpret_cast<float*>(base_ptr + kOffStageFin + f * 512)[r] = 1.f / l;
          fence_proxy_async_smem();
          bar_or(2, 128, false);
          if (r == 0 && !*aborted)
            copy_to_cta(peer_fin + f * 512, base + kOffStageFin + f * 512, 512,
                        map_rank(smem_u32(&bars.fin_full[f]), 1));
        }
      }
      if (it.g != 0) ++fin_n;
      // sum_sh is read before the next item's sums are written: the tiles of
      // that item pass barrier 1 in between.
    }
    // Copies out of this CTA have landed, and every arrival from the other
    // side is in, before this CTA may leave.
    if (r == 0) {
      if (mine > 0) mbar_wait_cluster(smem_u32(&bars.p_ack[wg]), (mine - 1) & 1);
      if (wg == 0) {
        for (uint32_t g = g_n > kNP ? g_n - kNP : 0; g < g_n; ++g)
          if (!mbar_wait_cluster(smem_u32(&bars.p_empty[g % kNP]), (g / kNP) & 1))
            break;
        for (uint32_t f = fin_n > 2 ? fin_n - 2 : 0; f < fin_n; ++f)
          if (!mbar_wait_cluster(smem_u32(&bars.fin_empty[f & 1]), (f / 2) & 1))
            break;
      }
    }
  } else if (scores && warp == kMmaWarp) {
    // ---- score CTA, products -------------------------------------------------
    if (lane == 0) {
      constexpr uint32_t id = idesc(128, kT, false);
      uint32_t tn = 0, kn = 0, in = 0;
      bool ok = true;
      while (ok && loop.next(it)) {
        ok = mbar_wait(smem_u32(&bars.q_full), in & 1);
        ++in;
        const int nt = n_tiles(it);
        for (int j = 0; j < nt && ok; ++j, ++tn) {
          const int b = tn & 1;
          if (tn >= 2) ok = mbar_wait(smem_u32(&bars.s_empty[b]), ((tn >> 1) - 1) & 1);
          const uint32_t d = tmem + kColS + b * kT;
          for (int c = 0; c < 4 && ok; ++c, ++kn) {
            const uint32_t s = kn % kNK;
            ok = mbar_wait(smem_u32(&bars.k_full[s]), (kn / kNK) & 1);
            if (!ok) break;
            fence_after_sync();
            const uint32_t kst = base + kOffK + s * kKStage;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              umma_ts(d, tmem + c * 64 + kk * 8,
                      sdesc(kst + (kk >> 2) * 1024 + (kk & 3) * 32, 16, 2048),
                      id, (c > 0 || kk > 0) ? 1u : 0u);
            umma_commit(smem_u32(&bars.k_empty[s]));
          }
          if (!ok) break;
          const uint32_t s = tn % kNR;
          ok = mbar_wait(smem_u32(&bars.r_full[s]), (tn / kNR) & 1);
          if (!ok) break;
          fence_after_sync();
          const uint32_t rst = base + kOffR + s * kRStage;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_ss(d, sdesc(base + kk * 32, 16, 1024),
                    sdesc(rst + kk * 32, 16, 1024), id, 1u);
          umma_commit(smem_u32(&bars.r_empty[s]));
          umma_commit(smem_u32(&bars.s_full[b]));
        }
        ok = ok && !*aborted;
      }
      if (!ok) timed_out(34);
      umma_commit(smem_u32(&bars.drain));
      mbar_wait(smem_u32(&bars.drain), 0);
    }
  } else if (scores && warp < 11) {
    // ---- score CTA, K: warp 9 the first four blocks of a tile, warp 10 the
    // other four; one box is a block x 128 dimensions.
    const int half = warp - 9;
    uint32_t kn = 0;
    bool ok = true;
    while (ok && loop.next(it)) {
      const int nt = n_tiles(it);
      for (int j = 0; j < nt && ok; ++j) {
        bool bad = false;
        int phys = -1;
        if (lane < kTB / 2)
          phys = block_of(p, it, it.blk_begin + j * kTB + half * (kTB / 2) + lane, bad);
        if (bad) record_status(p.status, KV_ERR_DEVICE,
                               p.tables[(int64_t)it.branch0 * p.max_blocks +
                                        it.blk_begin + j * kTB + half * (kTB / 2) + lane]);
        const int n = __popc(__ballot_sync(0xffffffffu, phys >= 0));
        for (int c = 0; c < 4; ++c, ++kn) {
          const uint32_t s = kn % kNK;
          if (lane == 0) {
            ok = !*aborted && (kn < kNK || mbar_wait(smem_u32(&bars.k_empty[s]),
                                                     (kn / kNK - 1) & 1));
            if (ok) {
              if (n > 0)
                mbar_expect_tx(smem_u32(&bars.k_full[s]), n * 4096);
              else
                mbar_arrive(smem_u32(&bars.k_full[s]));
            }
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
          if (phys >= 0)
            tma_load_5d_at(base + kOffK + s * kKStage +
                               (half * (kTB / 2) + lane) * 4096,
                           &tmK, 2 * c, phys, smem_u32(&bars.k_full[s]));
          __syncwarp();
        }
      }
    }
    if (lane == 0) {
      if (!ok) timed_out(35);
      for (uint32_t k = kn > kNK ? kn - kNK : 0; k < kn; ++k)
        if (!mbar_wait(smem_u32(&bars.k_full[k % kNK]), (k / kNK) & 1)) break;
    }
  } else if (scores) {
    // ---- score CTA, position keys (warp 11) --------------------------------
    uint32_t tn = 0;
    bool ok = true;
    while (ok && loop.next(it)) {
      const int nt = n_tiles(it);
      for (int j = 0; j < nt; ++j, ++tn) {
        bool bad;
        int phys = -1;
        if (lane < kTB) phys = block_of(p, it, it.blk_begin + j * kTB + lane, bad);
        const int n = __popc(__ballot_sync(0xffffffffu, phys >= 0));
        const uint32_t s = tn % kNR;
        if (lane == 0) {
          ok = !*aborted && (tn < kNR || mbar_wait(smem_u32(&bars.r_empty[s]),
                                                   (tn / kNR - 1) & 1));
          if (ok) {
            if (n > 0)
              mbar_expect_tx(smem_u32(&bars.r_full[s]), n * 2048);
            else
              mbar_arrive(smem_u32(&bars.r_full[s]));
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        if (phys >= 0)
          tma_load_2d(base + kOffR + s * kRStage + lane * 2048, &tmR, 0, phys * 16,
                      smem_u32(&bars.r_full[s]));
        __syncwarp();
      }
    }
    if (lane == 0) {
      if (!ok) timed_out(36);
      for (uint32_t k = tn > kNR ? tn - kNR : 0; k < tn; ++k)
        if (!mbar_wait(smem_u32(&bars.r_full[k % kNR]), (k / kNR) & 1)) break;
    }
  } else if (warp < 8) {
    // ---- output CTA, rows: thread = (row r, half of the 512 columns) ---------
    const int wg = warp >> 2;
    const int r = threadIdx.x & 127;
    const uint32_t orow =
        tmem + ((uint32_t)((warp & 3) * 32) << 16) + wg * (kRank / 2);
    uint32_t ev = 0, fin_n = 0;
    bool ok = true;
    if (threadIdx.x == 0) {
      mbar_expect_tx(smem_u32(&bars.fin_full[0]), 512);
      mbar_expect_tx(smem_u32(&bars.fin_full[1]), 512);
    }
    while (ok && loop.next(it)) {
      for (;;) {
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bars.event), ev & 1));
        if (!ok) break;
        ++ev;
        fence_after_sync();
        const int slot = *(volatile int*)&event_sh;
        if (slot < 0) break;
        // A maximum moved: this row of O times its factor.
        const float alpha =
            reinterpret_cast<const float*>(base_ptr + kOffHdr + slot * kHdrStride)[r];
#pragma unroll 1
        for (int c = 0; c < kRank / 2; c += 32) {
          uint32_t v[32];
          tmem_ld32(orow + c, v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i)
            v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
          tmem_st32(orow + c, v);
        }
        tmem_wait_st();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars.o_ok));
      }
      if (!ok) break;
      // The item is done: its rows out.
      const bool direct = it.g != 0;
      float inv = 1.f;
      if (direct) {
        const int f = fin_n & 1;
        ok = __all_sync(0xffffffffu, mbar_wait_cluster(smem_u32(&bars.fin_full[f]),
                                                       (fin_n >> 1) & 1));
        if (!ok) break;
        inv = reinterpret_cast<const float*>(base_ptr + kOffFin + f * 512)[r];
        ++fin_n;
        // The factors are in registers: once every row warp says so, the slot
        // (armed again by the first) may be filled for the item after next.
        __syncwarp();
        if (lane == 0) {
          if (warp == 0) mbar_expect_tx(smem_u32(&bars.fin_full[f]), 512);
          remote_arrive(map_rank(smem_u32(&bars.fin_empty[f]), 0));
        }
      }
      const int64_t row = (int64_t)it.branch0 * p.Hq + it.row0 + r;
#pragma unroll 1
      for (int c = 0; c < kRank / 2; c += 32) {
        uint32_t v[32];
        tmem_ld32(orow + c, v);
        tmem_wait_ld();
        const int col = wg * (kRank / 2) + c;
        if (r >= it.nrows) {
          // A row past the item's: its MMA row is padding.
        } else if (direct) {
          uint4* dst = reinterpret_cast<uint4*>(p.out + row * kRank + col);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              w[k] = pack_bf16(__uint_as_float(v[8 * i + 2 * k]) * inv,
                               __uint_as_float(v[8 * i + 2 * k + 1]) * inv);
            dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else {
          float4* dst = reinterpret_cast<float4*>(
              p.o + (int64_t)(it.prow_base + r) * kRank + col);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            dst[i] = make_float4(__uint_as_float(v[4 * i]),
                                 __uint_as_float(v[4 * i + 1]),
                                 __uint_as_float(v[4 * i + 2]),
                                 __uint_as_float(v[4 * i + 3]));
        }
      }
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars.o_ok));
    }
    if (!ok && lane == 0) timed_out(40);
  } else if (warp == kMmaWarp) {
    // ---- output CTA, products ------------------------------------------------
    if (lane == 0) {
      constexpr uint32_t id = idesc(128, 256, true);
      uint32_t g = 0, vn = 0, ev = 0, fixes = 0;
      bool ok = true;
      auto event = [&](int what) {
        *(volatile int*)&event_sh = what;
        mbar_arrive(smem_u32(&bars.event));
        umma_commit(smem_u32(&bars.event));
        const bool done = mbar_wait(smem_u32(&bars.o_ok), ev & 1);
        ++ev;
        fence_after_sync();
        return done;
      };
      while (ok && loop.next(it)) {
        const int nblk = it.blk_end - it.blk_begin;
        const int tail = it.masked ? p.seq_lens[it.branch0] - (it.blk_end - 1) * 16 : 16;
        for (int k0 = 0; k0 < nblk && ok; k0 += kGB, ++g) {
          const uint32_t slot = g % kNP;
          ok = mbar_wait_cluster(smem_u32(&bars.p_full[slot]), (g / kNP) & 1);
          if (!ok) break;
          if (k0 > 0 && k0 % kTB == 0 &&
              *reinterpret_cast<volatile uint32_t*>(base_ptr + kOffHdr +
                                                    slot * kHdrStride + 512)) {
            ok = event((int)slot);
            if (!ok) break;
          }
          const uint32_t pst = base + kOffP + slot * kP;
          const int nk = min(kGB, nblk - k0);
          for (int k = 0; k < nk && ok; ++k, ++vn) {
            const uint32_t s = vn % kNV;
            ok = mbar_wait(smem_u32(&bars.v_full[s]), (vn / kNV) & 1);
            if (ok && k0 + k == nblk - 1 && tail < 16) {
              ok = mbar_wait(smem_u32(&bars.v_fix[s]), (fixes >> s) & 1);
              fixes ^= 1u << s;  // the stage's next fix has the other parity
            }
            if (!ok) break;
            fence_after_sync();
            const uint32_t vst = base + s * kVBlk;
            const uint64_t a = sdesc(pst + k * 32, 16, 1024);
            const uint32_t acc = (k0 > 0 || k > 0) ? 1u : 0u;
            umma_ss(tmem, a, sdesc(vst, 1024, 8192), id, acc);
            umma_ss(tmem + 256, a, sdesc(vst + 4096, 1024, 8192), id, acc);
            umma_commit(smem_u32(&bars.v_empty[s]));
          }
          // The other CTA may refill the slot.
          umma_commit_to(smem_u32(&bars.p_empty[slot]), 1);
        }
        if (ok) ok = event(-1);
        ok = ok && !*aborted;
      }
      if (!ok) timed_out(41);
      umma_commit(smem_u32(&bars.drain));
      mbar_wait(smem_u32(&bars.drain), 0);
    }
  } else if (warp < 11) {
    // ---- output CTA, V: blocks alternate between warps 9 and 10 -------------
    const uint32_t me = warp - 9;
    uint32_t vn = 0;
    bool ok = true;
    while (ok && loop.next(it)) {
      const int nblk = it.blk_end - it.blk_begin;
      const int tail = it.masked ? p.seq_lens[it.branch0] - (it.blk_end - 1) * 16 : 16;
      for (int k0 = 0; k0 < nblk && ok; k0 += 32) {
        bool bad;
        const int mineb = block_of(p, it, it.blk_begin + k0 + lane, bad);
        const int n = min(32, nblk - k0);
        for (int k = 0; k < n; ++k, ++vn) {
          const int phys = __shfl_sync(0xffffffffu, mineb, k);
          if ((vn & 1) != me) continue;
          const uint32_t s = vn % kNV;
          const uint32_t bar = smem_u32(&bars.v_full[s]);
          if (lane == 0) {
            ok = !*aborted && (vn < kNV || mbar_wait(smem_u32(&bars.v_empty[s]),
                                                     (vn / kNV - 1) & 1));
            if (ok) {
              if (phys >= 0) {
                mbar_expect_tx(bar, kVBlk);
                tma_load_5d_at(base + s * kVBlk, &tmV, 0, phys, bar);
              } else {
                mbar_arrive(bar);
              }
            }
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
          if (k0 + k == nblk - 1 && tail < 16) {
            // Rows past the branch's length: zero.
            ok = __all_sync(0xffffffffu, mbar_wait(bar, (vn / kNV) & 1));
            if (!ok) break;
            for (int i = lane; i < (16 - max(tail, 0)) * 64; i += 32) {
              const int row = max(tail, 0) + (i >> 6), c = i & 63;
              st_shared_zero16(base + s * kVBlk + (row >> 3) * 8192 +
                               (c >> 3) * 1024 + (row & 7) * 128 + (c & 7) * 16);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars.v_fix[s]));
          }
        }
      }
    }
    if (lane == 0) {
      if (!ok) timed_out(42);
      // The stages this warp may still have loads in flight for.
      for (uint32_t k = vn > kNV ? vn - kNV : 0; k < vn; ++k)
        if ((k & 1) == me &&
            !mbar_wait(smem_u32(&bars.v_full[k % kNV]), (k / kNV) & 1))
          break;
    }
  } else {
    // ---- output CTA, arrivals of P (warp 11): arm each slot ahead of its
    // copies, and tell the score CTA that its staging tile is free again.
    if (lane == 0) {
      const uint32_t ack = map_rank(smem_u32(&bars.p_ack[0]), 0);
      for (int s = 0; s < kNP; ++s)
        mbar_expect_tx(smem_u32(&bars.p_full[s]), kP + kHdr);
      uint32_t g = 0;
      bool ok = true;
      while (ok && loop.next(it)) {
        const int nblk = it.blk_end - it.blk_begin;
        for (int k0 = 0; k0 < nblk; k0 += kGB, ++g) {
          const uint32_t slot = g % kNP;
          ok = mbar_wait_cluster(smem_u32(&bars.p_full[slot]), (g / kNP) & 1);
          if (!ok) break;
          mbar_expect_tx(smem_u32(&bars.p_full[slot]), kP + kHdr);
          remote_arrive(ack + ((k0 / kGB) & 1) * 8);
        }
      }
      if (!ok) timed_out(43);
    }
  }
  __syncwarp();
  fence_before_sync();
  __syncthreads();
  cluster_sync();
  fence_after_sync();
  if (warp == kMmaWarp) {
    asm volatile(
        "tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
        "r"(kTmemCols)
        : "memory");
  }
}

// ---- merge -------------------------------------------------------------------

struct MergeArgs {
  const int32_t* branches;  // with partial results
  const int32_t* csr_ptr;
  const MergeEntry* csr;
  const float2* ml;
  const float* o;
  __nv_bfloat16* out;
  int n, nb, Hq;
  int64_t partial_rows;
};

// One warp per (branch, head): m* = max m_i, out = sum o_i 2^(m_i - m*) /
// sum l_i 2^(m_i - m*), in one pass with a running maximum.  Bound by the
// partial rows it reads (2 KB each).
__global__ void __launch_bounds__(256) latent_merge_kernel(const MergeArgs a) {
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (w >= (int64_t)a.n * a.Hq) return;
  const int b = a.branches[w / a.Hq], r = (int)(w % a.Hq);
  if (b < 0 || b >= a.nb) return;
  float m = -INFINITY, l = 0.f;
  float4 acc[4] = {};
  const int e1 = a.csr_ptr[b + 1];
  for (int e = a.csr_ptr[b]; e < e1; ++e) {
    const MergeEntry me = a.csr[e];
    if (r < me.r_lo || r >= me.r_hi) continue;
    const int64_t row = (int64_t)me.base + (r - me.r_lo);
    if (row < 0 || row >= a.partial_rows) continue;
    const float2 ml = a.ml[row];
    const float4* src = reinterpret_cast<const float4*>(a.o + row * kRank) + lane;
    float4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = src[i * 32];
    const float m_new = fmaxf(m, ml.x);
    const float x = m == -INFINITY ? 0.f : ex2(m - m_new);
    const float y = ml.x == -INFINITY ? 0.f : ex2(ml.x - m_new);
    l = l * x + ml.y * y;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc[i].x = acc[i].x * x + v[i].x * y;
      acc[i].y = acc[i].y * x + v[i].y * y;
      acc[i].z = acc[i].z * x + v[i].z * y;
      acc[i].w = acc[i].w * x + v[i].w * y;
    }
    m = m_new;
  }
  const float inv = 1.f / l;
  uint2* dst = reinterpret_cast<uint2*>(a.out + ((int64_t)b * a.Hq + r) * kRank) + lane;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    dst[i * 32] = make_uint2(pack_bf16(acc[i].x * inv, acc[i].y * inv),
                             pack_bf16(acc[i].z * inv, acc[i].w * inv));
}

// ---- host side -----------------------------------------------------------------

// One layer's latent pool as 5-D boxes: 64 columns, 8 rows (1024 bytes apart),
// `chunks` 64-column chunks (128), 2 groups of 8 rows (8192), a block (16384).
// A box lands as [group][chunk][8 rows][128 bytes]: 8-row groups a fixed
// chunks x 1024 bytes apart over consecutive blocks, as the K-major and the
// MN-major operands need.
kv_status make_latent_map(CUtensorMap* tm, const void* pool, int64_t blocks,
                          int chunks) {
  const cuuint64_t dims[5] = {64, 8, 8, 2, (cuuint64_t)blocks};
  const cuuint64_t strides[4] = {1024, 128, 8192, 16384};
  const cuuint32_t box[5] = {64, 8, (cuuint32_t)chunks, 2, 1};
  return encode_bf16_map(tm, pool, 5, dims, strides, box);
}

// The position keys: rows of 64, boxes of a block (16 rows).
kv_status make_rope_map(CUtensorMap* tm, const void* pool, int64_t blocks) {
  const cuuint64_t dims[2] = {64, (cuuint64_t)blocks * 16};
  const cuuint64_t strides[1] = {128};
  const cuuint32_t box[2] = {64, 16};
  return encode_bf16_map(tm, pool, 2, dims, strides, box);
}

}  // namespace lat
}  // namespace pkv

using pkv::fail;

extern "C" kv_status paged_latent_decode_attn(
    const void* q, const void* c_pool, const void* r_pool, int64_t num_blocks,
    const int32_t* block_tables, const int32_t* seq_lens,
    const int32_t* prefix_groups, int32_t n_groups, int32_t nb,
    int32_t max_blocks, int32_t Hq, int32_t rank, int32_t rope_dim,
    int32_t block_size, float scale, void* out, const int32_t* plan,
    const kv_decode_plan_info* info, void* workspace, size_t ws_bytes,
    void* stream) {
  namespace lat = pkv::lat;
  pkv::clear_error();
  if (!q || !c_pool || !r_pool || !block_tables || !seq_lens || !out || !plan ||
      !info || !workspace)
    return fail(KV_ERR_INVALID_ARG, "null argument");
  if (n_groups < 0 || (n_groups > 0 && !prefix_groups))
    return fail(KV_ERR_INVALID_ARG, "bad prefix_groups");
  if (rank != KV_LATENT_RANK || rope_dim != KV_LATENT_ROPE)
    return fail(KV_ERR_INVALID_ARG, "a latent cache has rank 512 and rope_dim "
                                    "64, got %d and %d", rank, rope_dim);
  if (nb < 1 || Hq < 1 || max_blocks < 1 || (int64_t)nb * Hq > INT32_MAX / 2)
    return fail(KV_ERR_INVALID_ARG, "bad nb/Hq/max_blocks");
  if (block_size != 16) return fail(KV_ERR_INVALID_ARG, "block_size must be 16");
  if (num_blocks < 1 || num_blocks > (int64_t)INT32_MAX / 16)
    return fail(KV_ERR_INVALID_ARG, "num_blocks out of range");
  if (((uintptr_t)q | (uintptr_t)c_pool | (uintptr_t)r_pool | (uintptr_t)out) & 15)
    return fail(KV_ERR_INVALID_ARG, "q, pools and out must be 16-byte aligned");
  if ((uintptr_t)workspace & 255)
    return fail(KV_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if (!std::isfinite(scale) || !(scale > 0.f))
    return fail(KV_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (!(info->flags & KV_PLAN_LATENT))
    return fail(KV_ERR_INVALID_ARG, "a latent step needs a plan made with "
                                    "KV_PLAN_LATENT");
  if (info->n_tile_items < 1 || info->n_tile_wide_items < 1 ||
      info->n_tile_wide_items > 4096 || info->n_merge_rows < 0 ||
      info->n_merge_rows > nb || info->partial_rows < 0)
    return fail(KV_ERR_INVALID_ARG, "plan info does not match the step");
  const size_t need = pkv::ws_total(info->partial_rows, rank);
  if (ws_bytes < need || (size_t)info->workspace_bytes != need)
    return fail(KV_ERR_INVALID_ARG, "workspace %zu bytes < %zu needed", ws_bytes,
                need);
  CUtensorMap tk, tv, tr;
  if (kv_status s = lat::make_latent_map(&tk, c_pool, num_blocks, 2)) return s;
  if (kv_status s = lat::make_latent_map(&tv, c_pool, num_blocks, 8)) return s;
  if (kv_status s = lat::make_rope_map(&tr, r_pool, num_blocks)) return s;
  const int64_t off_item = pkv::kPlanHeaderInts;
  const int64_t off_pair = off_item + 8 * (int64_t)info->n_tile_items;
  const int64_t off_merge = off_pair + info->n_tile_wide_items + 1;
  const int64_t off_ptr = off_merge + info->n_merge_rows;
  const int64_t off_ent = off_ptr + nb + 1;
  auto* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t st = (cudaStream_t)stream;
  lat::Params p;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.tables = block_tables;
  p.seq_lens = seq_lens;
  p.items = reinterpret_cast<const pkv::WorkItem*>(plan + off_item);
  p.pair_ptr = plan + off_pair;
  p.ml = reinterpret_cast<float2*>(ws + pkv::ws_ml_offset());
  p.o = reinterpret_cast<float*>(ws + pkv::ws_o_offset(info->partial_rows));
  p.out = static_cast<__nv_bfloat16*>(out);
  p.status = reinterpret_cast<pkv::DeviceStatus*>(ws);
  p.nb = nb;
  p.Hq = Hq;
  p.max_blocks = max_blocks;
  p.n_items = info->n_tile_items;
  p.n_pairs = info->n_tile_wide_items;
  p.num_blocks = num_blocks;
  p.partial_rows = info->partial_rows;
  p.scale_log2 = scale * 1.4426950408889634f;
  static std::atomic<uint64_t> opted{0};
  cudaError_t e = pkv::opt_in_smem(lat::latent_decode_kernel, lat::kSmem, opted);
  if (e == cudaSuccess) e = cudaMemsetAsync(ws, 0, sizeof(pkv::DeviceStatus), st);
  if (e != cudaSuccess)
    return fail(KV_ERR_CUDA, "latent step: %s", cudaGetErrorString(e));
  lat::latent_decode_kernel<<<2 * p.n_pairs, lat::kThreads, lat::kSmem, st>>>(
      tk, tv, tr, p);
  e = cudaGetLastError();
  if (e != cudaSuccess)
    return fail(KV_ERR_CUDA, "latent kernel: %s", cudaGetErrorString(e));
  if (info->n_merge_rows > 0) {
    lat::MergeArgs m;
    m.branches = plan + off_merge;
    m.csr_ptr = plan + off_ptr;
    m.csr = reinterpret_cast<const pkv::MergeEntry*>(plan + off_ent);
    m.ml = p.ml;
    m.o = p.o;
    m.out = p.out;
    m.n = info->n_merge_rows;
    m.nb = nb;
    m.Hq = Hq;
    m.partial_rows = p.partial_rows;
    const int64_t warps = (int64_t)m.n * Hq;
    lat::latent_merge_kernel<<<(unsigned)((warps + 7) / 8), 256, 0, st>>>(m);
    e = cudaGetLastError();
    if (e != cudaSuccess)
      return fail(KV_ERR_CUDA, "latent merge: %s", cudaGetErrorString(e));
  }
  return KV_OK;
}
