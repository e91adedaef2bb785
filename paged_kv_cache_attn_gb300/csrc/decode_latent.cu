// Decode attention over a latent pool, absorbed form (paged_latent_decode_attn):
// the entry, the merge, and the kernel for items of more than 16 rows (the others
// run on one SM each, decode_latent_few.cu, beside this one).
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
//     (256 columns, bf16 pairs; an item's Q comes through the K ring and is
//     copied by the tensor pipe itself, so that the next item's scores follow
//     the last ones) and two S buffers (2 x 128 fp32 columns); the
//     position part of Q in shared memory.  K streams through a ring of
//     128-token x 128-dimension stages.  256 softmax threads (two per row, 64
//     columns each, maxima exchanged through shared memory) turn S into P
//     (bf16, base 2, lazy maximum) and store it into the other CTA's shared
//     memory, two tiles of 64 tokens.
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
// Measured: 1.7 us a 128-token tile and pair of SMs (1.13 us of products).  The
// latents pass from L2 twice, as K into one SM and as V into the other: 272 KB a
// tile, 12 TB/s over all SMs while all are in the tile loop, near to what L2 gave a
// kernel that does nothing else (13.9).  An item's end costs 128 rows 4 us (256 KB of
// partial results; an SM stores 29 bytes a cycle, by bulk copies too), a step's start
// 5 to 7 us.  These fixed costs bound a step of 64 branches of 512 to 4096 tokens with
// 128 heads: its 1250 tiles are 29 us of the 56 that 73 pairs take here, with the
// starts and ends of 106 items and 10112 partial rows in the rest; over those 56 us
// nothing is saturated (L2 6.3 TB/s, DRAM 3.4, tensor pipe 32%).
// Prefetches of K or of the position keys into L2 changed nothing or made it
// slower.
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

#include "latent.cuh"
#include "tensor_map.h"

namespace pkv {
namespace lat {

using tc::all_wait;
using tc::all_wait_cluster;
using tc::bar_and;
using tc::cluster_rank;
using tc::cluster_sync;
using tc::elect_one;
using tc::fence_after_sync;
using tc::fence_before_sync;
using tc::idesc;
using tc::map_rank;
using tc::mbar_wait_cluster;
using tc::remote_arrive;
using tc::remote_store16;
using tc::remote_store4;
using tc::sdesc;
using tc::sdesc_plain;
using tc::tma_load_5d_at;
using tc::tmem_ld32;
using tc::tmem_st32;
using tc::tmem_wait_ld;
using tc::tmem_wait_st;
using tc::umma_commit;
using tc::umma_commit_to;
using tc::umma_copy;
using tc::umma_ss;
using tc::umma_ts;
using tc::uniform;

constexpr int kT = 128;            // tokens of a score tile
constexpr int kTB = kT / 16;       // its blocks
constexpr int kG = 64;             // tokens of a P tile
constexpr int kGB = kG / 16;

// Score CTA's shared memory.
constexpr int kQr = 128 * 128;               // position part of Q
constexpr int kKDim = 128;                   // dimensions of a K stage
constexpr int kKParts = kRank / kKDim;       // stages of a tile
constexpr int kKBox = 16 * kKDim * 2;        // one block's part: a box
constexpr int kKStage = kTB * kKBox;
// Stages are refilled one by one, but waited for in pairs: a wait costs the
// issuing warp as much as one or two MMAs.
constexpr int kNK = 6;
static_assert(kKParts % 2 == 0 && kNK % 2 == 0, "stages come in pairs");
constexpr int kRTile = kT * 128;             // position keys of a tile
constexpr int kOffK = kQr;
constexpr int kOffR = kOffK + kNK * kKStage;
constexpr int kScoreSmem = kOffR + kRTile;
// Output CTA's shared memory.
constexpr int kVBlk = 16 * kRank * 2;        // one block
constexpr int kVB = 2;                       // blocks of a V stage
constexpr int kVStage = kVB * kVBlk;
constexpr int kNV = 4;
// A P tile: [8 chunks of 8 tokens][128 rows][16 bytes], the K-major layout
// without swizzle; a warp's store of a chunk is 512 contiguous bytes.
constexpr int kP = 128 * 128;
constexpr int kPChunk = 128 * 16;
constexpr int kNP = 4;
// With it 128 rescale factors and a flag word for each row warp.
constexpr int kHdr = 512 + 16;
constexpr int kOffP = kNV * kVStage;
constexpr int kOffHdr = kOffP + kNP * kP;
constexpr int kOffFin = kOffHdr + kNP * kHdr;
constexpr int kOffTurn = (kOffFin + 2 * 512 + 127) & ~127;  // 2 KB a row warp
constexpr int kOutSmem = kOffTurn + 8 * 2048;
constexpr int kTiles = kScoreSmem > kOutSmem ? kScoreSmem : kOutSmem;

constexpr int kThreads = 13 * 32;
constexpr int kRowThreads = 256;             // warps 0-7
constexpr int kMmaWarp = 8;                  // with 12 (score) or 11 (output CTA)
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 256;              // score CTA: Q 0..255, S 256..511
constexpr float kRescale = 8.f;              // lazy-max threshold (log2 units)

// Barriers and small arrays, behind the tiles; at the same place in both CTAs.
struct Small {
  // score CTA
  uint64_t k_full[kNK / 2], k_empty[kNK], r_full[2], r_empty;
  uint64_t qr_full, qr_empty, q_ready, q_free, turn[2], s_full[2], s_empty[2];
  uint64_t p_empty[kNP];   // the other side has consumed P slot i
  uint64_t fin_empty[2];
  // output CTA
  uint64_t v_full[kNV / 2], v_empty[kNV], v_fix[kNV], p_full[kNP], fin_full[2];
  uint64_t event, o_ok;
  uint64_t drain[2];
  uint32_t tmem_base;
  int aborted;
  int event_what;          // slot of a rescale, or -1: item done
  float max_of[2][2][128]; // [tile parity][half][row]
  float sum_of[128];
};
// The tiles need 1024-byte alignment and nearly all of the shared memory, so
// there is no static shared memory in front of them.
constexpr int kSmem = kTiles + (int)sizeof(Small);
static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");

__device__ __forceinline__ int n_tiles(const WorkItem& it) {
  return (it.blk_end - it.blk_begin + kTB - 1) / kTB;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    latent_decode_kernel(const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV,
                         const __grid_constant__ CUtensorMap tmR,
                         const __grid_constant__ CUtensorMap tmQ,
                         const __grid_constant__ CUtensorMap tmQall,
                         const Params p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Small& bars = *reinterpret_cast<Small*>(smem + kTiles);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool scores = rank == 0;
  const int pair = blockIdx.x >> 1;
  const uint32_t base = smem_u32(smem);
  volatile int* aborted = &bars.aborted;
  if (base & 1023) {  // never, with no static shared memory; both CTAs agree
    if (threadIdx.x == 0) record_status(p.status, KV_ERR_INTERNAL, (int)base);
    return;
  }

  if (threadIdx.x == 0) {
    for (int s = 0; s < kNK; ++s) {
      mbar_init(smem_u32(&bars.k_full[s / 2]), 2);  // both producer warps
      mbar_init(smem_u32(&bars.k_empty[s]), 1);
    }
    mbar_init(smem_u32(&bars.r_empty), 1);
    mbar_init(smem_u32(&bars.qr_full), 1);
    mbar_init(smem_u32(&bars.qr_empty), 2);      // both product warps
    mbar_init(smem_u32(&bars.q_ready), 1);
    mbar_init(smem_u32(&bars.q_free), 2);
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&bars.r_full[b]), 1);
      mbar_init(smem_u32(&bars.turn[b]), 1);
      mbar_init(smem_u32(&bars.s_full[b]), 1);
      mbar_init(smem_u32(&bars.s_empty[b]), 8);
      mbar_init(smem_u32(&bars.fin_empty[b]), 8);  // the other side's row warps
      mbar_init(smem_u32(&bars.fin_full[b]), 1);
    }
    for (int s = 0; s < kNP; ++s) {
      mbar_init(smem_u32(&bars.p_empty[s]), 2);    // both product warps
      mbar_init(smem_u32(&bars.p_full[s]), 1);
    }
    for (int s = 0; s < kNV; ++s) {
      mbar_init(smem_u32(&bars.v_full[s / 2]), 2);  // both producer warps
      mbar_init(smem_u32(&bars.v_empty[s]), 2);
      mbar_init(smem_u32(&bars.v_fix[s]), 1);    // masked rows zeroed
    }
    mbar_init(smem_u32(&bars.event), 4);         // two product warps, each
                                                 // itself and its commit
    mbar_init(smem_u32(&bars.o_ok), 8);
    mbar_init(smem_u32(&bars.drain[0]), 1);
    mbar_init(smem_u32(&bars.drain[1]), 1);
    bars.aborted = 0;
    fence_mbar_init();
    // What will arrive here from the other CTA, armed a phase ahead.
    if (!scores) {
      for (int s = 0; s < kNP; ++s)
        mbar_expect_tx(smem_u32(&bars.p_full[s]), kP + kHdr);
      for (int f = 0; f < 2; ++f) mbar_expect_tx(smem_u32(&bars.fin_full[f]), 512);
    }
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    tma_prefetch_desc(&tmR);
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmQall);
  }
  if (warp == kMmaWarp) {
    asm volatile(
        "tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::
            "r"(smem_u32(&bars.tmem_base)),
        "r"(kTmemCols)
        : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::
                     : "memory");
  }
  // Launched early (the status word is being cleared): no global memory before
  // this point.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (p.trigger) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  ItemLoop<false> loop(p, pair);
  fence_before_sync();
  __syncthreads();
  cluster_sync();  // the other CTA's barriers are ready too
  fence_after_sync();
  const uint32_t tmem = bars.tmem_base;
  WorkItem it;
  auto timed_out = [&](int site) {
    if (!*aborted) record_status(p.status, KV_ERR_TIMEOUT, site);
    atomicExch(&bars.aborted, 1);
  };

  if (scores && warp < 8) {
    // ---- score CTA, rows: thread = (row r, half of a tile's columns) --------
    const int wg = warp >> 2;
    const int r = threadIdx.x & 127;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t peer_p = map_rank(base + kOffP, 1) + r * 16;
    const uint32_t peer_hdr = map_rank(base + kOffHdr, 1);
    const uint32_t peer_fin = map_rank(base + kOffFin, 1) + r * 4;
    const uint32_t peer_full = map_rank(smem_u32(&bars.p_full[0]), 1);
    uint32_t tc_n = 0;   // tiles so far
    uint32_t g_n = 0;    // P tiles sent so far, by both halves
    uint32_t fin_n = 0;  // items whose sums were sent
    bool ok = true;
    while (ok && loop.next(it)) {
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
        const bool w = all_wait(smem_u32(&bars.s_full[b]), (tc_n >> 1) & 1);
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
        bars.max_of[b][wg][r] = mx;
        // Every row thread agrees whether to go on.
        ok = bar_and(1, kRowThreads, w && !*aborted);
        if (!ok) break;
        const float m_tile = fmaxf(mx, bars.max_of[b][wg ^ 1][r]) * p.scale_log2;
        // Rows past the item's hold whatever was there: they never ask.
        const bool need = m_tile > m_used + kRescale && r < it.nrows;
        const float m_new = need ? m_tile : m_used;
        const float alpha = need ? ex2(m_used - m_new) : 1.f;
        m_used = m_new;
        l *= alpha;
        const bool two = left > kG;  // the tile has a second P tile
        if (wg == 0 || two) {
          const uint32_t g = g_n + wg, slot = g % kNP;
          if (g >= kNP && !all_wait_cluster(smem_u32(&bars.p_empty[slot]),
                                             (g / kNP - 1) & 1))
            timed_out(32);
          const uint32_t bar = peer_full + slot * 8;
          const uint32_t dst = peer_p + slot * kP;
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
            remote_store16(dst + c * kPChunk, pk[0], pk[1], pk[2], pk[3], bar);
          }
          l += (sum4[0] + sum4[1]) + (sum4[2] + sum4[3]);
          // O is rescaled once a tile, before any of its products: the first P
          // tile's flags say so, the second's are 0.
          const uint32_t hdr = peer_hdr + slot * kHdr;
          const bool moved = __any_sync(0xffffffffu, need && j > 0) && wg == 0;
          remote_store4(hdr + r * 4, __float_as_uint(alpha), bar);
          if (lane == 0) remote_store4(hdr + 512 + (warp & 3) * 4, moved, bar);
        }
        g_n += two ? 2 : 1;
      }
      if (!ok) break;
      // The row's sum over both halves.
      if (wg == 1) bars.sum_of[r] = l;
      ok = bar_and(1, kRowThreads, !*aborted);
      if (!ok) break;
      if (wg == 0) {
        l += bars.sum_of[r];
        if (it.g == 0) {
          if (r < it.nrows) p.ml[it.prow_base + r] = make_float2(m_used, l);
        } else {
          const int f = fin_n & 1;
          if (fin_n >= 2 &&
              !all_wait_cluster(smem_u32(&bars.fin_empty[f]), (fin_n / 2 - 1) & 1))
            timed_out(33);
          remote_store4(peer_fin + f * 512, __float_as_uint(1.f / l),
                        map_rank(smem_u32(&bars.fin_full[f]), 1));
        }
      }
      if (it.g != 0) ++fin_n;
      // bars.sum_of is read before the next item's sums are written: the tiles of
      // that item pass barrier 1 in between.
    }
    // What this CTA stored has been consumed, and every arrival from the other
    // side is in, before this CTA may leave.
    if (threadIdx.x == 0) {
      for (uint32_t g = g_n > kNP ? g_n - kNP : 0; g < g_n; ++g)
        if (!mbar_wait_cluster(smem_u32(&bars.p_empty[g % kNP]), (g / kNP) & 1))
          break;
      for (uint32_t f = fin_n > 2 ? fin_n - 2 : 0; f < fin_n; ++f)
        if (!mbar_wait_cluster(smem_u32(&bars.fin_empty[f & 1]), (f / 2) & 1))
          break;
    }
  } else if (scores && (warp == kMmaWarp || warp == 12)) {
    // ---- score CTA, products (uniform warps, one lane issues): warp 8 the even
    // tiles (S buffer 0), warp 12 the odd ones, so that one warp's waits lie
    // behind the other's products.  A warp waits for K only in its turn (the
    // other has seen all of the stages before), which also keeps each
    // barrier's phases unambiguous.
    constexpr uint32_t id = idesc(128, kT, false);
    const bool lead = elect_one();
    const uint32_t w = warp == kMmaWarp ? 0 : 1;
    const uint32_t d = tmem + kColS + w * kT;
    uint32_t tn = 0, kp = 0, in = 0, turns = 0;  // tiles, pairs of stages, items
    bool ok = true;
    auto wait_pair = [&](uint32_t q) {
      const bool got = all_wait(smem_u32(&bars.k_full[q % (kNK / 2)]),
                                (q / (kNK / 2)) & 1);
      fence_after_sync();
      return got;
    };
    while (ok && loop.next(it)) {
      const int nt = uniform(n_tiles(it));
      const bool first = (tn & 1) == w;
      // The previous item's products have read their Q.
      if (in > 0) ok = all_wait(smem_u32(&bars.q_free), (in - 1) & 1);
      if (first) {
        // The warp of the item's first tile brings Q: its latent part comes
        // through the K ring and is copied to TMEM.
        for (int c = 0; c < kKParts / 2 && ok; ++c) {
          ok = wait_pair(kp + c);
          const uint32_t s = 2 * ((kp + c) % (kNK / 2));
          if (ok && lead) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint64_t src = sdesc(base + kOffK + (s + h) * kKStage, 16, 1024);
#pragma unroll
              for (int kk = 0; kk < kKDim / 16; ++kk)
                umma_copy(tmem + (c * 2 + h) * (kKDim / 2) + kk * 8,
                          src + (((kk >> 2) * kQr + (kk & 3) * 32) >> 4));
              umma_commit(smem_u32(&bars.k_empty[s + h]));
            }
          }
          __syncwarp();
        }
        if (lead) umma_commit(smem_u32(&bars.q_ready));
        __syncwarp();
      } else if (ok) {
        ok = all_wait(smem_u32(&bars.q_ready), in & 1);
      }
      if (ok) ok = all_wait(smem_u32(&bars.qr_full), in & 1);
      fence_after_sync();
      for (int j = first ? 0 : 1; j < nt && ok; j += 2) {
        const uint32_t t = (tn + j) >> 1;  // this warp's tiles so far
        if (t > 0) ok = all_wait(smem_u32(&bars.s_empty[w]), (t - 1) & 1);
        // The position part first; after the item's last, the next item's may
        // be loaded.
        ok = ok && all_wait(smem_u32(&bars.r_full[w]), t & 1);
        if (!ok) break;
        fence_after_sync();
        const uint64_t qd = sdesc(base, 16, 1024);
        const uint64_t rd = sdesc(base + kOffR, 16, 1024);
        if (lead) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_ss(d, qd + kk * 2, rd + kk * 2, id, kk > 0 ? 1u : 0u);
          umma_commit(smem_u32(&bars.r_empty));
          if (j + 2 >= nt) umma_commit(smem_u32(&bars.qr_empty));
        }
        __syncwarp();
        if (j > 0) {
          ok = all_wait(smem_u32(&bars.turn[w]), turns & 1);
          ++turns;
        }
        for (int c = 0; c < kKParts / 2 && ok; ++c) {
          const uint32_t q = kp + (1 + j) * (kKParts / 2) + c;
          ok = wait_pair(q);
          if (!ok) break;
          const uint32_t s = 2 * (q % (kNK / 2));
          if (lead) {
            if (c == kKParts / 2 - 1 && j + 1 < nt)
              mbar_arrive(smem_u32(&bars.turn[w ^ 1]));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint64_t kd =
                  sdesc(base + kOffK + (s + h) * kKStage, 16, kKBox / 2);
              const uint32_t qa = tmem + (c * 2 + h) * (kKDim / 2);
#pragma unroll
              for (int kk = 0; kk < kKDim / 16; ++kk)
                umma_ts(d, qa + kk * 8,
                        kd + (((kk >> 2) * 1024 + (kk & 3) * 32) >> 4), id, 1u);
              umma_commit(smem_u32(&bars.k_empty[s + h]));
            }
          }
          __syncwarp();
        }
        if (!ok) break;
        if (lead) umma_commit(smem_u32(&bars.s_full[w]));
        __syncwarp();
      }
      if (!ok) break;
      if (lead) {
        if (first || nt > 1) {
          umma_commit(smem_u32(&bars.q_free));
        } else {  // no tile of this item was this warp's
          mbar_arrive(smem_u32(&bars.qr_empty));
          mbar_arrive(smem_u32(&bars.q_free));
        }
      }
      __syncwarp();
      ++in;
      tn += nt;
      kp += (1 + nt) * (kKParts / 2);
      ok = !*aborted;
    }
    if (lead) {
      if (!ok) timed_out(34);
      umma_commit(smem_u32(&bars.drain[w]));
      mbar_wait(smem_u32(&bars.drain[w]), 0);
    }
  } else if (scores && warp < 11) {
    // ---- score CTA, K: warps 9 and 10 take every other stage; one box is a
    // block x 128 dimensions, the eight of a stage issued by eight lanes at
    // once (an issue costs a warp about 220 ns and 30 ns a box).
    const uint32_t me = warp - 9;
    uint32_t kn = 0;
    bool ok = true;
    // Stage kn is free; arm it.
    auto arm = [&](uint32_t bytes) {
      const uint32_t s = kn % kNK;
      ok = kn < kNK || all_wait(smem_u32(&bars.k_empty[s]), (kn / kNK - 1) & 1);
      ok = __all_sync(0xffffffffu, ok && !*aborted);
      if (ok && lane == 0) {
        if (bytes > 0)
          mbar_expect_tx(smem_u32(&bars.k_full[s / 2]), bytes);
        else
          mbar_arrive(smem_u32(&bars.k_full[s / 2]));
      }
      __syncwarp();
      return ok;
    };
    while (ok && loop.next(it)) {
      const int nt = n_tiles(it);
      const int blk = it.blk_begin + lane;
      // A tile's block ids are read while the one before waits for its stages.
      bool bad = false, next_bad = false;
      int next = lane < kTB ? block_of(p, it, blk, next_bad) : -1;
      // Q comes first, as stages of 128 rows x 128 dimensions in boxes of 64
      // dimensions and 16 rows, or of 128 rows for an item with more than 64
      // (the rows behind the item's are computed on and not stored).
      const bool tall = it.nrows > 64;
      const int qb = tall ? 8 : (it.nrows + 15) / 16;
      for (int c = 0; c < kKParts; ++c, ++kn) {
        if ((kn & 1) != me) continue;
        if (!arm(qb * (kKDim / 64) * 2048)) break;
        const uint32_t s = kn % kNK;
        const int part = lane / 8, row = lane % 8;
        if (lane < 8 * (kKDim / 64) && row < (tall ? 1 : qb))
          tma_load_2d(base + kOffK + s * kKStage + part * kQr + row * 2048,
                      tall ? &tmQall : &tmQ,
                      c * kKDim + part * 64,
                      it.branch0 * p.Hq + it.row0 + row * 16,
                      smem_u32(&bars.k_full[s / 2]));
        __syncwarp();
      }
      for (int j = 0; j < nt && ok; ++j) {
        const int phys = next;
        bad = next_bad;
        next = -1;
        if (lane < kTB && j + 1 < nt)
          next = block_of(p, it, blk + (j + 1) * kTB, next_bad);
        if (bad && me == 0)
          record_status(p.status, KV_ERR_DEVICE,
                        p.tables[(int64_t)it.branch0 * p.max_blocks + blk + j * kTB]);
        const int n = __popc(__ballot_sync(0xffffffffu, phys >= 0));
        for (int c = 0; c < kKParts; ++c, ++kn) {
          if ((kn & 1) != me) continue;
          if (!arm(n * kKBox)) break;
          const uint32_t s = kn % kNK;
          if (phys >= 0)
            tma_load_5d_at(base + kOffK + s * kKStage + lane * kKBox, &tmK,
                           c * (kKDim / 64), phys, smem_u32(&bars.k_full[s / 2]));
          __syncwarp();
        }
      }
    }
    if (lane == 0) {
      if (!ok) timed_out(35);
      for (uint32_t k = kn > kNK ? kn - kNK : 0; k < kn; ++k)
        if ((k & 1) == me &&
            !mbar_wait(smem_u32(&bars.k_full[k % kNK / 2]), (k / kNK) & 1))
          break;
    }
  } else if (scores) {
    // ---- score CTA, position parts of Q and K (warp 11) ---------------------
    uint32_t tn = 0, in = 0;
    bool ok = true;
    while (ok && loop.next(it)) {
      const int nt = n_tiles(it);
      const int qb = (it.nrows + 15) / 16;
      bool bad;
      int next = lane < kTB ? block_of(p, it, it.blk_begin + lane, bad) : -1;
      ok = in == 0 || all_wait(smem_u32(&bars.qr_empty), (in - 1) & 1);
      ok = __all_sync(0xffffffffu, ok && !*aborted);
      if (!ok) break;
      if (lane == 0) mbar_expect_tx(smem_u32(&bars.qr_full), qb * 2048);
      __syncwarp();
      ++in;
      if (lane < qb)
        tma_load_2d(base + lane * 2048, &tmQ, kRank,
                    it.branch0 * p.Hq + it.row0 + lane * 16,
                    smem_u32(&bars.qr_full));
      __syncwarp();
      for (int j = 0; j < nt; ++j, ++tn) {
        const int phys = next;
        next = -1;
        if (lane < kTB && j + 1 < nt)
          next = block_of(p, it, it.blk_begin + (j + 1) * kTB + lane, bad);
        const int n = __popc(__ballot_sync(0xffffffffu, phys >= 0));
        ok = tn == 0 || all_wait(smem_u32(&bars.r_empty), (tn - 1) & 1);
        ok = __all_sync(0xffffffffu, ok && !*aborted);
        if (!ok) break;
        if (lane == 0) {
          if (n > 0)
            mbar_expect_tx(smem_u32(&bars.r_full[tn & 1]), n * 2048);
          else
            mbar_arrive(smem_u32(&bars.r_full[tn & 1]));
        }
        __syncwarp();
        if (phys >= 0)
          tma_load_2d(base + kOffR + lane * 2048, &tmR, 0, phys * 16,
                      smem_u32(&bars.r_full[tn & 1]));
        __syncwarp();
      }
    }
    if (lane == 0) {
      if (!ok) timed_out(36);
      report_bad<false>(p, pair);
      if (tn > 0)
        mbar_wait(smem_u32(&bars.r_full[(tn - 1) & 1]), ((tn - 1) >> 1) & 1);
      if (in > 0) mbar_wait(smem_u32(&bars.qr_full), (in - 1) & 1);
    }
  } else if (warp < 8) {
    // ---- output CTA, rows: thread = (row r, half of the 512 columns) ---------
    const int wg = warp >> 2;
    const int r = threadIdx.x & 127;
    const uint32_t orow =
        tmem + ((uint32_t)((warp & 3) * 32) << 16) + wg * (kRank / 2);
    uint32_t ev = 0, fin_n = 0;
    bool ok = true;
    while (ok && loop.next(it)) {
      for (;;) {
        ok = all_wait(smem_u32(&bars.event), ev & 1);
        if (!ok) break;
        ++ev;
        fence_after_sync();
        const int slot = *(volatile int*)&bars.event_what;
        if (slot < 0) break;
        // A maximum moved: this row of O times its factor.
        const float alpha =
            reinterpret_cast<const float*>(smem + kOffHdr + slot * kHdr)[r];
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
        ok = all_wait_cluster(smem_u32(&bars.fin_full[f]), (fin_n >> 1) & 1);
        if (!ok) break;
        inv = reinterpret_cast<const float*>(smem + kOffFin + f * 512)[r];
        ++fin_n;
        // The factors are in registers: once every row warp says so, the slot
        // (armed again by the first) may be filled for the item after next.
        __syncwarp();
        if (lane == 0) {
          if (warp == 0) mbar_expect_tx(smem_u32(&bars.fin_full[f]), 512);
          remote_arrive(map_rank(smem_u32(&bars.fin_empty[f]), 0));
        }
      }
      // A warp turns 32 rows x 64 bytes at a time in its 2 KB of shared memory
      // (16-byte pieces swizzled by the row), so that a store covers whole
      // sectors of eight rows instead of 16-byte pieces of 32 (128 rows of
      // partial results took 10 us that way).  The prefill's put_rows in its place
      // made steps of 17 to 30 us 0.1 us slower.
      const int wrow = (warp & 3) * 32;          // the warp's first row
      if (wrow < it.nrows) {
        uint8_t* turn = smem + kOffTurn + warp * 2048;
        const int n = min(32, it.nrows - wrow);
        uint8_t* dst = direct
            ? reinterpret_cast<uint8_t*>(
                  p.out + ((int64_t)it.branch0 * p.Hq + it.row0 + wrow) * kRank +
                  wg * (kRank / 2))
            : reinterpret_cast<uint8_t*>(
                  p.o + ((int64_t)it.prow_base + wrow) * kRank + wg * (kRank / 2));
        const int pitch = direct ? kRank * 2 : kRank * 4;  // bytes of a row
        auto put = [&](const uint32_t (&w)[16]) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(
                turn + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4)) =
                make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int rr = k * 8 + (lane >> 2), c = lane & 3;
            const uint4 x = *reinterpret_cast<const uint4*>(
                turn + rr * 64 + ((c ^ ((rr >> 1) & 3)) << 4));
            if (rr < n)
              *reinterpret_cast<uint4*>(dst + (int64_t)rr * pitch + c * 16) = x;
          }
          dst += 64;
          __syncwarp();
        };
#pragma unroll 1
        for (int c = 0; c < kRank / 2; c += 32) {
          uint32_t v[32], w[16];
          tmem_ld32(orow + c, v);
          tmem_wait_ld();
          if (direct) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              w[i] = pack_bf16(__uint_as_float(v[2 * i]) * inv,
                               __uint_as_float(v[2 * i + 1]) * inv);
            put(w);
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
              for (int i = 0; i < 16; ++i) w[i] = v[h * 16 + i];
              put(w);
            }
          }
        }
      }
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars.o_ok));
    }
    if (!ok && lane == 0) timed_out(40);
  } else if (warp == kMmaWarp || warp == 11) {
    // ---- output CTA, products (uniform warps, one lane issues): warp 8 the
    // first 256 columns of O, warp 11 the others.  A warp waits about half of
    // the time that its products take; two keep the tensor pipe busy.
    const int oh = warp == kMmaWarp ? 0 : 1;
    constexpr uint32_t id = idesc(128, 256, true);
    const bool lead = elect_one();
    uint32_t g = 0, ev = 0, fixes = 0;
    bool ok = true;
    // Once every product so far is done, the rows act: rescale O with the
    // factors in P slot `what`, or (-1) write the item's result.
    auto event = [&](int what) {
      if (lead) {
        if (oh == 0) *(volatile int*)&bars.event_what = what;
        mbar_arrive(smem_u32(&bars.event));
        umma_commit(smem_u32(&bars.event));
      }
      __syncwarp();
      const bool done = all_wait(smem_u32(&bars.o_ok), ev & 1);
      ++ev;
      fence_after_sync();
      return done;
    };
    while (ok && loop.next(it)) {
      const int nblk = uniform(it.blk_end - it.blk_begin);
      const int tail =
          uniform(it.masked ? p.seq_lens[it.branch0] - (it.blk_end - 1) * 16 : 16);
      for (int k0 = 0; k0 < nblk && ok; k0 += kGB, ++g) {
        const uint32_t slot = g % kNP;
        ok = all_wait_cluster(smem_u32(&bars.p_full[slot]), (g / kNP) & 1);
        if (!ok) break;
        // Arm the slot's next phase; P came as ordinary stores.
        if (lead && oh == 0)
          mbar_expect_tx(smem_u32(&bars.p_full[slot]), kP + kHdr);
        fence_proxy_async_smem();
        if (k0 > 0 && k0 % kTB == 0) {
          const int f = lane < 4 ? *reinterpret_cast<volatile int*>(
                                       smem + kOffHdr + slot * kHdr + 512 + lane * 4)
                                 : 0;
          if (__any_sync(0xffffffffu, f != 0)) {
            ok = event((int)slot);
            if (!ok) break;
          }
        }
        const uint64_t pd = sdesc_plain(base + kOffP + slot * kP, kPChunk, 128);
        const int nk = min(kGB, nblk - k0);
        // All of the P tile's V (a pair of stages) first, so that its products
        // are issued without a pause.
        ok = all_wait(smem_u32(&bars.v_full[g % (kNV / 2)]), (g / (kNV / 2)) & 1);
        const uint32_t v0 = 2 * (g % (kNV / 2));  // its first stage
        if (ok && k0 + nk == nblk && tail < 16) {
          const uint32_t s = v0 + (nk - 1) / kVB;
          ok = all_wait(smem_u32(&bars.v_fix[s]), (fixes >> s) & 1);
          fixes ^= 1u << s;  // the stage's next fix has the other parity
        }
        if (!ok) break;
        fence_after_sync();
        if (lead) {
#pragma unroll
          for (int k = 0; k < kGB; ++k) {
            if (k < nk) {
              const uint64_t vd = sdesc(base + (v0 + k / kVB) * kVStage +
                                            (k % kVB) * kVBlk + oh * 4096,
                                        1024, 8192);
              umma_ss(tmem + oh * 256, pd + k * (2 * kPChunk >> 4), vd, id,
                      (k0 > 0 || k > 0) ? 1u : 0u);
            }
            if (k % kVB == kVB - 1) umma_commit(smem_u32(&bars.v_empty[v0 + k / kVB]));
          }
          // The other CTA may refill the slot.
          umma_commit_to(smem_u32(&bars.p_empty[slot]), 1);
        }
        __syncwarp();
      }
      if (ok) ok = event(-1);
      ok = ok && !*aborted;
    }
    if (lead) {
      if (!ok) timed_out(41);
      umma_commit(smem_u32(&bars.drain[oh]));
      mbar_wait(smem_u32(&bars.drain[oh]), 0);
    }
  } else if (warp < 11) {
    // ---- output CTA, V: the two stages (of two blocks) of a P tile, warp 9 the
    // first and warp 10 the second, empty or not.
    const uint32_t me = warp - 9;
    uint32_t vn = 0;  // P tiles so far
    bool ok = true;
    while (ok && loop.next(it)) {
      const int nblk = it.blk_end - it.blk_begin;
      const int tail = max(
          it.masked ? p.seq_lens[it.branch0] - (it.blk_end - 1) * 16 : 16, 0);
      const int blk = it.blk_begin + me * kVB + lane;
      bool bad;
      int next = lane < kVB ? block_of(p, it, blk, bad) : -1;
      for (int k0 = 0; k0 < nblk && ok; k0 += kGB, ++vn) {
        const int phys = next;
        next = lane < kVB && k0 + kGB < nblk ? block_of(p, it, blk + k0 + kGB, bad)
                                             : -1;
        const uint32_t s = 2 * (vn % (kNV / 2)) + me;
        const uint32_t use = vn / (kNV / 2);  // earlier uses of the stage
        const uint32_t bar = smem_u32(&bars.v_full[s / 2]);
        const int n_load = __popc(__ballot_sync(0xffffffffu, phys >= 0));
        ok = use == 0 || all_wait(smem_u32(&bars.v_empty[s]), (use - 1) & 1);
        ok = __all_sync(0xffffffffu, ok && !*aborted);
        if (!ok) break;
        if (lane == 0) {
          if (n_load > 0)
            mbar_expect_tx(bar, n_load * kVBlk);
          else
            mbar_arrive(bar);
        }
        __syncwarp();
        if (phys >= 0)
          tma_load_5d_at(base + s * kVStage + lane * kVBlk, &tmV, 0, phys, bar);
        __syncwarp();
        const int last = nblk - 1 - k0 - me * kVB;  // the last block's place here
        if (tail < 16 && last >= 0 && last < kVB) {
          // Rows of the last block past the branch's length: zero.
          ok = all_wait(bar, use & 1);
          if (!ok) break;
          const uint32_t dst = base + s * kVStage + last * kVBlk;
          for (int i = lane; i < (16 - tail) * 64; i += 32) {
            const int row = tail + (i >> 6), c = i & 63;
            st_shared_zero16(dst + (row >> 3) * 8192 + (c >> 3) * 1024 +
                             (row & 7) * 128 + (c & 7) * 16);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bars.v_fix[s]));
        }
      }
    }
    if (lane == 0) {
      if (!ok) timed_out(42);
      // The stages this warp may still have loads in flight for.
      for (uint32_t k = vn > kNV / 2 ? vn - kNV / 2 : 0; k < vn; ++k)
        if (!mbar_wait(smem_u32(&bars.v_full[k % (kNV / 2)]), (k / (kNV / 2)) & 1))
          break;
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

// Clears the status word; a kernel, so that the attention kernel's launch and
// set-up overlap it.
__global__ void latent_clear_kernel(DeviceStatus* status) {
  if (threadIdx.x == 0) *status = DeviceStatus{};
}

// ---- merge -------------------------------------------------------------------

struct MergeArgs {
  const int32_t* branches;  // with partial results
  const int32_t* csr_ptr;
  const MergeEntry* csr;
  const float2* ml;
  const float* o;
  __nv_bfloat16* out;
  DeviceStatus* status;
  int n, nb, Hq, n_csr;
  int64_t partial_rows;
};

// One warp per (branch, head): m* = max m_i, out = sum o_i 2^(m_i - m*) /
// sum l_i 2^(m_i - m*), in one pass with a running maximum.  Bound by the
// partial rows it reads (2 KB each).  In a malformed plan, a row without an entry or
// with entries behind the list's end is recorded and left as it was.
__global__ void __launch_bounds__(256) latent_merge_kernel(const MergeArgs a) {
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  // Its launch overlaps the end of the attention kernel (which lets nothing start
  // beside it but the other one); results are complete and visible from here on.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (w >= (int64_t)a.n * a.Hq) return;
  const int b = a.branches[w / a.Hq], r = (int)(w % a.Hq);
  if (b < 0 || b >= a.nb) return;
  // A lane an entry for the weights, then every entry's row over the lanes: the
  // rows' loads depend on nothing of one another.
  float m = -INFINITY, l = 0.f;
  float4 acc[4] = {};
  int e0 = a.csr_ptr[b], e1 = a.csr_ptr[b + 1];
  if (e0 < 0 || e1 > a.n_csr) e0 = e1;
  for (; e0 < e1; e0 += 32) {
    const int n = min(32, e1 - e0);
    int row = -1;
    float2 ml = make_float2(-INFINITY, 0.f);
    if (lane < n) {
      const MergeEntry me = a.csr[e0 + lane];
      const int64_t at = (int64_t)me.base + (r - me.r_lo);
      if (r >= me.r_lo && r < me.r_hi && at >= 0 && at < a.partial_rows) {
        row = (int)at;
        ml = a.ml[row];
      }
    }
    float m_new = fmaxf(m, ml.x);
#pragma unroll
    for (int k = 16; k > 0; k >>= 1)
      m_new = fmaxf(m_new, __shfl_xor_sync(0xffffffffu, m_new, k));
    const float w = ml.x == -INFINITY ? 0.f : ex2(ml.x - m_new);
    float sum = ml.y * w;
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
    const float x = m == -INFINITY ? 0.f : ex2(m - m_new);
    l = l * x + sum;
    m = m_new;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc[i].x *= x;
      acc[i].y *= x;
      acc[i].z *= x;
      acc[i].w *= x;
    }
#pragma unroll 2
    for (int e = 0; e < n; ++e) {
      const int at = __shfl_sync(0xffffffffu, row, e);
      const float y = __shfl_sync(0xffffffffu, w, e);
      if (at < 0 || y == 0.f) continue;
      const float4* src =
          reinterpret_cast<const float4*>(a.o + (int64_t)at * kRank) + lane;
      float4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = src[i * 32];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[i].x += v[i].x * y;
        acc[i].y += v[i].y * y;
        acc[i].z += v[i].z * y;
        acc[i].w += v[i].w * y;
      }
    }
  }
  if (l == 0.f) {  // no entry
    if (lane == 0) record_status(a.status, KV_ERR_DEVICE, -1 - b);
    return;
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

// Rows of `width` values in boxes of 64 values (a block's position keys, or
// query rows).
kv_status make_rows_map(CUtensorMap* tm, const void* base, int64_t rows, int width,
                        int box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)width * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  return encode_bf16_map(tm, base, 2, dims, strides, box);
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
  if (info->n_tile_items < 1 || info->n_tile_wide_items < 0 ||
      info->n_tile_wide_items > 4096 || info->n_row_warp_items < 0 ||
      info->n_row_warp_items > 8192 || info->n_row_items < 0 ||
      info->n_row_items > info->n_tile_items ||
      (info->n_row_items > 0) != (info->n_row_warp_items > 0) ||
      (info->n_row_items < info->n_tile_items) != (info->n_tile_wide_items > 0) ||
      info->n_merge_rows < 0 || info->n_merge_rows > nb || info->partial_rows < 0 ||
      info->latent_rows != nb * Hq)
    return fail(KV_ERR_INVALID_ARG, "plan info does not match the step");
  const size_t need = pkv::ws_total(info->partial_rows, rank);
  if (ws_bytes < need || (size_t)info->workspace_bytes != need)
    return fail(KV_ERR_INVALID_ARG, "workspace %zu bytes < %zu needed", ws_bytes,
                need);
  const int64_t off_item = pkv::kPlanHeaderInts;
  const int64_t off_pair = off_item + 8 * (int64_t)info->n_tile_items;
  const int64_t off_few = off_pair + info->n_tile_wide_items + 1;
  const int64_t off_merge = off_few + info->n_row_warp_items + 1;
  const int64_t off_ptr = off_merge + info->n_merge_rows;
  const int64_t off_ent = off_ptr + nb + 1;
  if (info->plan_ints < off_ent || info->plan_ints > INT32_MAX ||
      (info->plan_ints - off_ent) % 4 != 0)
    return fail(KV_ERR_INVALID_ARG, "plan info does not match the step");
  CUtensorMap tk, tv, tr, tq, tq_all;
  if (kv_status s = lat::make_latent_map(&tk, c_pool, num_blocks, lat::kKDim / 64))
    return s;
  if (kv_status s = lat::make_latent_map(&tv, c_pool, num_blocks, 8)) return s;
  if (kv_status s = lat::make_rows_map(&tr, r_pool, num_blocks * 16, rope_dim, 16))
    return s;
  const int64_t q_rows = (int64_t)nb * Hq;
  if (kv_status s = lat::make_rows_map(&tq, q, q_rows, rank + rope_dim, 16)) return s;
  if (kv_status s = lat::make_rows_map(&tq_all, q, q_rows, rank + rope_dim, 128))
    return s;
  auto* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t st = (cudaStream_t)stream;
  lat::Params p;
  p.tables = block_tables;
  p.seq_lens = seq_lens;
  p.items = reinterpret_cast<const pkv::WorkItem*>(plan + off_item);
  p.pair_ptr = plan + off_pair;
  p.few_ptr = plan + off_few;
  p.ml = reinterpret_cast<float2*>(ws + pkv::ws_ml_offset());
  p.o = reinterpret_cast<float*>(ws + pkv::ws_o_offset(info->partial_rows));
  p.out = static_cast<__nv_bfloat16*>(out);
  p.status = reinterpret_cast<pkv::DeviceStatus*>(ws);
  p.nb = nb;
  p.Hq = Hq;
  p.max_blocks = max_blocks;
  p.n_items = info->n_tile_items;
  p.n_pairs = info->n_tile_wide_items;
  p.n_few_lists = info->n_row_warp_items;
  p.num_blocks = num_blocks;
  p.partial_rows = info->partial_rows;
  p.scale_log2 = scale * 1.4426950408889634f;
  static std::atomic<uint64_t> opted{0};
  cudaError_t e = pkv::opt_in_smem(lat::latent_decode_kernel, lat::kSmem, opted);
  if (e != cudaSuccess)
    return fail(KV_ERR_CUDA, "latent step: %s", cudaGetErrorString(e));
  lat::latent_clear_kernel<<<1, 32, 0, st>>>(p.status);
  e = cudaGetLastError();
  const bool few = info->n_row_items > 0;
  const bool many = info->n_row_items < info->n_tile_items;
  p.trigger = few && many;
  if (e == cudaSuccess && many)
    e = pkv::launch_early(lat::latent_decode_kernel, 2 * p.n_pairs, lat::kThreads,
                          lat::kSmem, st, tk, tv, tr, tq, tq_all, p);
  if (e == cudaSuccess && few)
    e = pkv::launch_latent_few(tv, tr, tq, p, many, st);
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
    m.status = p.status;
    m.n = info->n_merge_rows;
    m.nb = nb;
    m.Hq = Hq;
    m.n_csr = (int)((info->plan_ints - off_ent) / 4);
    m.partial_rows = p.partial_rows;
    const int64_t warps = (int64_t)m.n * Hq;
    e = pkv::launch_early(lat::latent_merge_kernel, (int)((warps + 7) / 8), 256, 0,
                          st, m);
    if (e != cudaSuccess)
      return fail(KV_ERR_CUDA, "latent merge: %s", cudaGetErrorString(e));
  }
  return KV_OK;
}
