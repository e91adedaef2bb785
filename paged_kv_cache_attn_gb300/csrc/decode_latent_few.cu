// Decode attention over a latent pool for items of few rows (at most 16: the
// heads of one branch, or few of a segment), one SM each.
//
// With the tokens and the dimensions as the rows of the products and the item's
// rows as their 16 columns, S and O are small and the latents are the A operand
// of both:
//   S^T [64 tokens x 16] = C Q^T      (A: C, 512 + 64 wide, K-major),
//   O^T [512 x 16]      += C^T P^T    (A: the same bytes, MN-major),
// so a tile is loaded once (the kernel for many rows loads it into two SMs), and
// O^T takes 64 columns of tensor memory.  Per 64 tokens 36 products of 32 cycles
// (M = 64) and 16 of 45 (M = 128), measured: 1.0 us, against 1.65 us that HBM takes
// to bring 72 KB to every SM.  That is the bound; three stages of 64 tokens (128 KB
// of latents in flight while one is computed on, and 8 KB of position keys once S's
// products have released their stage) keep it fed.  16 contexts of 32768 tokens with
// 16 heads: 106 us with the merge, 5.7 TB/s (on pairs of SMs, as items of more rows
// run, 124); stages of 48 tokens, which leave room for two of position keys, took
// 133: the step from tile to tile costs more than the wait.
//
// Warps 0-3 rows: warp w has the tile's tokens 16 w to 16 w + 15, a lane a token
// with its 16 scores; maxima go across lanes by shuffles (each step halves the
// columns a lane keeps) and across warps through shared memory; base 2, lazy
// maximum.  P^T (bf16) goes to shared memory as the B operand.  Warps 4 and 7
// products, S(j + 1) ahead of O += P(j) C(j).  Warp 5 loads latents, warp 6 Q and
// position keys (one stage: they are the last part of S, and asked into L2 a tile
// ahead).  Slots of a last block past the branch's length are zeroed by warp 7
// before O's products (0 x NaN would not be 0).
//
// Scores of tokens past the length or the range are -inf before the maximum;
// blocks past the range are not loaded and take no part in O.  Columns past the
// item's rows hold whatever lies behind its rows of Q, and are not stored.
// Every wait is bounded, as in decode_latent.cu.

#include <cmath>

#include "latent.cuh"
#include "tensor_map.h"

namespace pkv {
namespace lat {
namespace few {

using tc::all_wait;
using tc::bar_and;
using tc::elect_one;
using tc::fence_after_sync;
using tc::fence_before_sync;
using tc::idesc;
using tc::sdesc;
using tc::tmem_wait_ld;
using tc::tmem_wait_st;
using tc::umma_commit;
using tc::umma_ss;
using tc::uniform;

constexpr int kN = kFewRows;                  // columns of the products
constexpr int kT = 64, kTB = 4;               // tokens and blocks of a tile
constexpr int kBlk = 16 * kRank * 2;          // a block's latents
constexpr int kStage = kTB * kBlk;
constexpr int kNS = 3;
constexpr int kR = kT * 128;                  // a tile's position keys
constexpr int kQPart = kN * 128;              // 64 dimensions of Q
constexpr int kQParts = (KV_LATENT_RANK + KV_LATENT_ROPE) / 64;
constexpr int kP = kN * 128;                  // P^T of a tile
constexpr int kOffR = kNS * kStage;
constexpr int kOffQ = kOffR + kR;
constexpr int kOffP = kOffQ + kQParts * kQPart;
constexpr int kTiles = kOffP + 2 * kP;
constexpr int kThreads = 8 * 32;
constexpr int kRowThreads = 128;
constexpr uint32_t kTmemCols = 128;
constexpr uint32_t kColO = 64;                // S^T at 0 and 16, O^T at 64
constexpr float kRescale = 8.f;               // lazy-max threshold (log2 units)
static_assert(kN == 16, "one 16-row box of Q, 16 scores a lane");

struct Small {
  uint64_t full[kNS], empty[kNS], r_full, r_empty, q_full, q_empty,
      s_full[2], p_full[2], pv_done, o_empty;
  float max_of[2][4][kN], sum_of[4][kN];
  uint32_t tmem_base;
  int aborted;
};
constexpr int kSmem = kTiles + (int)sizeof(Small);
static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]),
        "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]),
        "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}

// x[c] of the 16 lanes of a half warp combined over its lanes: lane i ends with
// column i & 15.
template <typename Op>
__device__ __forceinline__ float across(float (&x)[16], int lane, Op op) {
#pragma unroll
  for (int w = 8; w > 0; w >>= 1) {
    const bool up = lane & w;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < w) {
        const float give = up ? x[i] : x[i + w];
        const float keep = up ? x[i + w] : x[i];
        x[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, w));
      }
  }
  return x[0];
}

__global__ void __launch_bounds__(kThreads, 1)
    latent_few_kernel(const __grid_constant__ CUtensorMap tmC,
                      const __grid_constant__ CUtensorMap tmR,
                      const __grid_constant__ CUtensorMap tmQ, const Params p,
                      const bool beside) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  Small& sh = *reinterpret_cast<Small*>(smem + kTiles);
  volatile int* aborted = &sh.aborted;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kNS; ++s) {
      mbar_init(smem_u32(&sh.full[s]), 1);
      mbar_init(smem_u32(&sh.empty[s]), 1);
    }
    mbar_init(smem_u32(&sh.r_full), 1);
    mbar_init(smem_u32(&sh.r_empty), 1);
    mbar_init(smem_u32(&sh.q_full), 1);
    mbar_init(smem_u32(&sh.q_empty), 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&sh.s_full[b]), 1);
      mbar_init(smem_u32(&sh.p_full[b]), 4);
    }
    mbar_init(smem_u32(&sh.pv_done), 1);
    mbar_init(smem_u32(&sh.o_empty), 4);
    sh.aborted = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmC);
    tma_prefetch_desc(&tmR);
    tma_prefetch_desc(&tmQ);
  }
  __syncwarp();
  if (warp == 4) {
    asm volatile(
        "tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
            smem_u32(&sh.tmem_base)),
        "r"(kTmemCols)
        : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" :::
                     "memory");
  }
  // Behind the status word's clearing; beside the pairs' kernel that has happened.
  if (!beside) asm volatile("griddepcontrol.wait;" ::: "memory");
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = sh.tmem_base;
  ItemLoop<true> loop(p, blockIdx.x);
  WorkItem it;
  auto timed_out = [&](int site) {
    if (!*aborted) record_status(p.status, KV_ERR_TIMEOUT, site);
    atomicExch(&sh.aborted, 1);
  };
  if ((base & 1023) != 0) {  // never, with no static shared memory
    if (threadIdx.x == 0) {
      record_status(p.status, KV_ERR_INTERNAL, (int)base);
      sh.aborted = 1;
    }
    __syncthreads();
    loop.i = loop.end;
  }
  auto tiles_of = [](const WorkItem& w) {
    return (w.blk_end - w.blk_begin + kTB - 1) / kTB;
  };
  // Slots of the last block that the branch fills (16: all, nothing to zero).
  auto tail_of = [&](const WorkItem& w) {
    return w.masked ? min(16, p.seq_lens[w.branch0] - (w.blk_end - 1) * 16) : 16;
  };
  uint32_t q0 = 0, item = 0;  // tiles and items before this one

  if (warp < 4) {
    // ---- rows -------------------------------------------------------------------
    const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
    const int c = lane & 15, tok = warp * 16 + c;  // column, token of the tile
    bool ok = true;
    while (ok && loop.next(it)) {
      const int nt = tiles_of(it);
      const int seq_len = it.masked ? p.seq_lens[it.branch0] : 0x7fffffff;
      float m_used = -INFINITY;  // column c's
      float l[kN];               // this token's share of every column's sum
#pragma unroll
      for (int i = 0; i < kN; ++i) l[i] = 0.f;
      for (int j = 0; j < nt; ++j) {
        const uint32_t q = q0 + j;
        const int b = q & 1, blk0 = it.blk_begin + j * kTB;
        const int valid =
            min(min(kT, (it.blk_end - blk0) * 16), max(seq_len - blk0 * 16, 0));
        const bool w = all_wait(smem_u32(&sh.s_full[b]), (q >> 1) & 1);
        float s[kN], x[kN];
        if (w) {
          fence_after_sync();
          uint32_t u[kN];
          tmem_ld16(lanes + b * kN, u);
          tmem_wait_ld();
          const bool in = lane < 16 && tok < valid;
#pragma unroll
          for (int i = 0; i < kN; ++i)
            x[i] = s[i] = in ? __uint_as_float(u[i]) : -INFINITY;
          const float top =
              across(x, lane, [](float a, float d) { return fmaxf(a, d); });
          if (lane < kN) sh.max_of[b][warp][c] = top;
        } else {
          timed_out(70);
        }
        ok = bar_and(1, kRowThreads, w && !*aborted);
        if (!ok) break;
        const float m_tile = fmaxf(fmaxf(sh.max_of[b][0][c], sh.max_of[b][1][c]),
                                   fmaxf(sh.max_of[b][2][c], sh.max_of[b][3][c])) *
                             p.scale_log2;
        // Columns past the item's rows never ask.
        const bool need = m_tile > m_used + kRescale && c < it.nrows;
        const float alpha = need ? ex2(m_used - m_tile) : 1.f;
        if (need) m_used = m_tile;
        const float neg = m_used == -INFINITY ? 0.f : -m_used;
        const bool moved = __any_sync(0xffffffffu, need);
        if (moved) {
#pragma unroll
          for (int i = 0; i < kN; ++i) l[i] *= __shfl_sync(0xffffffffu, alpha, i);
        }
        uint16_t h[kN];
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          const float e =
              ex2(fmaf(s[i], p.scale_log2, __shfl_sync(0xffffffffu, neg, i)));
          l[i] += e;
          h[i] = __bfloat16_as_ushort(__float2bfloat16(e));
        }
        // Row i of P^T: 64 tokens, 16-byte pieces swizzled by the row.
        if (lane < 16) {
          const uint32_t prow = base + kOffP + b * kP + (tok & 7) * 2;
#pragma unroll
          for (int i = 0; i < kN; ++i)
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(
                             prow + (i >> 3) * 1024 + (i & 7) * 128 +
                             (((tok >> 3) ^ (i & 7)) << 4)),
                         "h"(h[i])
                         : "memory");
        }
        // O holds the products up to tile q - 1 once they are done.  Waited for at
        // every tile, before this one's P lets the next phase begin: a phase is
        // told by its parity alone; and P's place is free again two tiles later.
        if (q > 0 && !all_wait(smem_u32(&sh.pv_done), (q - 1) & 1)) {
          timed_out(76);  // all leave at the next tile's barrier, or the item's
        } else if (moved && j > 0) {
          fence_after_sync();
#pragma unroll 1
          for (int mt = 0; mt < 4; ++mt) {
            uint32_t v[16];
            tmem_ld16(lanes + kColO + mt * kN, v);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < kN; ++i)
              v[i] = __float_as_uint(__uint_as_float(v[i]) *
                                     __shfl_sync(0xffffffffu, alpha, i));
            tc::tmem_st16(lanes + kColO + mt * kN, v);
          }
          tmem_wait_st();
        }
        fence_proxy_async_smem();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.p_full[b]));
      }
      q0 += nt;
      // All four warps leave together.
      ok = bar_and(1, kRowThreads,
                   ok && all_wait(smem_u32(&sh.pv_done), (q0 - 1) & 1) && !*aborted);
      if (!ok) break;
      fence_after_sync();
      const float part = across(l, lane, [](float a, float d) { return a + d; });
      if (lane < kN) sh.sum_of[warp][c] = part;
      bar_and(1, kRowThreads, true);
      const float sum = (sh.sum_of[0][c] + sh.sum_of[1][c]) +
                        (sh.sum_of[2][c] + sh.sum_of[3][c]);
      const bool direct = it.g != 0;
      const float inv = 1.f / sum;
      const int64_t row0 = direct ? (int64_t)it.branch0 * p.Hq + it.row0
                                  : (int64_t)it.prow_base;
      if (!direct && warp == 0 && lane < it.nrows)
        p.ml[row0 + lane] = make_float2(m_used, sum);
      // A lane has one dimension of each 128: 64 or 128 contiguous bytes a row.
      const int64_t at = row0 * kRank + warp * 32 + lane;
#pragma unroll 1
      for (int mt = 0; mt < 4; ++mt) {
        uint32_t v[16];
        tmem_ld16(lanes + kColO + mt * kN, v);
        tmem_wait_ld();
        if (mt == 3) {  // O has been read
          fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh.o_empty));
        }
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          const float y = __uint_as_float(v[i]);
          const float scaled = y * __shfl_sync(0xffffffffu, inv, i);
          if (i < it.nrows) {
            const int64_t o = at + (int64_t)i * kRank + mt * 128;
            if (direct)
              p.out[o] = __float2bfloat16(scaled);
            else
              p.o[o] = y;
          }
        }
      }
    }
    if (!ok && lane == 0) timed_out(71);
  } else if (warp == 4) {
    // ---- S (uniform warp, one lane issues) -----------------------------------
    constexpr uint32_t id = idesc(64, kN, false);
    const bool lead = elect_one();
    bool ok = true;
    while (ok && loop.next(it)) {
      const int nt = uniform(tiles_of(it));
      ok = all_wait(smem_u32(&sh.q_full), item & 1);
      for (int j = 0; j < nt && ok; ++j) {
        const uint32_t q = q0 + j, st = q % kNS;
        const uint32_t d = tmem + (q & 1) * kN;
        const uint64_t ad = sdesc(base + st * kStage, 16, 8192);
        const uint64_t qd = sdesc(base + kOffQ, 16, 1024);
        const uint64_t rd = sdesc(base + kOffR, 16, 1024);
        // S(q - 2), which lies there, has been read.
        ok = all_wait(smem_u32(&sh.full[st]), (q / kNS) & 1) &&
             (q < 2 || all_wait(smem_u32(&sh.p_full[q & 1]), ((q >> 1) - 1) & 1));
        if (!ok) break;
        fence_after_sync();
        if (lead) {
#pragma unroll
          for (int k = 0; k < kRank / 16; ++k)
            umma_ss(d, ad + (((k >> 2) * 1024 + (k & 3) * 32) >> 4),
                    qd + (((k >> 2) * kQPart + (k & 3) * 32) >> 4), id,
                    k > 0 ? 1u : 0u);
        }
        __syncwarp();
        ok = all_wait(smem_u32(&sh.r_full), q & 1);
        if (!ok) break;
        fence_after_sync();
        if (lead) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_ss(d, rd + k * 2, qd + (((kQParts - 1) * kQPart) >> 4) + k * 2, id,
                    1u);
          umma_commit(smem_u32(&sh.s_full[q & 1]));
          umma_commit(smem_u32(&sh.r_empty));
          if (j == nt - 1) umma_commit(smem_u32(&sh.q_empty));
        }
        __syncwarp();
        ok = __all_sync(0xffffffffu, !*aborted);
      }
      q0 += nt;
      ++item;
    }
    if (!ok && lead) timed_out(72);
  } else if (warp == 7) {
    // ---- O (another warp: the waits of one lie behind the other's products) ---
    constexpr uint32_t id = idesc(128, kN, false) | (1u << 15);  // A MN-major
    const bool lead = elect_one();
    bool ok = true;
    while (ok && loop.next(it)) {
      const int nt = uniform(tiles_of(it));
      const int blocks = uniform(it.blk_end - it.blk_begin);
      const int tail = max(uniform(tail_of(it)), 0);
      for (int j = 0; j < nt && ok; ++j) {
        const uint32_t q = q0 + j, st = q % kNS;
        const int nb = min(kTB, blocks - j * kTB);
        ok = all_wait(smem_u32(&sh.full[st]), (q / kNS) & 1);
        if (ok && j == nt - 1 && tail < 16) {
          const uint32_t dst = base + st * kStage + (nb - 1) * kBlk;
          for (int x = lane; x < (16 - tail) * 64; x += 32) {
            const int row = tail + (x >> 6), k = x & 63;
            st_shared_zero16(dst + (row >> 3) * 8192 + (k >> 3) * 1024 +
                             (row & 7) * 128 + (k & 7) * 16);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        ok = ok && (j > 0 || item == 0 ||
                    all_wait(smem_u32(&sh.o_empty), (item - 1) & 1)) &&
             all_wait(smem_u32(&sh.p_full[q & 1]), (q >> 1) & 1);
        if (!ok) break;
        fence_after_sync();
        const uint64_t pd = sdesc(base + kOffP + (q & 1) * kP, 16, 1024);
        if (lead) {
#pragma unroll
          for (int k = 0; k < kTB; ++k)
            if (k < nb) {
              const uint64_t cd = sdesc(base + st * kStage + k * kBlk, 1024, 8192);
#pragma unroll
              for (int mt = 0; mt < 4; ++mt)
                umma_ss(tmem + kColO + mt * kN, cd + mt * (2048 >> 4), pd + k * 2, id,
                        j > 0 || k > 0 ? 1u : 0u);
            }
          umma_commit(smem_u32(&sh.pv_done));
          umma_commit(smem_u32(&sh.empty[st]));
        }
        __syncwarp();
        ok = __all_sync(0xffffffffu, !*aborted);
      }
      q0 += nt;
      ++item;
    }
    if (!ok && lead) timed_out(77);
  } else if (warp == 5) {
    // ---- latents -----------------------------------------------------------------
    bool ok = true;
    while (ok && loop.next(it)) {
      const int nt = tiles_of(it);
      bool bad = false, next_bad = false;
      int next = lane < kTB ? block_of(p, it, it.blk_begin + lane, next_bad) : -1;
      for (int j = 0; j < nt; ++j) {
        const uint32_t q = q0 + j, st = q % kNS, bar = smem_u32(&sh.full[st]);
        const int phys = next, blk = it.blk_begin + j * kTB + lane;
        bad = next_bad;
        next_bad = false;
        next = lane < kTB && j + 1 < nt ? block_of(p, it, blk + kTB, next_bad) : -1;
        if (bad)
          record_status(p.status, KV_ERR_DEVICE,
                        p.tables[(int64_t)it.branch0 * p.max_blocks + blk]);
        const int n = __popc(__ballot_sync(0xffffffffu, phys >= 0));
        if (q >= kNS) ok = all_wait(smem_u32(&sh.empty[st]), (q / kNS - 1) & 1);
        ok = __all_sync(0xffffffffu, ok && !*aborted);
        if (!ok) break;
        if (lane == 0) mbar_expect_tx(bar, n * kBlk);
        __syncwarp();
        if (phys >= 0)
          tc::tma_load_5d_at(base + st * kStage + lane * kBlk, &tmC, 0, phys, bar);
        __syncwarp();
      }
      q0 += nt;
    }
    if (!ok && lane == 0) timed_out(73);
  } else {
    // ---- Q and position keys ---------------------------------------------------
    bool ok = true;
    while (ok && loop.next(it)) {
      const int nt = tiles_of(it);
      bool bad;
      int next = lane < kTB ? block_of(p, it, it.blk_begin + lane, bad) : -1;
      if (item > 0) ok = all_wait(smem_u32(&sh.q_empty), (item - 1) & 1);
      ok = __all_sync(0xffffffffu, ok && !*aborted);
      if (!ok) break;
      if (lane == 0) mbar_expect_tx(smem_u32(&sh.q_full), kQParts * kQPart);
      __syncwarp();
      if (lane < kQParts)
        tma_load_2d(base + kOffQ + lane * kQPart, &tmQ, lane * 64,
                    it.branch0 * p.Hq + it.row0, smem_u32(&sh.q_full));
      __syncwarp();
      for (int j = 0; j < nt; ++j) {
        const uint32_t q = q0 + j;
        const int phys = next;
        next = lane < kTB && j + 1 < nt
                   ? block_of(p, it, it.blk_begin + (j + 1) * kTB + lane, bad)
                   : -1;
        const int n = __popc(__ballot_sync(0xffffffffu, phys >= 0));
        if (q > 0) ok = all_wait(smem_u32(&sh.r_empty), (q - 1) & 1);
        ok = __all_sync(0xffffffffu, ok && !*aborted);
        if (!ok) break;
        if (lane == 0) mbar_expect_tx(smem_u32(&sh.r_full), n * 2048);
        __syncwarp();
        if (phys >= 0)
          tma_load_2d(base + kOffR + lane * 2048, &tmR, 0, phys * 16,
                      smem_u32(&sh.r_full));
        if (next >= 0) tc::l2_prefetch_2d(&tmR, 0, next * 16);
        __syncwarp();
      }
      q0 += nt;
      ++item;
    }
    if (!ok && lane == 0) timed_out(74);
    if (lane == 0) report_bad<true>(p, blockIdx.x);
  }
  __syncwarp();
  fence_before_sync();
  __syncthreads();
  // After a time-out loads may be in flight (else a product has waited for every
  // one): about two milliseconds for them to land.
  if (*aborted) {
    const long long t0 = clock64();
    while (clock64() - t0 < (1 << 22)) {
    }
  }
  fence_after_sync();
  if (warp == 4)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols)
                 : "memory");
  // The pairs' kernel is complete when this one is.
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace few
}  // namespace lat

cudaError_t launch_latent_few(const CUtensorMap& tmC, const CUtensorMap& tmR,
                              const CUtensorMap& tmQ, const lat::Params& p,
                              bool beside, cudaStream_t st) {
  static std::atomic<uint64_t> opted{0};
  const cudaError_t e =
      opt_in_smem(lat::few::latent_few_kernel, lat::few::kSmem, opted);
  if (e != cudaSuccess) return e;
  return launch_early(lat::few::latent_few_kernel, p.n_few_lists,
                      lat::few::kThreads, lat::few::kSmem, st, tmC, tmR, tmQ, p,
                      beside);
}

}  // namespace pkv
