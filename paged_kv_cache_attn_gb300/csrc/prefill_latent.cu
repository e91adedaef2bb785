// Latent prefill, expanded form (paged_latent_prefill_attn): new tokens attend
// causally to all cached tokens of their branch, with keys and values expanded
// from the latents per head,
//   k[t][h] = [Wk_h c_t ; r_t] (128 + 64),  v[t][h] = Wv_h c_t (128),
//   out[i][h] = sum_{t <= pos(i)} softmax_t(scale q[i][h] . k[t][h]) v[t][h].
// Against the absorbed form this costs 2 x 320 flops a row and token instead of
// 2 x 1088, for 2 x 512 x 256 flops a token and head once.
//
// Expansion kernel: [128 tokens x 512] x [512 x 256] per token tile and head
// (the tokens are eight distinct blocks of the step, gathered through the
// plan's list; a block shared by branches is expanded once), written as bf16 to
// [slot][head][16][128] -- the rounding of a cached key or value.  Operands
// stream through a ring of 64-dimension stages (16 + 32 KB), products in two
// 256-column halves of TMEM so that a tile's epilogue overlaps the next one's
// products.  Bound by what L2 delivers to an SM (48 KB per four MMAs of 128
// cycles).
//
// Attention kernel: one CTA per tile of 256 query rows (two M-tiles of 128)
// and head.  TMEM: S of the two M-tiles (2 x 128 columns; P overwrites its S as
// bf16 pairs) and O (2 x 128).  Q in shared memory (96 KB), K in two stages of
// 128 tokens (128 expanded dimensions and the 64 shared position dimensions),
// V in one.  One product warp per M-tile runs PV(j - 1) and then QK(j); when
// S(j) is complete so is everything before it, so the rows may overwrite P and
// rescale O without another wait.  The softmax of one M-tile (a thread a row,
// base 2, lazy maximum) lies behind the other M-tile's products.  Bound by the
// chain of an M-tile, QK -> softmax -> PV.
//
// Tokens past a row's position are replaced by -inf before the maximum; values
// of slots past a branch's length are written as zeros by the expansion, and
// blocks past the tile's range take no part in PV.

#include <cmath>
#include <cstring>

#include "cluster.cuh"
#include "tensor_map.h"

namespace pkv {
namespace pre {

using tc::all_wait;
using tc::elect_one;
using tc::fence_after_sync;
using tc::fence_before_sync;
using tc::idesc;
using tc::sdesc;
using tc::tma_load_5d_at;
using tc::tmem_ld32;
using tc::tmem_st32;
using tc::tmem_wait_ld;
using tc::tmem_wait_st;
using tc::umma_commit;
using tc::umma_ss;
using tc::umma_ts;
using tc::uniform;
using tc::warp_wait;

constexpr int kRank = KV_LATENT_RANK, kRope = KV_LATENT_ROPE, kHead = KV_LATENT_HEAD;
constexpr uint32_t kTmemCols = 512;

struct Params {
  const int32_t* uniq;    // distinct blocks
  const int32_t* valid;   // their valid tokens
  const int32_t* slots;   // branches' tables, indices into uniq
  const PrefillTile* tiles;
  __nv_bfloat16* k_exp;   // [slot][Hq][16][128]
  __nv_bfloat16* v_exp;
  __nv_bfloat16* out;     // [total][Hq][128]
  DeviceStatus* status;
  int n_uniq, n_slots, n_tiles, Hq, total;
  int64_t num_blocks;
  float scale_log2;
};

__device__ __forceinline__ void tmem_alloc(uint32_t where) {
  asm volatile(
      "tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
          where),
      "r"(kTmemCols)
      : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" :::
                   "memory");
}

__device__ __forceinline__ void tmem_free(uint32_t tmem) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
               "r"(kTmemCols)
               : "memory");
}

// 32 rows x 64 bytes of a warp (lane = row, w = its 16 words) out to dst(row)
// through 2 KB of shared memory, 16-byte pieces swizzled by the row: a store
// covers whole sectors of eight rows.
template <typename Dst>
__device__ __forceinline__ void put_rows(uint8_t* turn, const uint32_t (&w)[16],
                                         int lane, Dst dst) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<uint4*>(turn + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4)) =
        make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int rr = k * 8 + (lane >> 2), c = lane & 3;
    const uint4 x = *reinterpret_cast<const uint4*>(
        turn + rr * 64 + ((c ^ ((rr >> 1) & 3)) << 4));
    if (uint8_t* d = dst(rr)) *reinterpret_cast<uint4*>(d + c * 16) = x;
  }
  __syncwarp();
}

// ---- expansion ------------------------------------------------------------------

namespace ex {

constexpr int kA = 128 * 128, kB = 256 * 128;   // a stage of X and of W
constexpr int kStage = kA + kB;
constexpr int kNS = 4;
constexpr int kChunks = kRank / 64;
constexpr int kOffTurn = kNS * kStage;
constexpr int kTiles = kOffTurn + 8 * 2048;
constexpr int kThreads = 11 * 32;  // warps 0-7 rows, 8 products, 9-10 loads

struct Small {
  uint64_t full[kNS], empty[kNS], d_full[2], d_empty[2], drain;
  uint32_t tmem_base;
  int aborted;
};
constexpr int kSmem = kTiles + (int)sizeof(Small) + 1024;
static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");

__global__ void __launch_bounds__(kThreads, 1)
    expand_kernel(const __grid_constant__ CUtensorMap tmX,
                  const __grid_constant__ CUtensorMap tmW, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - smem_u32(smem_raw));
  Small& sh = *reinterpret_cast<Small*>(smem + kTiles);
  volatile int* aborted = &sh.aborted;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kNS; ++s) {
      mbar_init(smem_u32(&sh.full[s]), 1);
      mbar_init(smem_u32(&sh.empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&sh.d_full[b]), 1);
      mbar_init(smem_u32(&sh.d_empty[b]), 8);
    }
    mbar_init(smem_u32(&sh.drain), 1);
    sh.aborted = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmW);
  }
  if (warp == 8) tmem_alloc(smem_u32(&sh.tmem_base));
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = sh.tmem_base;
  // Tiles of eight slots, heads innermost: a tile's latents stay in L2 while
  // its heads pass, and the weights of all heads do throughout.
  const int n_work = (p.n_uniq + 7) / 8 * p.Hq;
  auto timed_out = [&](int site) {
    if (!*aborted) record_status(p.status, KV_ERR_TIMEOUT, site);
    atomicExch(&sh.aborted, 1);
  };

  if (warp < 8) {
    const int wg = warp >> 2;  // 0: keys, 1: values
    const int r = (warp & 3) * 32 + lane;
    const uint32_t drow =
        tmem + ((uint32_t)((warp & 3) * 32) << 16) + wg * kHead;
    uint8_t* turn = smem + kOffTurn + warp * 2048;
    __nv_bfloat16* exp = wg == 0 ? p.k_exp : p.v_exp;
    uint32_t n = 0;
    bool ok = true;
    for (int i = blockIdx.x; i < n_work; i += gridDim.x, ++n) {
      const int slot0 = i / p.Hq * 8, h = i % p.Hq;
      const uint32_t b = n & 1;
      ok = warp_wait(smem_u32(&sh.d_full[b]), (n >> 1) & 1, lane) && !*aborted;
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      fence_after_sync();
      const int slot = slot0 + (r >> 4);
      // Values past the branch's length would meet weights of zero: zeros.
      const bool zero =
          wg == 1 && (slot >= p.n_uniq || (r & 15) >= p.valid[min(slot, p.n_uniq - 1)]);
      const int row0 = (warp & 3) * 32;
#pragma unroll 1
      for (int c = 0; c < kHead; c += 32) {
        uint32_t v[32], w[16];
        tmem_ld32(drow + b * 256 + c, v);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 16; ++k)
          w[k] = zero ? 0u
                      : pack_bf16(__uint_as_float(v[2 * k]),
                                  __uint_as_float(v[2 * k + 1]));
        put_rows(turn, w, lane, [&](int rr) -> uint8_t* {
          const int row = row0 + rr, s = slot0 + (row >> 4);
          if (s >= p.n_uniq) return nullptr;
          return reinterpret_cast<uint8_t*>(
              exp + (((int64_t)s * p.Hq + h) * 16 + (row & 15)) * kHead + c);
        });
      }
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.d_empty[b]));
    }
    if (!ok && lane == 0) timed_out(50);
  } else if (warp == 8) {
    constexpr uint32_t id = idesc(128, 256, false);
    const bool lead = elect_one();
    uint32_t n = 0, s = 0, ph = 0;
    bool ok = true;
    const int work = uniform(n_work);
    for (int i = blockIdx.x; i < work && ok; i += gridDim.x, ++n) {
      const uint32_t b = n & 1, d = tmem + b * 256;
      if (n >= 2) ok = all_wait(smem_u32(&sh.d_empty[b]), ((n >> 1) - 1) & 1);
      for (int c = 0; c < kChunks && ok; ++c) {
        ok = all_wait(smem_u32(&sh.full[s]), ph);
        if (!ok) break;
        fence_after_sync();
        const uint64_t ad = sdesc(base + s * kStage, 16, 1024);
        const uint64_t bd = sdesc(base + s * kStage + kA, 16, 1024);
        if (lead) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_ss(d, ad + k * 2, bd + k * 2, id, c > 0 || k > 0 ? 1u : 0u);
          umma_commit(smem_u32(&sh.empty[s]));
          if (c == kChunks - 1) umma_commit(smem_u32(&sh.d_full[b]));
        }
        __syncwarp();
        if (++s == kNS) {
          s = 0;
          ph ^= 1;
        }
      }
      ok = ok && !*aborted;
    }
    if (lead) {
      if (!ok) timed_out(51);
      umma_commit(smem_u32(&sh.drain));
      mbar_wait(smem_u32(&sh.drain), 0);
    }
  } else {
    // Stages alternate between the two warps: eight boxes of a block and one of
    // the head's weights.
    const uint32_t me = warp - 9;
    uint32_t k = 0;
    bool ok = true;
    for (int i = blockIdx.x; i < n_work && ok; i += gridDim.x) {
      const int slot = i / p.Hq * 8 + lane, h = i % p.Hq;
      int phys = lane < 8 && slot < p.n_uniq ? p.uniq[slot] : -1;
      if (lane < 8 && slot < p.n_uniq && (phys < 0 || phys >= p.num_blocks)) {
        if (me == 0) record_status(p.status, KV_ERR_DEVICE, phys);
        phys = -1;
      }
      const int nb = __popc(__ballot_sync(0xffffffffu, phys >= 0));
      for (int c = 0; c < kChunks; ++c, ++k) {
        if ((k & 1) != me) continue;
        const uint32_t s = k % kNS, bar = smem_u32(&sh.full[s]);
        if (lane == 0) {
          ok = !*aborted && (k < kNS || mbar_wait(smem_u32(&sh.empty[s]),
                                                  (k / kNS - 1) & 1));
          if (ok) mbar_expect_tx(bar, nb * 2048 + kB);
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        if (phys >= 0)
          tma_load_2d(base + s * kStage + lane * 2048, &tmX, c * 64, phys * 16, bar);
        else if (lane == 8)
          tma_load_2d(base + s * kStage + kA, &tmW, c * 64, h * 256, bar);
        __syncwarp();
      }
    }
    if (lane == 0) {
      if (!ok) timed_out(52);
      for (uint32_t j = k > kNS ? k - kNS : 0; j < k; ++j)
        if ((j & 1) == me && !mbar_wait(smem_u32(&sh.full[j % kNS]), (j / kNS) & 1))
          break;
    }
  }
  __syncwarp();
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (warp == 8) tmem_free(tmem);
}

}  // namespace ex

// ---- attention ------------------------------------------------------------------

namespace at {

constexpr int kT = 128, kTB = 8;             // tokens and blocks of a key tile
constexpr int kQ = 3 * 128 * 128;            // Q of an M-tile: three 64-wide parts
constexpr int kBlk = 16 * kHead * 2;         // a block's expanded keys of a head
constexpr int kKn = kTB * kBlk;              // a K stage: expanded part,
constexpr int kK = kKn + kT * 128;           // and position part
constexpr int kV = kTB * kBlk;
constexpr int kOffK = 2 * kQ;
constexpr int kOffV = kOffK + 2 * kK;
constexpr int kTiles = kOffV + kV;
constexpr int kThreads = 12 * 32;  // warps 0-7 rows, 8 and 11 products, 9-10 loads
constexpr uint32_t kColO = 256;
constexpr float kRescale = 8.f;    // lazy-max threshold (log2 units)

struct Small {
  uint64_t q_full, k_full[2], k_empty[2], v_full, v_empty, s_full[2], p_full[2],
      o_ready[2], turn[2];
  uint32_t tmem_base;
  int aborted;
};
constexpr int kSmem = kTiles + (int)sizeof(Small);
static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");

__global__ void __launch_bounds__(kThreads, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap tmQ,
                   const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV,
                   const __grid_constant__ CUtensorMap tmR, const Params p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  Small& sh = *reinterpret_cast<Small*>(smem + kTiles);
  volatile int* aborted = &sh.aborted;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (base & 1023) {  // never, with no static shared memory
    if (threadIdx.x == 0) record_status(p.status, KV_ERR_INTERNAL, (int)base);
    return;
  }
  // Launched while the expansion runs: nothing of global memory before this.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int h = blockIdx.x / p.n_tiles;
  PrefillTile t = p.tiles[blockIdx.x % p.n_tiles];
  const int len = t.pos0 + t.nrows;  // tokens the tile's last row sees
  const int nblk = (len + 15) / 16;
  if (t.nrows < 1 || t.nrows > kPrefillRows || t.pos0 < 0 || t.row0 < 0 ||
      t.row0 + t.nrows > p.total || t.table < 0 || t.table + nblk > p.n_slots) {
    if (threadIdx.x == 0)
      record_status(p.status, KV_ERR_DEVICE, -1 - (int)blockIdx.x);
    return;  // the whole CTA, before any barrier
  }
  const int n_m = t.nrows > 128 ? 2 : 1;
  // Key tiles of M-tile m: up to its last row's position.
  auto tiles_of = [&](int m) {
    return (t.pos0 + min(t.nrows, 128 * (m + 1)) - 1) / kT + 1;
  };
  const int nt = tiles_of(n_m - 1);

  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&sh.q_full), 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&sh.k_full[s]), 1);
      mbar_init(smem_u32(&sh.k_empty[s]), n_m);
      mbar_init(smem_u32(&sh.s_full[s]), 1);
      mbar_init(smem_u32(&sh.p_full[s]), 4);
      mbar_init(smem_u32(&sh.o_ready[s]), 1);
      mbar_init(smem_u32(&sh.turn[s]), 1);
    }
    mbar_init(smem_u32(&sh.v_full), 1);
    mbar_init(smem_u32(&sh.v_empty), n_m);
    sh.aborted = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    tma_prefetch_desc(&tmR);
  }
  if (warp == 8) tmem_alloc(smem_u32(&sh.tmem_base));
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = sh.tmem_base;
  auto timed_out = [&](int site) {
    if (!*aborted) record_status(p.status, KV_ERR_TIMEOUT, site);
    atomicExch(&sh.aborted, 1);
  };

  if (warp < 8) {
    // ---- rows: thread = row r of M-tile m ------------------------------------
    const int m = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    if (m < n_m) {
      const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
      const uint32_t srow = lane_base + m * kT;
      const uint32_t orow = lane_base + kColO + m * kHead;
      const int pos = t.pos0 + m * 128 + r;     // this row's position
      const int pos_lo = t.pos0 + m * 128 + (warp & 3) * 32;  // the warp's first
      const int my_nt = tiles_of(m);
      float m_used = -INFINITY, l = 0.f;
      bool ok = true;
      for (int j = 0; j < my_nt; ++j) {
        ok = warp_wait(smem_u32(&sh.s_full[m]), j & 1, lane);
        if (!ok) break;
        fence_after_sync();
        uint32_t u[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(srow + c * 32, u[c]);
        tmem_wait_ld();
        const int seen = pos - j * kT + 1;      // tokens of the tile this row sees
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        if (pos_lo - j * kT + 1 >= kT) {        // every row of the warp: all
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              m4[i & 3] = fmaxf(m4[i & 3], __uint_as_float(u[c][i]));
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              if (c * 32 + i >= seen) u[c][i] = 0xff800000u;  // -inf
              m4[i & 3] = fmaxf(m4[i & 3], __uint_as_float(u[c][i]));
            }
        }
        const float m_tile =
            fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * p.scale_log2;
        const bool need = m_tile > m_used + kRescale;
        const float alpha = need ? ex2(m_used - m_tile) : 1.f;
        if (need) m_used = m_tile;
        l *= alpha;
        const float neg_m = m_used == -INFINITY ? 0.f : -m_used;
        float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          uint32_t pk[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int c = g * 2 + (i >> 4), k = (2 * i) & 31;
            const float a = ex2(fmaf(__uint_as_float(u[c][k]), p.scale_log2, neg_m));
            const float b =
                ex2(fmaf(__uint_as_float(u[c][k + 1]), p.scale_log2, neg_m));
            s4[i & 3] += a + b;
            pk[i] = pack_bf16(a, b);
          }
          tmem_st32(srow + g * 32, pk);
        }
        l += (s4[0] + s4[1]) + (s4[2] + s4[3]);
        // O holds the products up to tile j - 1, all of them done.
        if (__any_sync(0xffffffffu, need) && j > 0) tc::rescale_o_row(orow, alpha);
        tmem_wait_st();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.p_full[m]));
      }
      if (!ok && lane == 0) timed_out(60);
      ok = warp_wait(smem_u32(&sh.o_ready[m]), 0, lane) && ok && !*aborted;
      ok = __all_sync(0xffffffffu, ok);
      fence_after_sync();
      if (ok) {
        const float inv = 1.f / l;
        // The M-tile's Q has been read: its place turns the rows.
        uint8_t* turn = smem + m * kQ + (warp & 3) * 2048;
        const int n = t.nrows - m * 128 - (warp & 3) * 32;  // rows of the warp
        const int64_t row0 = t.row0 + m * 128 + (warp & 3) * 32;
#pragma unroll 1
        for (int c = 0; c < kHead; c += 32) {
          uint32_t v[32], w[16];
          tmem_ld32(orow + c, v);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 16; ++k)
            w[k] = pack_bf16(__uint_as_float(v[2 * k]) * inv,
                             __uint_as_float(v[2 * k + 1]) * inv);
          put_rows(turn, w, lane, [&](int rr) -> uint8_t* {
            if (rr >= n) return nullptr;
            return reinterpret_cast<uint8_t*>(
                p.out + ((row0 + rr) * p.Hq + h) * kHead + c);
          });
        }
      }
    }
  } else if (warp == 8 || warp == 11) {
    // ---- products of one M-tile (uniform warp, one lane issues) ---------------
    const int m = warp == 8 ? 0 : 1;
    if (m < n_m) {
      constexpr uint32_t id_qk = idesc(128, kT, false);
      constexpr uint32_t id_pv = idesc(128, kHead, true);
      const bool lead = elect_one();
      const int all = uniform(nt), mine = uniform(tiles_of(m));
      const int blocks = uniform(nblk);
      const uint32_t ds = tmem + m * kT, dout = tmem + kColO + m * kHead;
      bool ok = all_wait(smem_u32(&sh.q_full), 0);
      // PV(j) needs P and V; where the M-tile is past its last key tile, the
      // tile is only released.
      auto pv_ready = [&](int j) {
        if (j < mine && !all_wait(smem_u32(&sh.p_full[m]), j & 1)) return false;
        return all_wait(smem_u32(&sh.v_full), j & 1);
      };
      auto pv = [&](int j) {  // one lane: O += P(j) V(j)
        if (j < mine) {
          const int nb = min(kTB, blocks - j * kTB);
#pragma unroll
          for (int k = 0; k < kTB; ++k)
            if (k < nb)
              umma_ts(dout, ds + k * 8, sdesc(base + kOffV + k * kBlk, 1024, 2048),
                      id_pv, j > 0 || k > 0 ? 1u : 0u);
          umma_commit(smem_u32(&sh.v_empty));
          if (j == mine - 1) umma_commit(smem_u32(&sh.o_ready[m]));
        } else {
          mbar_arrive(smem_u32(&sh.v_empty));
        }
      };
      for (int j = 0; j < all && ok; ++j) {
        if (j > 0) ok = pv_ready(j - 1);
        ok = ok && all_wait(smem_u32(&sh.k_full[j & 1]), (j >> 1) & 1);
        // The M-tiles' products alternate in whole blocks: issued side by side
        // they would interleave, both softmaxes would start when both were done,
        // and the tensor pipe would idle meanwhile (2.6 us a key tile instead of
        // 1.9).
        if (n_m == 2 && (m == 1 || j > 0))
          ok = ok && all_wait(smem_u32(&sh.turn[m]), (m == 1 ? j : j - 1) & 1);
        if (!ok) break;
        fence_after_sync();
        const uint32_t kst = base + kOffK + (j & 1) * kK;
        if (lead) {
          if (j > 0) pv(j - 1);
          if (j < mine) {
            const uint64_t qd = sdesc(base + m * kQ, 16, 1024);
            const uint64_t kd = sdesc(kst, 16, 2048);
            const uint64_t rd = sdesc(kst + kKn, 16, 1024);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              umma_ss(ds, qd + (((k >> 2) * 16384 + (k & 3) * 32) >> 4),
                      kd + (((k >> 2) * 1024 + (k & 3) * 32) >> 4), id_qk,
                      k > 0 ? 1u : 0u);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_ss(ds, qd + ((2 * 16384 + k * 32) >> 4), rd + k * 2, id_qk, 1u);
            umma_commit(smem_u32(&sh.k_empty[j & 1]));
            umma_commit(smem_u32(&sh.s_full[m]));
          } else {
            mbar_arrive(smem_u32(&sh.k_empty[j & 1]));
          }
          if (n_m == 2) mbar_arrive(smem_u32(&sh.turn[m ^ 1]));
        }
        __syncwarp();
        ok = !*aborted;
      }
      if (ok) ok = pv_ready(all - 1);
      if (ok) {
        fence_after_sync();
        if (lead) pv(all - 1);
      }
      if (lead) {
        if (!ok) {
          timed_out(61);
          umma_commit(smem_u32(&sh.o_ready[m]));  // let the rows end
        }
        // Every product this warp issued has finished once this lands.
        if (!ok) mbar_wait(smem_u32(&sh.o_ready[m]), 0);
      }
    }
  } else {
    // ---- loads: warp 9 Q and K, warp 10 V ---------------------------------------
    const bool is_v = warp == 10;
    bool ok = true;
    // The expansion's stores, read by bulk copies from here on.
    asm volatile("fence.proxy.async;" ::: "memory");
    if (!is_v) {
      if (lane == 0) mbar_expect_tx(smem_u32(&sh.q_full), n_m * kQ);
      __syncwarp();
      if (lane < 3 * n_m)
        tc::tma_load_3d(base + (lane / 3) * kQ + (lane % 3) * 16384, &tmQ,
                        (lane % 3) * 64, h, t.row0 + (lane / 3) * 128,
                        smem_u32(&sh.q_full));
      __syncwarp();
    }
    auto slot_of = [&](int blk) {
      if (blk >= nblk) return -1;
      const int s = p.slots[t.table + blk];
      if (s >= 0 && s < p.n_uniq) return s;
      if (!is_v && lane < 8) record_status(p.status, KV_ERR_DEVICE, s);
      return -1;
    };
    // K: lanes 0-7 the blocks' expanded keys, lanes 8-15 their position keys.
    const int bi = lane & 7;
    const bool part = lane < (is_v ? 8 : 16);
    int next = part ? slot_of(bi) : -1;
    int next_phys = !is_v && lane >= 8 && next >= 0 ? p.uniq[next] : -1;
    int j = 0;
    for (; j < nt; ++j) {
      const int slot = next, phys = next_phys;
      next = part && j + 1 < nt ? slot_of((j + 1) * kTB + bi) : -1;
      next_phys = !is_v && lane >= 8 && next >= 0 ? p.uniq[next] : -1;
      const bool pos_ok = phys >= 0 && phys < p.num_blocks;
      const bool load = slot >= 0 && (is_v || lane < 8 || pos_ok);
      const uint32_t act = __ballot_sync(0xffffffffu, load);
      const uint32_t bar =
          is_v ? smem_u32(&sh.v_full) : smem_u32(&sh.k_full[j & 1]);
      if (lane == 0) {
        if (is_v)
          ok = j == 0 || mbar_wait(smem_u32(&sh.v_empty), (j - 1) & 1);
        else
          ok = j < 2 || mbar_wait(smem_u32(&sh.k_empty[j & 1]), ((j >> 1) - 1) & 1);
        ok = ok && !*aborted;
        const uint32_t bytes = __popc(act & 0xff) * kBlk + __popc(act >> 8) * 2048;
        if (ok) {
          if (bytes > 0)
            mbar_expect_tx(bar, bytes);
          else
            mbar_arrive(bar);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      if (load) {
        if (is_v)
          tc::tma_load_5d(base + kOffV + bi * kBlk, &tmV, slot * p.Hq + h, bar);
        else if (lane < 8)
          tc::tma_load_5d(base + kOffK + (j & 1) * kK + bi * kBlk, &tmK,
                          slot * p.Hq + h, bar);
        else
          tma_load_2d(base + kOffK + (j & 1) * kK + kKn + bi * 2048, &tmR, 0,
                      phys * 16, bar);
      }
      __syncwarp();
    }
    if (lane == 0) {
      if (!ok) timed_out(is_v ? 63 : 62);
      // Loads in flight land before the CTA can leave.
      if (is_v) {
        if (j > 0) mbar_wait(smem_u32(&sh.v_full), (j - 1) & 1);
      } else {
        mbar_wait(smem_u32(&sh.q_full), 0);
        for (int k = j > 2 ? j - 2 : 0; k < j; ++k)
          mbar_wait(smem_u32(&sh.k_full[k & 1]), (k >> 1) & 1);
      }
    }
  }
  __syncwarp();
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (warp == 8) tmem_free(tmem);
}

}  // namespace at

// ---- host side ------------------------------------------------------------------

// Expanded keys or values, [slot][Hq][16][128] bf16: a box is a (slot, head)
// tile of 4 KB, landing as four 1 KB atoms of 8 rows x 64 columns ordered (rows
// 0-7, half 0), (0-7, 1), (8-15, 0), (8-15, 1).
kv_status make_expanded_map(CUtensorMap* tm, const void* base, int64_t tiles) {
  const cuuint64_t dims[5] = {64, 8, 2, 2, (cuuint64_t)tiles};
  const cuuint64_t strides[4] = {256, 128, 2048, 4096};
  const cuuint32_t box[5] = {64, 8, 2, 2, 1};
  return encode_bf16_map(tm, base, 5, dims, strides, box);
}

kv_status make_matrix_map(CUtensorMap* tm, const void* base, int64_t rows,
                          int width, int box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)width * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  return encode_bf16_map(tm, base, 2, dims, strides, box);
}

// Queries [total][Hq][192]: boxes of 128 tokens x one head x 64 values.
kv_status make_query_map(CUtensorMap* tm, const void* q, int64_t total, int Hq) {
  const int w = kHead + kRope;
  const cuuint64_t dims[3] = {(cuuint64_t)w, (cuuint64_t)Hq, (cuuint64_t)total};
  const cuuint64_t strides[2] = {(cuuint64_t)w * 2, (cuuint64_t)w * 2 * Hq};
  const cuuint32_t box[3] = {64, 1, 128};
  return encode_bf16_map(tm, q, 3, dims, strides, box);
}

__global__ void clear_kernel(DeviceStatus* status) {
  if (threadIdx.x == 0) *status = DeviceStatus{};
}

}  // namespace pre
}  // namespace pkv

using pkv::fail;

extern "C" kv_status paged_latent_prefill_attn(
    const void* q, const void* c_pool, const void* r_pool, int64_t num_blocks,
    const void* w_kv, int32_t total, int32_t nb, int32_t Hq, int32_t rank,
    int32_t rope_dim, int32_t head_dim, int32_t block_size, float scale,
    void* out, const int32_t* plan, const kv_decode_plan_info* info,
    void* workspace, size_t ws_bytes, void* stream) {
  namespace pre = pkv::pre;
  pkv::clear_error();
  if (!info || !plan || !workspace || !c_pool || !r_pool || !w_kv || !q || !out)
    return fail(KV_ERR_INVALID_ARG, "null argument");
  if (rank != KV_LATENT_RANK || rope_dim != KV_LATENT_ROPE ||
      head_dim != KV_LATENT_HEAD)
    return fail(KV_ERR_INVALID_ARG, "a latent cache has rank 512, rope_dim 64 and "
                "heads of 128, got %d, %d and %d", rank, rope_dim, head_dim);
  if (nb < 1 || Hq < 1 || Hq > 65535 || total < 0)
    return fail(KV_ERR_INVALID_ARG, "bad nb/Hq/total");
  if (block_size != 16) return fail(KV_ERR_INVALID_ARG, "block_size must be 16");
  if (num_blocks < 1 || num_blocks > (int64_t)INT32_MAX / 16)
    return fail(KV_ERR_INVALID_ARG, "num_blocks out of range");
  if (((uintptr_t)q | (uintptr_t)c_pool | (uintptr_t)r_pool | (uintptr_t)w_kv |
       (uintptr_t)out) & 15)
    return fail(KV_ERR_INVALID_ARG, "q, pools, w_kv and out must be 16-byte aligned");
  if ((uintptr_t)workspace & 255)
    return fail(KV_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if (!std::isfinite(scale) || !(scale > 0.f))
    return fail(KV_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (info->flags != pkv::kPrefillPlan)
    return fail(KV_ERR_INVALID_ARG, "the plan is not one of "
                                    "paged_latent_prefill_plan");
  if (info->n_merge_rows != total || info->n_row_items < 0 ||
      info->n_tile_items < 0 || info->partial_rows < 0 ||
      info->partial_rows > INT32_MAX || (total > 0) != (info->n_tile_items > 0) ||
      (total > 0) != (info->n_row_items > 0) ||
      (int64_t)info->n_tile_items * Hq > INT32_MAX ||
      (int64_t)info->n_row_items * Hq > INT32_MAX / 2)
    return fail(KV_ERR_INVALID_ARG, "plan info does not match the step");
  const size_t need = pkv::prefill_workspace(info->n_row_items, Hq);
  if (ws_bytes < need || (size_t)info->workspace_bytes != need)
    return fail(KV_ERR_INVALID_ARG, "workspace %zu bytes < %zu needed", ws_bytes,
                need);
  auto* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t st = (cudaStream_t)stream;
  pre::clear_kernel<<<1, 32, 0, st>>>(reinterpret_cast<pkv::DeviceStatus*>(ws));
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess)
    return fail(KV_ERR_CUDA, "latent prefill: %s", cudaGetErrorString(e));
  if (total == 0) return KV_OK;
  const int64_t tiles = (int64_t)info->n_row_items * Hq;
  pre::Params p;
  p.uniq = plan + pkv::kPlanHeaderInts;
  p.valid = p.uniq + info->n_row_items;
  p.slots = p.valid + info->n_row_items;
  p.tiles = reinterpret_cast<const pkv::PrefillTile*>(p.slots + info->partial_rows);
  p.k_exp = reinterpret_cast<__nv_bfloat16*>(ws + pkv::kStatusBytes);
  p.v_exp = reinterpret_cast<__nv_bfloat16*>(
      ws + pkv::kStatusBytes + pkv::prefill_half(info->n_row_items, Hq));
  p.out = static_cast<__nv_bfloat16*>(out);
  p.status = reinterpret_cast<pkv::DeviceStatus*>(ws);
  p.n_uniq = info->n_row_items;
  p.n_slots = (int)info->partial_rows;
  p.n_tiles = info->n_tile_items;
  p.Hq = Hq;
  p.total = total;
  p.num_blocks = num_blocks;
  p.scale_log2 = scale * 1.4426950408889634f;
  CUtensorMap tx, tw, tq, tk, tv, tr;
  if (kv_status s = pre::make_matrix_map(&tx, c_pool, num_blocks * 16, rank, 16))
    return s;
  if (kv_status s = pre::make_matrix_map(&tw, w_kv, (int64_t)Hq * 2 * head_dim,
                                         rank, 2 * head_dim))
    return s;
  if (kv_status s = pre::make_query_map(&tq, q, total, Hq)) return s;
  if (kv_status s = pre::make_expanded_map(&tk, p.k_exp, tiles)) return s;
  if (kv_status s = pre::make_expanded_map(&tv, p.v_exp, tiles)) return s;
  if (kv_status s = pre::make_matrix_map(&tr, r_pool, num_blocks * 16, rope_dim, 16))
    return s;
  static std::atomic<uint64_t> opted_ex{0}, opted_at{0};
  int dev = 0, sms = 152;
  e = cudaGetDevice(&dev);
  if (e == cudaSuccess)
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess)
    e = pkv::opt_in_smem(pre::ex::expand_kernel, pre::ex::kSmem, opted_ex);
  if (e == cudaSuccess)
    e = pkv::opt_in_smem(pre::at::prefill_kernel, pre::at::kSmem, opted_at);
  if (e != cudaSuccess)
    return fail(KV_ERR_CUDA, "latent prefill: %s", cudaGetErrorString(e));
  const int64_t work = (int64_t)((p.n_uniq + 7) / 8) * Hq;
  pre::ex::expand_kernel<<<(unsigned)std::min<int64_t>(work, sms),
                           pre::ex::kThreads, pre::ex::kSmem, st>>>(tx, tw, p);
  e = cudaGetLastError();
  if (e != cudaSuccess)
    return fail(KV_ERR_CUDA, "expansion kernel: %s", cudaGetErrorString(e));
  e = pkv::launch_early(pre::at::prefill_kernel, p.n_tiles * Hq,
                        pre::at::kThreads, pre::at::kSmem, st, tq, tk, tv, tr, p);
  if (e != cudaSuccess)
    return fail(KV_ERR_CUDA, "prefill kernel: %s", cudaGetErrorString(e));
  return KV_OK;
}
