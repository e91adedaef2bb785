// Latent prefill, expanded form (paged_latent_prefill_attn): new tokens attend
// causally to all cached tokens of their branch, with keys and values expanded
// from the latents per head,
//   k[t][h] = [Wk_h c_t ; r_t] (128 + 64),  v[t][h] = Wv_h c_t (128),
//   out[i][h] = sum_{t <= pos(i)} softmax_t(scale q[i][h] . k[t][h]) v[t][h].
// Against the absorbed form this costs 2 x 320 flops a row and token instead of
// 2 x 1088, for 2 x 512 x 256 flops a token and head once.
//
// Expansion kernel: pairs of CTAs (cta_group::2), [256 tokens x 512] x [512 x 256]
// per token tile and head (the tokens are sixteen distinct blocks of the step,
// gathered through the plan's list; a block shared by branches is expanded once),
// written as bf16 to [slot][head][16][128] -- the rounding of a cached key or
// value.  A pair's work is a run of (tile, head), heads innermost: each CTA keeps
// its 128 tokens' latents in shared memory (128 KB) while the heads pass, and half
// of a head's weights stream through a ring of 64-dimension stages (16 KB each;
// with both operands streamed to single CTAs, 48 KB per four products of 128
// cycles, L2 bounded it: 63 us for 8192 tokens and 32 heads, 45 now).  Products
// go to two 256-column halves of TMEM so that a tile's epilogue, which bounds it
// now, overlaps the next one's products.
//
// Attention kernel: pairs of CTAs (cta_group::2), one on every two SMs, that take
// work items (a tile of 256 query rows and a head) as they come.  Each CTA has 128
// of the rows and loads half of every key tile of 128 tokens (64 tokens of K, 64
// columns of V), which leaves room for four stages of each: with whole tiles in
// one CTA, V had one stage and its load (1.3 us) lay on every tile's path (a tile of
// 256 rows and 128 keys took 2.4 us of one SM; here 0.70 us of two, 1410 cycles, 1280
// of them products).
// The rows' two warpgroups take the key tiles in turn, each with its own maximum,
// sum and O, joined at the item's end.  TMEM: S (128 columns), P of the two
// warpgroups (2 x 64, bf16 pairs), O of the two (2 x 128).  QK(j) may overwrite S
// once it has been read, which the rows do while PV(j - 2) runs; the softmax of a
// tile (a thread a row, base 2, lazy maximum, two columns to an instruction) lies
// behind the products of two others.  Bound by power: 1 x 8192 tokens with 32
// heads run at 1.65 PFLOP/s, 1.55 when repeated without a pause.  Tiles of 256 rows
// waste what a chunk's last one does not fill: 13 of them for 2698 rows in six chunks
// are 19% padding.
//
// Tokens past a row's position are replaced by -inf before the maximum; values
// of slots past a branch's length, and those of tokens whose latents are not
// finite, are written as zeros by the expansion, and blocks past the tile's range
// take no part in PV.

#include <algorithm>
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
using tc::tmem_ld32;
using tc::tmem_st32;
using tc::tmem_wait_ld;
using tc::tmem_wait_st;
using tc::uniform;

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
  int* next;              // work items handed out past the first of each pair
  int n_uniq, n_slots, n_tiles, Hq, total, heads;  // heads of a group
  int64_t num_blocks;
  float scale_log2;
};

// After a time-out loads may be in flight (else a product has waited for every
// one): about two milliseconds for them to land.
__device__ __forceinline__ void wait_for_copies() {
  const long long t0 = clock64();
  while (clock64() - t0 < (1 << 22)) {
  }
}

// Two fp32 in one operation.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
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

constexpr int kX = 128 * 128;                   // 64 dimensions of a CTA's latents
constexpr int kW = 128 * 128;                   // and of half a head's weights
constexpr int kNS = 5;                          // stages of W
constexpr int kChunks = kRank / 64;
constexpr int kSlots = 16;                      // slots of a pair's token tile
constexpr int kOffW = kChunks * kX;
constexpr int kOffTurn = kOffW + kNS * kW;
constexpr int kTiles = kOffTurn + 8 * 2048;
constexpr int kThreads = 12 * 32;  // warps 0-7 rows, 8 products, 9-10 W, 11 X

struct Small {
  // x_full, w_full and d_empty are used in the even CTA alone.
  uint64_t x_full[kChunks], x_empty[kChunks], w_full[kNS], w_empty[kNS], d_full[2],
      d_empty[2], drain;
  uint32_t tmem_base;
  int aborted;
};
constexpr int kSmem = kTiles + (int)sizeof(Small);
static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    expand_kernel(const __grid_constant__ CUtensorMap tmX,
                  const __grid_constant__ CUtensorMap tmW, const Params p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  Small& sh = *reinterpret_cast<Small*>(smem + kTiles);
  volatile int* aborted = &sh.aborted;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (base & 1023) {  // never, with no static shared memory
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (threadIdx.x == 0) record_status(p.status, KV_ERR_INTERNAL, (int)base);
    return;
  }
  const int rank = (int)tc::cluster_rank();
  if (threadIdx.x == 0) {
    for (int c = 0; c < kChunks; ++c) {
      mbar_init(smem_u32(&sh.x_full[c]), 2);
      mbar_init(smem_u32(&sh.x_empty[c]), 1);
    }
    for (int s = 0; s < kNS; ++s) {
      mbar_init(smem_u32(&sh.w_full[s]), 2);
      mbar_init(smem_u32(&sh.w_empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&sh.d_full[b]), 1);
      mbar_init(smem_u32(&sh.d_empty[b]), 16);
    }
    mbar_init(smem_u32(&sh.drain), 1);
    sh.aborted = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmW);
  }
  __syncwarp();
  if (warp == 8) tc::tmem_alloc2(smem_u32(&sh.tmem_base), kTmemCols);
  fence_before_sync();
  tc::cluster_sync();
  fence_after_sync();
  const uint32_t tmem = sh.tmem_base;
  // Launched while the status is cleared: nothing of it before this.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // A pair's work: consecutive (token tile, head), heads innermost; a tile's
  // latents stay in shared memory while its heads pass.
  const int pairs = gridDim.x >> 1, pair = blockIdx.x >> 1;
  const int64_t n_work = (int64_t)((p.n_uniq + kSlots - 1) / kSlots) * p.Hq;
  const int begin = (int)(n_work * pair / pairs);
  const int end = (int)(n_work * (pair + 1) / pairs);
  auto timed_out = [&](int site) {
    if (!*aborted) record_status(p.status, KV_ERR_TIMEOUT, site);
    atomicExch(&sh.aborted, 1);
    tc::cluster_store4(tc::map_rank(smem_u32(&sh.aborted), rank ^ 1), 1u);
  };

  if (warp < 8) {
    const int wg = warp >> 2;  // 0: keys, 1: values
    const int row0 = (warp & 3) * 32, r = row0 + lane;
    const uint32_t drow = tmem + ((uint32_t)row0 << 16) + wg * kHead;
    uint8_t* turn = smem + kOffTurn + warp * 2048;
    __nv_bfloat16* exp = wg == 0 ? p.k_exp : p.v_exp;
    uint32_t n = 0;
    bool ok = true;
    for (int i = begin; i < end; ++i, ++n) {
      const int slot0 = i / p.Hq * kSlots + rank * 8, h = i % p.Hq;
      const uint32_t b = n & 1;
      const int slot = slot0 + (r >> 4);
      // Values past the branch's length would meet weights of zero: zeros.
      const bool zero =
          wg == 1 && (slot >= p.n_uniq || (r & 15) >= p.valid[min(slot, p.n_uniq - 1)]);
      ok = all_wait(smem_u32(&sh.d_full[b]), (n >> 1) & 1);
      ok = __all_sync(0xffffffffu, ok && !*aborted);
      if (!ok) break;
      fence_after_sync();
#pragma unroll 1
      for (int c = 0; c < kHead; c += 32) {
        uint32_t v[32], w[16];
        tmem_ld32(drow + b * 256 + c, v);
        tmem_wait_ld();
        if (c == kHead - 32) {  // D has been read
          fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::remote_arrive(tc::map_rank(smem_u32(&sh.d_empty[b]), 0));
        }
        // A latent with an infinity or a NaN makes every value expanded from it one
        // (w x inf, 0 included).  Rows that do not see the token have weight 0, and
        // 0 x NaN would be theirs too: zeros instead.  Those that see it have NaN
        // from its keys.
        float least = fabsf(__uint_as_float(v[0]));  // NaN if all are
#pragma unroll
        for (int k = 1; k < 32; ++k) least = fminf(least, fabsf(__uint_as_float(v[k])));
        const bool none = zero || (wg == 1 && !(least < INFINITY));
#pragma unroll
        for (int k = 0; k < 16; ++k)
          w[k] = none ? 0u
                      : pack_bf16(__uint_as_float(v[2 * k]),
                                  __uint_as_float(v[2 * k + 1]));
        put_rows(turn, w, lane, [&](int rr) -> uint8_t* {
          const int row = row0 + rr, s = slot0 + (row >> 4);
          if (s >= p.n_uniq) return nullptr;
          return reinterpret_cast<uint8_t*>(
              exp + (((int64_t)s * p.Hq + h) * 16 + (row & 15)) * kHead + c);
        });
      }
    }
    if (!ok && lane == 0) timed_out(50);
  } else if (warp == 8) {
    if (rank == 0) {
      constexpr uint32_t id = idesc(256, 256, false);
      const bool lead = elect_one();
      const int heads = uniform(p.Hq);
      uint32_t n = 0, s = 0, ph = 0, tile = 0;  // tile: of the pair's
      bool ok = true;
      for (int i = uniform(begin); i < end && ok; ++i, ++n) {
        const uint32_t b = n & 1, d = tmem + b * 256;
        const bool first = n == 0 || i % heads == 0;
        const bool last = i == end - 1 || (i + 1) % heads == 0;
        if (n >= 2) ok = all_wait(smem_u32(&sh.d_empty[b]), ((n >> 1) - 1) & 1);
        for (int c = 0; c < kChunks && ok; ++c) {
          if (first) ok = all_wait(smem_u32(&sh.x_full[c]), tile & 1);
          ok = ok && all_wait(smem_u32(&sh.w_full[s]), ph);
          if (!ok) break;
          fence_after_sync();
          const uint64_t xd = sdesc(base + c * kX, 16, 1024);
          const uint64_t wd = sdesc(base + kOffW + s * kW, 16, 1024);
          if (lead) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc::umma2_ss(d, xd + k * 2, wd + k * 2, id, c > 0 || k > 0 ? 1u : 0u);
            tc::umma2_commit(smem_u32(&sh.w_empty[s]));
            if (last) tc::umma2_commit(smem_u32(&sh.x_empty[c]));
            if (c == kChunks - 1) tc::umma2_commit(smem_u32(&sh.d_full[b]));
          }
          __syncwarp();
          if (++s == kNS) {
            s = 0;
            ph ^= 1;
          }
        }
        tile += last;
        ok = __all_sync(0xffffffffu, ok && !*aborted);
      }
      if (lead) {
        if (!ok) timed_out(51);
        // Every product has finished once this lands.
        tc::umma2_commit(smem_u32(&sh.drain));
        mbar_wait(smem_u32(&sh.drain), 0);
      }
    }
  } else if (warp < 11) {
    // Half of a head's weights: keys' rows in the even CTA, values' in the odd
    // one; stages alternate between the two warps.
    const uint32_t me = warp - 9;
    uint32_t k = 0;
    bool ok = true;
    for (int i = begin; i < end && ok; ++i) {
      const int h = i % p.Hq;
      for (int c = 0; c < kChunks; ++c, ++k) {
        if ((k & 1) != me) continue;
        const uint32_t s = k % kNS, bar = tc::map_rank(smem_u32(&sh.w_full[s]), 0);
        if (k >= kNS) ok = all_wait(smem_u32(&sh.w_empty[s]), (k / kNS - 1) & 1);
        ok = __all_sync(0xffffffffu, ok && !*aborted);
        if (!ok) break;
        if (lane == 0) tc::remote_expect_tx(bar, kW);
        __syncwarp();
        if (lane < 2)
          tc::tma2_load_2d(base + kOffW + s * kW + lane * (kW / 2), &tmW, c * 64,
                           h * 256 + rank * 128 + lane * 64, bar);
        __syncwarp();
      }
    }
    if (!ok && lane == 0) timed_out(52);
  } else {
    // Latents: eight slots of each token tile, a box a slot and 64 dimensions.
    bool ok = true;
    uint32_t tile = 0;
    for (int i = begin; i < end && ok; i = (i / p.Hq + 1) * p.Hq, ++tile) {
      const int slot = i / p.Hq * kSlots + rank * 8 + lane;
      int phys = lane < 8 && slot < p.n_uniq ? p.uniq[slot] : -1;
      if (lane < 8 && slot < p.n_uniq && (phys < 0 || phys >= p.num_blocks)) {
        record_status(p.status, KV_ERR_DEVICE, phys);
        phys = -1;
      }
      const int nb = __popc(__ballot_sync(0xffffffffu, phys >= 0));
      for (int c = 0; c < kChunks; ++c) {
        const uint32_t bar = tc::map_rank(smem_u32(&sh.x_full[c]), 0);
        if (tile > 0) ok = all_wait(smem_u32(&sh.x_empty[c]), (tile - 1) & 1);
        ok = __all_sync(0xffffffffu, ok && !*aborted);
        if (!ok) break;
        if (lane == 0) tc::remote_expect_tx(bar, nb * 2048);
        __syncwarp();
        if (phys >= 0)
          tc::tma2_load_2d(base + c * kX + lane * 2048, &tmX, c * 64, phys * 16, bar);
        __syncwarp();
      }
    }
    if (!ok && lane == 0) timed_out(53);
  }
  __syncwarp();
  fence_before_sync();
  __syncthreads();
  if (*aborted) wait_for_copies();
  __syncwarp();
  tc::cluster_sync();
  fence_after_sync();
  if (warp == 8) tc::tmem_free2(tmem, kTmemCols);
  tc::cluster_sync();  // neither CTA leaves before both have given it back
}

}  // namespace ex

// ---- attention ------------------------------------------------------------------

namespace at {

constexpr int kT = 128, kTB = 8;             // tokens and blocks of a key tile
constexpr int kM = 128;                      // query rows of a CTA
constexpr int kQ = 3 * kM * 128;             // Q: three 64-wide parts
constexpr int kBlk = 16 * kHead * 2;         // a block's expanded keys of a head
constexpr int kKn = kTB / 2 * kBlk;          // a K stage (64 tokens): expanded part,
constexpr int kK = kKn + kT / 2 * 128;       // and position part
constexpr int kV = kT * 128;                 // a V stage: 128 tokens x 64 columns
constexpr int kNS = 4;                       // stages of K and of V
constexpr int kOffK = kQ;
constexpr int kOffV = kOffK + kNS * kK;
constexpr int kOffTurn = kOffV + kNS * kV;
constexpr int kTiles = kOffTurn + 8 * 2048;
constexpr int kLoads = 3;                    // load warps
constexpr int kThreads = (9 + kLoads) * 32;  // warps 0-7 rows, 8 products, 9- loads
constexpr uint32_t kColP = 128, kColO = 256;  // TMEM: S, P (2), O (2)
constexpr float kRescale = 8.f;    // lazy-max threshold (log2 units)

struct Small {
  // q_full, k_full, v_full, s_empty, p_full and o_empty are used in the even CTA
  // alone, item_empty in the odd one.
  uint64_t q_full, k_full[kNS], k_empty[kNS], v_full[kNS], v_empty[kNS],
      s_full[2], s_empty, p_full[2], p_empty[2], o_ready, o_empty, q_empty,
      item_full[2], item_empty[2];
  int4 item[2];          // PrefillTile,
  int item_head[2];      // and head, -1: no more
  float stat[2][2][kM];  // maximum and sum of the two halves' rows
  uint32_t tmem_base;
  int aborted;
};
constexpr int kSmem = kTiles + (int)sizeof(Small);
static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");

__device__ __forceinline__ int next_index(const Params& p, int pairs, int lane) {
  int i = 0;
  if (lane == 0) i = pairs + atomicAdd(p.next, 1);
  return __shfl_sync(0xffffffffu, i, 0);
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
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
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (threadIdx.x == 0) record_status(p.status, KV_ERR_INTERNAL, (int)base);
    return;
  }
  const int rank = (int)tc::cluster_rank();

  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&sh.q_full), 2);
    for (int s = 0; s < kNS; ++s) {
      mbar_init(smem_u32(&sh.k_full[s]), 2);
      mbar_init(smem_u32(&sh.k_empty[s]), 1);
      mbar_init(smem_u32(&sh.v_full[s]), 2);
      mbar_init(smem_u32(&sh.v_empty[s]), 1);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(smem_u32(&sh.s_full[g]), 1);
      mbar_init(smem_u32(&sh.p_full[g]), 8);
      mbar_init(smem_u32(&sh.p_empty[g]), 1);
    }
    mbar_init(smem_u32(&sh.s_empty), 8);
    mbar_init(smem_u32(&sh.o_ready), 1);
    mbar_init(smem_u32(&sh.o_empty), 16);
    mbar_init(smem_u32(&sh.q_empty), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh.item_full[i]), 1);
      mbar_init(smem_u32(&sh.item_empty[i]), 2 * (8 + kLoads) + 1);
    }
    sh.aborted = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    tma_prefetch_desc(&tmR);
  }
  __syncwarp();
  if (warp == 8) tc::tmem_alloc2(smem_u32(&sh.tmem_base), kTmemCols);
  fence_before_sync();
  tc::cluster_sync();
  fence_after_sync();
  const uint32_t tmem = sh.tmem_base;
  // Launched while the expansion runs: nothing of global memory before this.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  auto timed_out = [&](int site) {
    if (!*aborted) record_status(p.status, KV_ERR_TIMEOUT, site);
    atomicExch(&sh.aborted, 1);
    tc::cluster_store4(tc::map_rank(smem_u32(&sh.aborted), rank ^ 1), 1u);
  };

  // The pair's items in turn; `tiles0` key tiles came before the item, and its
  // tile j is tile tiles0 + j of the pair's stream, which the stages, barriers and
  // the warpgroups' turns go by.
  struct Items {
    PrefillTile t;
    int h, nt = 0, nblk;
    uint32_t n = 0, tiles0 = 0;  // n: items taken
  } it;
  auto next_item = [&](bool& ok) {
    it.tiles0 += it.nt;
    const uint32_t slot = it.n & 1;
    ok = ok && tc::all_wait_cluster(smem_u32(&sh.item_full[slot]), (it.n >> 1) & 1);
    if (!ok) return false;
    const int4 v = sh.item[slot];
    it.t = {v.x, v.y, v.z, v.w};
    it.h = sh.item_head[slot];
    __syncwarp();
    if (lane == 0)
      tc::remote_arrive(tc::map_rank(smem_u32(&sh.item_empty[slot]), 1));
    ++it.n;
    const int len = it.t.pos0 + it.t.nrows;  // tokens the tile's last row sees
    it.nblk = (len + 15) / 16;
    it.nt = (len - 1) / kT + 1;
    return it.h >= 0;
  };

  if (warp < 8) {
    // ---- rows: thread = row r, every second key tile ----------------------------
    const int g = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t prow = lane_base + kColP + g * 64;
    const uint32_t orow = lane_base + kColO + g * kHead;
    const uint32_t s_empty = tc::map_rank(smem_u32(&sh.s_empty), 0);
    const uint32_t p_full = tc::map_rank(smem_u32(&sh.p_full[g]), 0);
    const uint32_t o_empty = tc::map_rank(smem_u32(&sh.o_empty), 0);
    bool ok = true;
    // All or none go on: they meet at the item's end.
    while (tc::bar_and(1, 256, next_item(ok))) {
      const PrefillTile t = it.t;
      const int nt = it.nt, h = it.h;
      const int pos = t.pos0 + rank * kM + r;  // this row's position
      const int pos_lo = pos - lane;           // the warp's first
      float m_used = -INFINITY, l = 0.f;
      for (int j = (it.tiles0 ^ g) & 1; j < nt; j += 2) {
        const uint32_t q = it.tiles0 + j;
        ok = all_wait(smem_u32(&sh.s_full[g]), (q >> 1) & 1);
        if (!ok) break;
        fence_after_sync();
        uint32_t u[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(lane_base + c * 32, u[c]);
        tmem_wait_ld();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::remote_arrive(s_empty);  // S may be overwritten
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
        const uint64_t scale2 = pack2(p.scale_log2, p.scale_log2);
        const uint64_t neg2 = pack2(neg_m, neg_m);
        uint64_t s2[2] = {0, 0};  // sums of the even and the odd columns, twice
#pragma unroll
        for (int c2 = 0; c2 < 2; ++c2) {
          uint32_t pk[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int c = c2 * 2 + (i >> 4), k = (2 * i) & 31;
            float a, b;
            unpack2(fma2((uint64_t)u[c][k + 1] << 32 | u[c][k], scale2, neg2), a, b);
            a = ex2(a);
            b = ex2(b);
            s2[i & 1] = add2(s2[i & 1], pack2(a, b));
            pk[i] = pack_bf16(a, b);
          }
          if (c2 == 0 && j > 1) {
            // PV(j - 2) done: P may be overwritten, and O rescaled.
            ok = all_wait(smem_u32(&sh.p_empty[g]), ((q - 2) >> 1) & 1);
            if (!ok) break;
            fence_after_sync();
          }
          tmem_st32(prow + c2 * 32, pk);
        }
        if (!ok) break;
        float s_even, s_odd;
        unpack2(add2(s2[0], s2[1]), s_even, s_odd);
        l += s_even + s_odd;
        if (__any_sync(0xffffffffu, need) && j > 1) tc::rescale_o_row(orow, alpha);
        tmem_wait_st();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::remote_arrive(p_full);
      }
      ok = ok && all_wait(smem_u32(&sh.o_ready), (it.n - 1) & 1);
      sh.stat[g][0][r] = m_used;
      sh.stat[g][1][r] = l;
      ok = tc::bar_and(1, 256, ok && !*aborted);
      if (!ok) break;
      fence_after_sync();
      // The two halves of the key tiles joined, that of tile 0 first: which
      // warpgroup has it depends on the items before, and a fused multiply-add
      // rounds its two products differently.  Each warp 64 columns.
      const int a = it.tiles0 & 1;  // the warpgroup of tile 0
      const float m0 = sh.stat[a][0][r], m1 = sh.stat[a ^ 1][0][r];
      const float top = fmaxf(m0, m1);  // finite: every row sees token 0
      const float e0 = ex2(m0 - top), e1 = ex2(m1 - top);
      const float inv = 1.f / (e0 * sh.stat[a][1][r] + e1 * sh.stat[a ^ 1][1][r]);
      const float w0 = e0 * inv, w1 = e1 * inv;
      const bool has1 = nt > 1;  // an item of one tile has written one O
      const uint32_t o0 = lane_base + kColO + a * kHead;
      const uint32_t o1 = lane_base + kColO + (a ^ 1) * kHead;
      uint8_t* turn = smem + kOffTurn + warp * 2048;
      const int n = t.nrows - rank * kM - (warp & 3) * 32;  // rows of the warp
      const int64_t row0 = t.row0 + rank * kM + (warp & 3) * 32;
#pragma unroll 1
      for (int c = g * 64; c < g * 64 + 64; c += 32) {
        uint32_t v[32], v1[32], w[16];
        tmem_ld32(o0 + c, v);
        tmem_ld32(o1 + c, v1);
        tmem_wait_ld();
        if (c & 32) {  // O has been read
          fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::remote_arrive(o_empty);
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          float o[2];
#pragma unroll
          for (int x = 0; x < 2; ++x)
            o[x] = __uint_as_float(v[2 * k + x]) * w0 +
                   (has1 ? __uint_as_float(v1[2 * k + x]) * w1 : 0.f);
          w[k] = pack_bf16(o[0], o[1]);
        }
        put_rows(turn, w, lane, [&](int rr) -> uint8_t* {
          if (rr >= n) return nullptr;
          return reinterpret_cast<uint8_t*>(
              p.out + ((row0 + rr) * p.Hq + h) * kHead + c);
        });
      }
    }
    if (!ok && lane == 0) timed_out(60);
  } else if (warp == 8) {
    bool ok = true;
    if (rank == 0) {
      // ---- products of both CTAs (uniform warp, one lane issues) -----------------
      constexpr uint32_t id_qk = idesc(256, kT, false);
      constexpr uint32_t id_pv = idesc(256, kHead, true);
      const bool lead = elect_one();
      while (next_item(ok)) {
        const int n = uniform(it.nt), blocks = uniform(it.nblk);
        const uint32_t t0 = uniform(it.tiles0), item = it.n - 1;
        ok = all_wait(smem_u32(&sh.q_full), item & 1);
        // QK(j) and PV(j - 2) in turn: the rows read S(j) while PV(j - 2) runs.
        for (int j = 0; j < n + 2 && ok; ++j) {
          if (j < n) {
            const uint32_t q = t0 + j, st = q % kNS;
            const uint32_t kst = base + kOffK + st * kK;
            const uint64_t qd = sdesc(base, 16, 1024);
            const uint64_t kd = sdesc(kst, 16, 2048);
            const uint64_t rd = sdesc(kst + kKn, 16, 1024);
            ok = all_wait(smem_u32(&sh.k_full[st]), (q / kNS) & 1) &&
                 (q == 0 || all_wait(smem_u32(&sh.s_empty), (q - 1) & 1));
            if (!ok) break;
            fence_after_sync();
            if (lead) {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                tc::umma2_ss(tmem, qd + (((k >> 2) * 16384 + (k & 3) * 32) >> 4),
                             kd + (((k >> 2) * 1024 + (k & 3) * 32) >> 4), id_qk,
                             k > 0 ? 1u : 0u);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                tc::umma2_ss(tmem, qd + ((2 * 16384 + k * 32) >> 4), rd + k * 2,
                             id_qk, 1u);
              tc::umma2_commit(smem_u32(&sh.s_full[q & 1]));
              tc::umma2_commit(smem_u32(&sh.k_empty[st]));
              if (j == n - 1) tc::umma2_commit(smem_u32(&sh.q_empty));
            }
            __syncwarp();
          }
          const int i = j - 2;
          if (i >= 0) {
            const uint32_t q = t0 + i, st = q % kNS;
            ok = all_wait(smem_u32(&sh.v_full[st]), (q / kNS) & 1) &&
                 all_wait(smem_u32(&sh.p_full[q & 1]), (q >> 1) & 1) &&
                 (i > 0 || item == 0 ||
                  all_wait(smem_u32(&sh.o_empty), (item - 1) & 1));
            if (!ok) break;
            fence_after_sync();
            if (lead) {
              const uint32_t pcol = tmem + kColP + (q & 1) * 64;
              const uint32_t dout = tmem + kColO + (q & 1) * kHead;
              const int nb = min(kTB, blocks - i * kTB);
              const uint64_t vd = sdesc(base + kOffV + st * kV, 1024, 1024);
#pragma unroll
              for (int k = 0; k < kTB; ++k)
                if (k < nb)
                  tc::umma2_ts(dout, pcol + k * 8, vd + k * (2048 >> 4), id_pv,
                               i > 1 || k > 0 ? 1u : 0u);
              tc::umma2_commit(smem_u32(&sh.p_empty[q & 1]));
              tc::umma2_commit(smem_u32(&sh.v_empty[st]));
              if (i == n - 1) tc::umma2_commit(smem_u32(&sh.o_ready));
            }
            __syncwarp();
          }
          ok = __all_sync(0xffffffffu, !*aborted);
        }
      }
      if (!ok && lead) {
        timed_out(61);
        // Every product issued has finished once this lands, or a time has passed.
        tc::umma2_commit(smem_u32(&sh.o_ready));
        mbar_wait(smem_u32(&sh.o_ready), (it.n - 1) & 1);
      }
    } else {
      // ---- the pair's work items (odd CTA): the first by its place in the grid,
      // then as they come.  Head groups in turn (what the pairs read at a time
      // stays in L2), in a group the longest tiles first.
      const int n_items = p.n_tiles * p.Hq, pairs = gridDim.x >> 1;
      int i = blockIdx.x >> 1;
      for (uint32_t n = 0;; ++n) {
        const uint32_t slot = n & 1;
        if (n >= 2) ok = all_wait(smem_u32(&sh.item_empty[slot]), ((n >> 1) - 1) & 1);
        ok = __all_sync(0xffffffffu, ok && !*aborted);
        if (!ok) break;
        PrefillTile t{0, 1, 0, 0};
        int h = -1;
        for (; i < n_items; i = next_index(p, pairs, lane)) {
          const int group = i / (p.n_tiles * p.heads);
          const int heads = min(p.heads, p.Hq - group * p.heads);
          const int rest = i - group * p.n_tiles * p.heads;
          t = p.tiles[rest / heads];
          h = group * p.heads + rest % heads;
          if (t.nrows >= 1 && t.nrows <= kPrefillRows && t.pos0 >= 0 &&
              t.row0 >= 0 && t.row0 + t.nrows <= p.total && t.table >= 0 &&
              t.table + (t.pos0 + t.nrows + 15) / 16 <= p.n_slots)
            break;
          if (lane == 0) record_status(p.status, KV_ERR_DEVICE, -1 - i);
          h = -1;
        }
        if (lane < 2) {
          const uint32_t bar = tc::map_rank(smem_u32(&sh.item_full[slot]), lane);
          tc::remote_expect_tx(bar, 20);
          tc::remote_store16(tc::map_rank(smem_u32(&sh.item[slot]), lane), t.row0,
                             t.nrows, t.pos0, t.table, bar);
          tc::remote_store4(tc::map_rank(smem_u32(&sh.item_head[slot]), lane), h, bar);
        }
        __syncwarp();
        if (h < 0) break;
        i = next_index(p, pairs, lane);
      }
      if (!ok && lane == 0) timed_out(65);
    }
  } else {
    // ---- loads of this CTA's halves: its rows of Q, half of a key tile's keys,
    // half of the values' columns; a warp takes every third key tile --------------
    const int me = warp - 9;
    bool ok = true;
    // The expansion's stores, read by bulk copies from here on.
    asm volatile("fence.proxy.async;" ::: "memory");
    // Lanes 0-3 the half's expanded keys, 4-7 its position keys, 8-15 values.
    const int bi = lane < 8 ? rank * 4 + (lane & 3) : lane & 7;
    while (next_item(ok)) {
      const int nt = it.nt, h = it.h;
      const uint32_t item = it.n - 1;
      if (me == 0) {
        if (item > 0) ok = all_wait(smem_u32(&sh.q_empty), (item - 1) & 1);
        ok = __all_sync(0xffffffffu, ok && !*aborted);
        if (!ok) break;
        const uint32_t bar = tc::map_rank(smem_u32(&sh.q_full), 0);
        if (lane == 0) tc::remote_expect_tx(bar, kQ);
        __syncwarp();
        if (lane < 3)
          tc::tma2_load_3d(base + lane * 16384, &tmQ, lane * 64, h,
                           it.t.row0 + rank * kM, bar);
        __syncwarp();
      }
      auto slot_of = [&](int tile) {
        const int blk = tile * kTB + bi;
        if (lane >= 16 || tile >= nt || blk >= it.nblk) return -1;
        const int s = p.slots[it.t.table + blk];
        if (s >= 0 && s < p.n_uniq) return s;
        record_status(p.status, KV_ERR_DEVICE, s);
        return -1;
      };
      auto phys_of = [&](int slot) {
        if (lane < 4 || lane >= 8 || slot < 0) return -1;
        const int b = p.uniq[slot];
        return b >= 0 && b < p.num_blocks ? b : -1;
      };
      int j = (me + kLoads - (int)(it.tiles0 % kLoads)) % kLoads;
      int next = slot_of(j), next_phys = phys_of(next);
      for (; j < nt; j += kLoads) {
        const int slot = next, phys = next_phys;
        next = slot_of(j + kLoads);
        next_phys = phys_of(next);
        const bool load = slot >= 0 && (lane < 4 || lane >= 8 || phys >= 0);
        const uint32_t act = __ballot_sync(0xffffffffu, load);
        const uint32_t q = it.tiles0 + j, s = q % kNS;
        const uint32_t kbar = tc::map_rank(smem_u32(&sh.k_full[s]), 0);
        const uint32_t vbar = tc::map_rank(smem_u32(&sh.v_full[s]), 0);
        if (q >= kNS) ok = all_wait(smem_u32(&sh.k_empty[s]), (q / kNS - 1) & 1);
        ok = __all_sync(0xffffffffu, ok && !*aborted);
        if (!ok) break;
        if (lane == 0)
          tc::remote_expect_tx(kbar, __popc(act & 0xf) * kBlk +
                                         __popc(act & 0xf0) * 2048);
        __syncwarp();
        const uint32_t kst = base + kOffK + s * kK;
        if (load && lane < 4)
          tc::tma2_load_5d_at(kst + lane * kBlk, &tmK, 0, slot * p.Hq + h, kbar);
        else if (load && lane < 8)
          tc::tma2_load_2d(kst + kKn + (lane - 4) * 2048, &tmR, 0, phys * 16, kbar);
        __syncwarp();
        if (q >= kNS) ok = all_wait(smem_u32(&sh.v_empty[s]), (q / kNS - 1) & 1);
        ok = __all_sync(0xffffffffu, ok && !*aborted);
        if (!ok) break;
        if (lane == 0) tc::remote_expect_tx(vbar, __popc(act >> 8) * 2048);
        __syncwarp();
        if (load && lane >= 8)
          tc::tma2_load_5d_at(base + kOffV + s * kV + bi * 2048, &tmV, rank,
                              slot * p.Hq + h, vbar);
        __syncwarp();
      }
    }
    if (!ok && lane == 0) timed_out(62);
  }
  __syncwarp();
  fence_before_sync();
  __syncthreads();
  if (*aborted) wait_for_copies();
  __syncwarp();
  tc::cluster_sync();
  fence_after_sync();
  if (warp == 8) tc::tmem_free2(tmem, kTmemCols);
  tc::cluster_sync();  // neither CTA leaves before both have given it back
}

}  // namespace at

// ---- host side ------------------------------------------------------------------

// Expanded keys or values, [slot][Hq][16][128] bf16.  Keys: a box is a (slot,
// head) tile of 4 KB, landing as four 1 KB atoms of 8 rows x 64 columns ordered
// (rows 0-7, half 0), (0-7, 1), (8-15, 0), (8-15, 1).  Values: one half of the
// columns, (rows 0-7), (8-15).
kv_status make_expanded_map(CUtensorMap* tm, const void* base, int64_t tiles,
                            int halves) {
  const cuuint64_t dims[5] = {64, 8, 2, 2, (cuuint64_t)tiles};
  const cuuint64_t strides[4] = {256, 128, 2048, 4096};
  const cuuint32_t box[5] = {64, 8, (cuuint32_t)halves, 2, 1};
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

__global__ void clear_kernel(DeviceStatus* status, int* next) {
  if (threadIdx.x != 0) return;
  *status = DeviceStatus{};
  *next = 0;
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
  // A step without queries may have empty tensors, which have no address.
  if (!info || !plan || !workspace || !c_pool || !r_pool || !w_kv ||
      (total != 0 && (!q || !out)))
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
      (int64_t)info->n_tile_items * Hq > INT32_MAX / 2 ||
      (int64_t)info->n_row_items * Hq > INT32_MAX / 2)
    return fail(KV_ERR_INVALID_ARG, "plan info does not match the step");
  const size_t need = pkv::prefill_workspace(info->n_row_items, Hq);
  if (ws_bytes < need || (size_t)info->workspace_bytes != need)
    return fail(KV_ERR_INVALID_ARG, "workspace %zu bytes < %zu needed", ws_bytes,
                need);
  auto* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t st = (cudaStream_t)stream;
  pre::Params p;
  p.status = reinterpret_cast<pkv::DeviceStatus*>(ws);
  p.next = reinterpret_cast<int*>(ws + sizeof(pkv::DeviceStatus));
  pre::clear_kernel<<<1, 32, 0, st>>>(p.status, p.next);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess)
    return fail(KV_ERR_CUDA, "latent prefill: %s", cudaGetErrorString(e));
  if (total == 0) return KV_OK;
  const int64_t tiles = (int64_t)info->n_row_items * Hq;
  p.uniq = plan + pkv::kPlanHeaderInts;
  p.valid = p.uniq + info->n_row_items;
  p.slots = p.valid + info->n_row_items;
  p.tiles = reinterpret_cast<const pkv::PrefillTile*>(p.slots + info->partial_rows);
  p.k_exp = reinterpret_cast<__nv_bfloat16*>(ws + pkv::kStatusBytes);
  p.v_exp = reinterpret_cast<__nv_bfloat16*>(
      ws + pkv::kStatusBytes + pkv::prefill_half(info->n_row_items, Hq));
  p.out = static_cast<__nv_bfloat16*>(out);
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
                                         rank, 64))
    return s;
  if (kv_status s = pre::make_query_map(&tq, q, total, Hq)) return s;
  if (kv_status s = pre::make_expanded_map(&tk, p.k_exp, tiles, 2)) return s;
  if (kv_status s = pre::make_expanded_map(&tv, p.v_exp, tiles, 1)) return s;
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
  // Heads whose expanded keys and values the pairs share L2 for.
  p.heads = (int)std::clamp<int64_t>(
      (48ll << 20) / ((int64_t)p.n_uniq * 16 * pre::kHead * 4), 1, Hq);
  const int sm_pairs = std::max(sms / 2, 1);
  const int64_t work =
      (int64_t)((p.n_uniq + pre::ex::kSlots - 1) / pre::ex::kSlots) * Hq;
  e = pkv::launch_early(pre::ex::expand_kernel,
                        2 * (int)std::min<int64_t>(work, sm_pairs),
                        pre::ex::kThreads, pre::ex::kSmem, st, tx, tw, p);
  if (e != cudaSuccess)
    return fail(KV_ERR_CUDA, "expansion kernel: %s", cudaGetErrorString(e));
  const int pairs = std::min(p.n_tiles * Hq, sm_pairs);
  e = pkv::launch_early(pre::at::prefill_kernel, 2 * pairs, pre::at::kThreads,
                        pre::at::kSmem, st, tq, tk, tv, tr, p);
  if (e != cudaSuccess)
    return fail(KV_ERR_CUDA, "prefill kernel: %s", cudaGetErrorString(e));
  return KV_OK;
}
