// Chunk attention (paged_chunk_attn): new tokens attend causally to all cached
// tokens of their branch,
//   out[i][h] = sum_{t <= pos(i)} softmax_t(scale q[i][h] . K[t][h / G]) V[t][h / G],
// K and V in the paged pool.  4 D flops for each query head and visible token; a
// prompt or a chunk is bound by the products, a few drafted tokens on long
// branches by the K and V bytes.
//
// Pairs of CTAs (cta_group::2), one on every two SMs, take work items (a tile of
// query tokens with the G heads of a kv-head, and a range of key tiles) as they
// come.  Rows are packed (token, head), so that a kv-head's keys are loaded once for
// all of its heads and single tokens fill G rows: a CTA has floor(128 / G) tokens.
// Each CTA loads half of every key tile of 128 tokens: 64 tokens of K, half of V's
// columns.  K and V tiles come in through TMA as they lie in the pool, a box per
// block, and land in the layouts the products take.
//
// The rows' two warpgroups take the key tiles in turn, each with its own maximum,
// sum and O, joined at the item's end.  TMEM: S (128 columns), P of the two
// warpgroups (2 x 64, bf16 pairs), O of the two (2 x D).  QK(j) may overwrite S
// once it has been read, which the rows do while PV(j - 2) runs; the softmax of a
// tile (a thread a row, base 2, lazy maximum, two columns to an instruction) lies
// behind the products of two others.
//
// Masks: scores of tokens past a row's position are replaced by -inf before the
// maximum.  Their weights are 0, but 0 x NaN is not: in key tiles that some row
// does not see whole, the load warp waits for V and writes zeros over slots past
// the item's last position and over values that are not finite, and the rows that
// do see such a value add it to their result at the end (from the pool; rare).
//
// Where the plan has cut a tile's keys, items write partial rows (maximum, sum, O
// in fp32) and a second kernel joins them.  e4m3 pools: the step's distinct blocks
// are widened to bf16 first, exactly, and read from there.

#include <algorithm>
#include <cmath>

#include "e4m3.cuh"
#include "prefill.cuh"
#include "tensor_map.h"

namespace pkv {
namespace chunk {

using tc::add2;
using tc::all_wait;
using tc::elect_one;
using tc::fence_after_sync;
using tc::fence_before_sync;
using tc::fma2;
using tc::idesc;
using tc::pack2;
using tc::put_rows;
using tc::sdesc;
using tc::tmem_ld32;
using tc::tmem_st32;
using tc::tmem_wait_ld;
using tc::tmem_wait_st;
using tc::uniform;
using tc::unpack2;

struct Params {
  const int32_t* slots;   // branches' tables
  const ChunkItem* items;
  const __nv_bfloat16* v; // [n_slots_pool][Hkv][16][D]
  __nv_bfloat16* out;     // [total][Hq][D]
  float2* ml;             // partial rows
  float* o;
  DeviceStatus* status;
  int* next;              // work items handed out past the first of each pair
  int n_slots, n_items, Hq, Hkv, G, total, heads;  // heads of a group
  int64_t blocks;         // blocks the slots may name
  int64_t partial_rows;
  float scale_log2;
};

constexpr int kT = kChunkKeys, kTB = kT / 16;  // tokens and blocks of a key tile
constexpr int kM = kChunkRows;                 // query rows of a CTA
constexpr int kLoads = 3;                      // load warps
constexpr int kThreads = (9 + kLoads) * 32;    // warps 0-7 rows, 8 products, 9- loads
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColP = 128, kColO = 256;   // TMEM: S, P (2), O (2)
constexpr float kRescale = 8.f;                // lazy-max threshold (log2 units)

template <int D>
struct Cfg {
  static constexpr int kQ = D / 64 * kM * 128;   // Q: 64-wide parts
  static constexpr int kBlkK = 16 * D * 2;       // a block's keys of a head
  static constexpr int kK = kTB / 2 * kBlkK;     // a K stage: 64 tokens
  static constexpr int kBlkV = 16 * D;           // half of a block's values
  static constexpr int kV = kTB * kBlkV;         // a V stage: 128 tokens, D / 2 columns
  static constexpr int kNS = D == 128 ? 5 : 8;   // stages of K and of V
  static constexpr int kOffK = kQ;
  static constexpr int kOffV = kOffK + kNS * kK;
  static constexpr int kOffTurn = kOffV + kNS * kV;
  static constexpr int kTiles = kOffTurn + 8 * 2048;
};

template <int NS>
struct Small {
  // q_full, k_full, v_full, s_empty, p_full and o_empty are used in the even CTA
  // alone, item_empty in the odd one, v_raw by the CTA's own load warps.
  uint64_t q_full, k_full[NS], k_empty[NS], v_full[NS], v_empty[NS], s_full[2],
      s_empty, p_full[2], p_empty[2], o_ready, o_empty, q_empty, item_full[2],
      item_empty[2], v_raw[kLoads];
  int4 item[2][2];       // ChunkItem, its pad the head (-1: no more)
  float stat[2][2][kM];  // maximum and sum of the two halves' rows
  uint32_t tmem_base;
  int aborted;
  int odd_values;        // a masked tile held a value that is not finite
};

template <int D>
constexpr int smem_bytes() {
  return Cfg<D>::kTiles + (int)sizeof(Small<Cfg<D>::kNS>);
}
static_assert(smem_bytes<128>() <= 227 * 1024, "shared memory of a CTA");
static_assert(smem_bytes<64>() <= 227 * 1024, "shared memory of a CTA");

// V as an MN-major operand.  D = 128: 64 columns of a CTA, rows of 128 bytes with
// 128-byte swizzle; D = 64: 32 columns, rows of 64 bytes with 64-byte swizzle
// (layout type 4).  Eight tokens are one atom.
template <int D>
__device__ __forceinline__ uint64_t vdesc(uint32_t addr) {
  if (D == 128) return sdesc(addr, 1024, 1024);
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(512 >> 4) << 16) |
         ((uint64_t)(512 >> 4) << 32) | (1ull << 46) | (4ull << 61);
}

template <int D>
__device__ __forceinline__ void rescale_row(uint32_t orow, float alpha) {
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    uint32_t v[32];
    tmem_ld32(orow + c, v);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i)
      v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
    tmem_st32(orow + c, v);
  }
}

// Zeros over what the bf16 pair w has that is not finite; whether it had.
__device__ __forceinline__ bool drop_odd(uint32_t& w) {
  const bool lo = (w & 0x7f80u) == 0x7f80u, hi = (w & 0x7f800000u) == 0x7f800000u;
  if (lo) w &= 0xffff0000u;
  if (hi) w &= 0x0000ffffu;
  return lo || hi;
}

// Arrive on a barrier of a CTA of the cluster; this CTA's writes before it are
// visible to who waits there.
__device__ __forceinline__ void remote_arrive_release(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                   cluster_bar)
               : "memory");
}

__device__ __forceinline__ int next_index(const Params& p, int pairs, int lane) {
  int i = 0;
  if (lane == 0) i = pairs + atomicAdd(p.next, 1);
  return __shfl_sync(0xffffffffu, i, 0);
}

template <int D>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    attention_kernel(const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const Params p) {
  using C = Cfg<D>;
  constexpr int kNS = C::kNS;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  Small<kNS>& sh = *reinterpret_cast<Small<kNS>*>(smem + C::kTiles);
  volatile int* aborted = &sh.aborted;
  volatile int* odd_values = &sh.odd_values;
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
    for (int i = 0; i < kLoads; ++i) mbar_init(smem_u32(&sh.v_raw[i]), 1);
    sh.aborted = 0;
    sh.odd_values = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  __syncwarp();
  if (warp == 8) tc::tmem_alloc2(smem_u32(&sh.tmem_base), kTmemCols);
  fence_before_sync();
  tc::cluster_sync();
  fence_after_sync();
  const uint32_t tmem = sh.tmem_base;
  // Launched while the kernel before runs: nothing of global memory before this.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  auto timed_out = [&](int site) {
    if (!*aborted) record_status(p.status, KV_ERR_TIMEOUT, site);
    atomicExch(&sh.aborted, 1);
    tc::cluster_store4(tc::map_rank(smem_u32(&sh.aborted), rank ^ 1), 1u);
  };
  const int G = p.G, ctok = kM / G;  // tokens of a CTA

  // The pair's items in turn; `tiles0` key tiles came before the item, and its j-th
  // key tile is tile tiles0 + j of the pair's stream, which the stages, barriers
  // and the warpgroups' turns go by.
  struct Items {
    ChunkItem t;
    int h, nt = 0, nblk;
    uint32_t n = 0, tiles0 = 0;  // n: items taken
  } it;
  auto next_item = [&](bool& ok) {
    it.tiles0 += it.nt;
    const uint32_t slot = it.n & 1;
    ok = ok && tc::all_wait_cluster(smem_u32(&sh.item_full[slot]), (it.n >> 1) & 1);
    if (!ok) return false;
    const int4 a = sh.item[slot][0], b = sh.item[slot][1];
    it.t = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, 0};
    it.h = b.w;
    __syncwarp();
    if (lane == 0)
      tc::remote_arrive(tc::map_rank(smem_u32(&sh.item_empty[slot]), 1));
    ++it.n;
    it.nblk = (it.t.pos0 + it.t.ntok + 15) / 16;  // blocks the last row sees
    it.nt = it.t.key_end - it.t.key_begin;
    return it.h >= 0;
  };

  if (warp < 8) {
    // ---- rows: thread = row r, every second key tile ----------------------------
    const int g = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t prow = lane_base + kColP + g * 64;
    const uint32_t orow = lane_base + kColO + g * D;
    const uint32_t s_empty = tc::map_rank(smem_u32(&sh.s_empty), 0);
    const uint32_t p_full = tc::map_rank(smem_u32(&sh.p_full[g]), 0);
    const uint32_t o_empty = tc::map_rank(smem_u32(&sh.o_empty), 0);
    const int tok = rank * ctok + r / G;                   // token of the tile
    const int tok_lo = rank * ctok + (warp & 3) * 32 / G;  // the warp's first
    bool ok = true;
    // All or none go on: they meet at the item's end.
    while (tc::bar_and(1, 256, next_item(ok))) {
      const ChunkItem t = it.t;
      const int nt = it.nt, h = it.h;
      const int pos = t.pos0 + tok;  // this row's position
      const int pos_lo = t.pos0 + tok_lo;
      // Rows of this warp: the CTA's rows are (token, head), tokens first.
      const int rows = min(max(t.ntok - rank * ctok, 0), ctok) * G;
      const int n = rows - (warp & 3) * 32;
      float m_used = -INFINITY, l = 0.f;
      for (int j = (it.tiles0 ^ g) & 1; j < nt; j += 2) {
        const uint32_t q = it.tiles0 + j;
        ok = all_wait(smem_u32(&sh.s_full[g]), (q >> 1) & 1);
        if (!ok) break;
        fence_after_sync();
        if (n <= 0) {
          // None: their P is whatever lies there, and goes to rows nobody stores.
          if (j > 1) ok = all_wait(smem_u32(&sh.p_empty[g]), ((q - 2) >> 1) & 1);
          if (!ok) break;
          if (lane == 0) {
            tc::remote_arrive(s_empty);
            tc::remote_arrive(p_full);
          }
          continue;
        }
        uint32_t u[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(lane_base + c * 32, u[c]);
        tmem_wait_ld();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::remote_arrive(s_empty);  // S may be overwritten
        const int key0 = (t.key_begin + j) * kT;
        const int seen = pos - key0 + 1;        // tokens of the tile this row sees
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        if (pos_lo - key0 + 1 >= kT) {          // every row of the warp: all
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
        if (__any_sync(0xffffffffu, need) && j > 1) rescale_row<D>(orow, alpha);
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
      if (n <= 0) {
        if (lane == 0) tc::remote_arrive(o_empty);
        continue;
      }
      // The two halves of the key tiles joined, that of the item's first tile
      // first: which warpgroup has it depends on the items before, and a fused
      // multiply-add rounds its two products differently.  Each warp D / 2 columns.
      const int a = it.tiles0 & 1;  // the warpgroup of the first tile
      const float m0 = sh.stat[a][0][r], m1 = sh.stat[a ^ 1][0][r];
      const float top = fmaxf(m0, m1);
      // A row may see nothing of a cut range: no weight, and a sum of 0.
      const float e0 = m0 == -INFINITY ? 0.f : ex2(m0 - top);
      const float e1 = m1 == -INFINITY ? 0.f : ex2(m1 - top);
      const float sum = e0 * sh.stat[a][1][r] + e1 * sh.stat[a ^ 1][1][r];
      const bool cut = t.partial >= 0;
      const float inv = cut ? 1.f : 1.f / sum;
      const float w0 = e0 * inv, w1 = e1 * inv;
      const bool has1 = nt > 1;  // an item of one tile has written one O
      const uint32_t o0 = lane_base + kColO + a * D;
      const uint32_t o1 = lane_base + kColO + (a ^ 1) * D;
      uint8_t* turn = smem + C::kOffTurn + warp * 2048;
      // This warp's first row: of the item's partial rows, and as a (token, head).
      const int row_lo = rank * ctok * G + (warp & 3) * 32;
      const int64_t prow_lo = (int64_t)t.partial + (int64_t)h * t.ntok * G + row_lo;
      if (cut && g == 0 && lane < n) p.ml[prow_lo + lane] = make_float2(top, sum);
      const bool odd = *odd_values != 0;
#pragma unroll 1
      for (int c = g * (D / 2); c < (g + 1) * (D / 2); c += 32) {
        uint32_t v[32], v1[32];
        tmem_ld32(o0 + c, v);
        tmem_ld32(o1 + c, v1);
        tmem_wait_ld();
        if (c + 32 == (g + 1) * (D / 2)) {  // O has been read
          fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::remote_arrive(o_empty);
        }
        float x[32];
#pragma unroll
        for (int k = 0; k < 32; ++k)
          x[k] = __uint_as_float(v[k]) * w0 +
                 (has1 ? __uint_as_float(v1[k]) * w1 : 0.f);
        if (odd && lane < n) {
          // Values that are not finite were left out of PV where some row does not
          // see them: added for the rows that do.
          const int end = min(pos + 1, t.key_end * kT);
          for (int key = max(t.pos0 + 1, t.key_begin * kT); key < end; ++key) {
            const int s = p.slots[t.table + key / 16];
            if (s < 0 || s >= p.blocks) continue;
            const __nv_bfloat16* val =
                p.v + (((int64_t)s * p.Hkv + h) * 16 + key % 16) * D + c;
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const float y = __bfloat162float(val[k]);
              if (!isfinite(y)) x[k] += y;
            }
          }
        }
        if (cut) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t w[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) w[k] = __float_as_uint(x[half * 16 + k]);
            put_rows(turn, w, lane, [&](int rr) -> uint8_t* {
              if (rr >= n) return nullptr;
              return reinterpret_cast<uint8_t*>(p.o + (prow_lo + rr) * D + c +
                                                half * 16);
            });
          }
        } else {
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) w[k] = pack_bf16(x[2 * k], x[2 * k + 1]);
          put_rows(turn, w, lane, [&](int rr) -> uint8_t* {
            if (rr >= n) return nullptr;
            const int row = row_lo + rr;
            return reinterpret_cast<uint8_t*>(
                p.out + ((int64_t)(t.row0 + row / G) * p.Hq + h * G + row % G) * D +
                c);
          });
        }
      }
    }
    if (!ok && lane == 0) timed_out(70);
  } else if (warp == 8) {
    bool ok = true;
    if (rank == 0) {
      // ---- products of both CTAs (uniform warp, one lane issues) -----------------
      constexpr uint32_t id_qk = idesc(256, kT, false);
      constexpr uint32_t id_pv = idesc(256, D, true);
      const bool lead = elect_one();
      while (next_item(ok)) {
        const int n = uniform(it.nt), first = uniform(it.t.key_begin);
        const int blocks = uniform(it.nblk) - first * kTB;
        const int masked = uniform(it.t.pos0) + 1;  // tokens every row sees
        const uint32_t t0 = uniform(it.tiles0), item = it.n - 1;
        ok = all_wait(smem_u32(&sh.q_full), item & 1);
        // QK(j) and PV(j - 2) in turn: the rows read S(j) while PV(j - 2) runs.
        for (int j = 0; j < n + 2 && ok; ++j) {
          if (j < n) {
            const uint32_t q = t0 + j, st = q % kNS;
            const uint64_t qd = sdesc(base, 16, 1024);
            const uint64_t kd =
                sdesc(base + C::kOffK + st * C::kK, 16, D == 128 ? 2048 : 1024);
            ok = all_wait(smem_u32(&sh.k_full[st]), (q / kNS) & 1) &&
                 (q == 0 || all_wait(smem_u32(&sh.s_empty), (q - 1) & 1));
            if (!ok) break;
            fence_after_sync();
            if (lead) {
#pragma unroll
              for (int k = 0; k < D / 16; ++k)
                tc::umma2_ss(tmem, qd + (((k >> 2) * 16384 + (k & 3) * 32) >> 4),
                             kd + (((k >> 2) * 1024 + (k & 3) * 32) >> 4), id_qk,
                             k > 0 ? 1u : 0u);
              tc::umma2_commit(smem_u32(&sh.s_full[q & 1]));
              tc::umma2_commit(smem_u32(&sh.k_empty[st]));
              if (j == n - 1) tc::umma2_commit(smem_u32(&sh.q_empty));
            }
            __syncwarp();
          }
          const int i = j - 2;
          if (i >= 0) {
            const uint32_t q = t0 + i, st = q % kNS;
            // Where a load warp has written over V: its writes, of both CTAs.
            ok = ((first + i + 1) * kT > masked
                      ? tc::all_wait_cluster(smem_u32(&sh.v_full[st]), (q / kNS) & 1)
                      : all_wait(smem_u32(&sh.v_full[st]), (q / kNS) & 1)) &&
                 all_wait(smem_u32(&sh.p_full[q & 1]), (q >> 1) & 1) &&
                 (i > 0 || item == 0 ||
                  all_wait(smem_u32(&sh.o_empty), (item - 1) & 1));
            if (!ok) break;
            fence_after_sync();
            if (lead) {
              const uint32_t pcol = tmem + kColP + (q & 1) * 64;
              const uint32_t dout = tmem + kColO + (q & 1) * D;
              const int nb = min(kTB, blocks - i * kTB);
              const uint64_t vd = vdesc<D>(base + C::kOffV + st * C::kV);
#pragma unroll
              for (int k = 0; k < kTB; ++k)
                if (k < nb)
                  tc::umma2_ts(dout, pcol + k * 8, vd + k * (C::kBlkV >> 4), id_pv,
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
        timed_out(71);
        // Every product issued has finished once this lands, or a time has passed.
        tc::umma2_commit(smem_u32(&sh.o_ready));
        mbar_wait(smem_u32(&sh.o_ready), (it.n - 1) & 1);
      }
    } else {
      // ---- the pair's work items (odd CTA): the first by its place in the grid,
      // then as they come.  Head groups in turn (what the pairs read at a time
      // stays in L2), in a group the longest items first.
      const int n_work = p.n_items * p.Hkv, pairs = gridDim.x >> 1;
      int i = blockIdx.x >> 1;
      for (uint32_t n = 0;; ++n) {
        const uint32_t slot = n & 1;
        if (n >= 2) ok = all_wait(smem_u32(&sh.item_empty[slot]), ((n >> 1) - 1) & 1);
        ok = __all_sync(0xffffffffu, ok && !*aborted);
        if (!ok) break;
        ChunkItem t{0, 1, 0, 0, 0, 1, -1, 0};
        int h = -1;
        for (; i < n_work; i = next_index(p, pairs, lane)) {
          const int group = i / (p.n_items * p.heads);
          const int heads = min(p.heads, p.Hkv - group * p.heads);
          const int rest = i - group * p.n_items * p.heads;
          t = p.items[rest / heads];
          h = group * p.heads + rest % heads;
          if (t.ntok >= 1 && t.ntok <= 2 * ctok && t.pos0 >= 0 &&
              t.pos0 <= (1 << 30) && t.row0 >= 0 && t.row0 <= p.total - t.ntok &&
              t.table >= 0 &&
              (int64_t)t.table + (t.pos0 + t.ntok + 15) / 16 <= p.n_slots &&
              t.key_begin >= 0 && t.key_begin < t.key_end &&
              t.key_end <= (t.pos0 + t.ntok - 1) / kT + 1 &&
              (t.partial < 0 ||
               (int64_t)t.partial + (int64_t)t.ntok * p.Hq <= p.partial_rows))
            break;
          if (lane == 0) record_status(p.status, KV_ERR_DEVICE, -1 - i);
          h = -1;
        }
        if (lane < 2) {
          const uint32_t bar = tc::map_rank(smem_u32(&sh.item_full[slot]), lane);
          const uint32_t to = tc::map_rank(smem_u32(&sh.item[slot]), lane);
          tc::remote_expect_tx(bar, 32);
          tc::remote_store16(to, t.row0, t.ntok, t.pos0, t.table, bar);
          tc::remote_store16(to + 16, t.key_begin, t.key_end, t.partial, h, bar);
        }
        __syncwarp();
        if (h < 0) break;
        i = next_index(p, pairs, lane);
      }
      if (!ok && lane == 0) timed_out(75);
    }
  } else {
    // ---- loads of this CTA's halves: its rows of Q, half of a key tile's keys,
    // half of the values' columns; a warp takes every third key tile --------------
    const int me = warp - 9;
    const uint32_t raw = smem_u32(&sh.v_raw[me]);
    uint32_t n_raw = 0;
    bool ok = true;
    // Widened blocks were stored by a kernel before, read by bulk copies here.
    asm volatile("fence.proxy.async;" ::: "memory");
    // Lanes 0-3 the half's keys, 8-15 values.
    const int bi = lane < 8 ? rank * 4 + (lane & 3) : lane & 7;
    while (next_item(ok)) {
      const int nt = it.nt, h = it.h;
      const uint32_t item = it.n - 1;
      if (me == 0) {
        if (item > 0) ok = all_wait(smem_u32(&sh.q_empty), (item - 1) & 1);
        ok = __all_sync(0xffffffffu, ok && !*aborted);
        if (!ok) break;
        const uint32_t bar = tc::map_rank(smem_u32(&sh.q_full), 0);
        if (lane == 0) tc::remote_expect_tx(bar, D / 64 * ctok * G * 128);
        __syncwarp();
        if (lane < D / 64)
          tc::tma2_load_3d(base + lane * 16384, &tmQ, lane * 64, h * G,
                           it.t.row0 + rank * ctok, bar);
        __syncwarp();
      }
      auto slot_of = [&](int tile) {
        const int blk = (it.t.key_begin + tile) * kTB + bi;
        if ((lane >= 4 && lane < 8) || lane >= 16 || tile >= nt || blk >= it.nblk)
          return -1;
        const int s = p.slots[it.t.table + blk];
        if (s >= 0 && s < p.blocks) return s;
        record_status(p.status, KV_ERR_DEVICE, s);
        return -1;
      };
      int j = (me + kLoads - (int)(it.tiles0 % kLoads)) % kLoads;
      int next = slot_of(j);
      for (; j < nt; j += kLoads) {
        const int slot = next;
        next = slot_of(j + kLoads);
        const bool load = slot >= 0;
        const uint32_t act = __ballot_sync(0xffffffffu, load);
        const uint32_t q = it.tiles0 + j, s = q % kNS;
        const uint32_t kbar = tc::map_rank(smem_u32(&sh.k_full[s]), 0);
        const uint32_t vbar = tc::map_rank(smem_u32(&sh.v_full[s]), 0);
        if (q >= kNS) ok = all_wait(smem_u32(&sh.k_empty[s]), (q / kNS - 1) & 1);
        ok = __all_sync(0xffffffffu, ok && !*aborted);
        if (!ok) break;
        if (lane == 0) tc::remote_expect_tx(kbar, __popc(act & 0xf) * C::kBlkK);
        __syncwarp();
        if (load && lane < 4) {
          const uint32_t dst = base + C::kOffK + s * C::kK + lane * C::kBlkK;
          if (D == 128)
            tc::tma2_load_5d_at(dst, &tmK, 0, slot * p.Hkv + h, kbar);
          else
            tc::tma2_load_2d(dst, &tmK, 0, (slot * p.Hkv + h) * 16, kbar);
        }
        __syncwarp();
        if (q >= kNS) ok = all_wait(smem_u32(&sh.v_empty[s]), (q / kNS - 1) & 1);
        ok = __all_sync(0xffffffffu, ok && !*aborted);
        if (!ok) break;
        // Tokens of the tile that every row of the item sees.
        const int key0 = (it.t.key_begin + j) * kT;
        const int whole = it.t.pos0 + 1 - key0;
        const bool masked = whole < kT;
        const uint32_t bar = masked ? tc::map_rank(raw, rank) : vbar;
        if (lane == 0) tc::remote_expect_tx(bar, __popc(act >> 8) * C::kBlkV);
        __syncwarp();
        const uint32_t vst = base + C::kOffV + s * C::kV;
        if (load && lane >= 8) {
          const uint32_t dst = vst + bi * C::kBlkV;
          if (D == 128)
            tc::tma2_load_5d_at(dst, &tmV, rank, slot * p.Hkv + h, bar);
          else
            tc::tma2_load_2d(dst, &tmV, rank * 32, (slot * p.Hkv + h) * 16, bar);
        }
        __syncwarp();
        if (!masked) continue;
        ok = all_wait(raw, n_raw++ & 1);
        if (!ok) break;
        // Rows of D bytes, half of a token's values (in the swizzle's order).
        const int rows = min(kTB, it.nblk - key0 / 16) * 16;
        const int len = it.t.pos0 + it.t.ntok - key0;  // tokens that a row sees
        bool odd = false;
        for (int k = max(whole, 0) * (D / 16) + lane; k < rows * (D / 16); k += 32) {
          uint4* x = reinterpret_cast<uint4*>(smem + C::kOffV + s * C::kV + k * 16);
          if (k / (D / 16) >= len) {
            *x = make_uint4(0, 0, 0, 0);
            continue;
          }
          uint4 y = *x;
          bool here = drop_odd(y.x);
          here |= drop_odd(y.y);
          here |= drop_odd(y.z);
          here |= drop_odd(y.w);
          if (here) *x = y;
          odd |= here;
        }
        odd = __any_sync(0xffffffffu, odd);
        if (odd && lane < 2)
          tc::cluster_store4(tc::map_rank(smem_u32(&sh.odd_values), lane), 1u);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) remote_arrive_release(vbar);
      }
    }
    if (!ok && lane == 0) timed_out(72);
  }
  __syncwarp();
  fence_before_sync();
  __syncthreads();
  if (*aborted) tc::wait_for_copies();
  __syncwarp();
  tc::cluster_sync();
  fence_after_sync();
  if (warp == 8) tc::tmem_free2(tmem, kTmemCols);
  tc::cluster_sync();  // neither CTA leaves before both have given it back
}

// Joins the partial rows of cut tiles: a warp for each (token, head).
template <int D>
__global__ void __launch_bounds__(256) join_kernel(const ChunkMerge* merges,
                                                   const Params p) {
  constexpr int V = D / 32;  // values per lane
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const ChunkMerge m = merges[blockIdx.x];
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.y * 8 + (threadIdx.x >> 5);  // (head, token, head of G)
  const int64_t stride = (int64_t)m.ntok * p.Hq;
  if (m.ntok < 1 || m.row0 < 0 || m.row0 > p.total - m.ntok || m.pieces < 1 ||
      m.partial < 0 || m.partial + stride * m.pieces > p.partial_rows) {
    if (row == 0 && lane == 0) record_status(p.status, KV_ERR_DEVICE, m.partial);
    return;
  }
  if (row >= stride) return;
  const int h = row / (m.ntok * p.G), rest = row % (m.ntok * p.G);
  float top = -INFINITY, sum = 0.f, acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
  for (int k = 0; k < m.pieces; ++k) {
    const int64_t at = m.partial + k * stride + row;
    const float2 ml = p.ml[at];
    float v[V];
#pragma unroll
    for (int i = 0; i < V; i += 2)
      *reinterpret_cast<float2*>(v + i) =
          *reinterpret_cast<const float2*>(p.o + at * D + lane * V + i);
    const float m_new = fmaxf(top, ml.x);
    const float a = top == -INFINITY ? 0.f : ex2(top - m_new);
    const float w = ml.x == -INFINITY ? 0.f : ex2(ml.x - m_new);
    sum = sum * a + w * ml.y;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = acc[i] * a + w * v[i];
    top = m_new;
  }
  const float inv = 1.f / sum;
  __nv_bfloat16* dst =
      p.out +
      ((int64_t)(m.row0 + rest / p.G) * p.Hq + h * p.G + rest % p.G) * D + lane * V;
#pragma unroll
  for (int i = 0; i < V; i += 2)
    *reinterpret_cast<uint32_t*>(dst + i) =
        pack_bf16(acc[i] * inv, acc[i + 1] * inv);
}

// An e4m3 step's distinct blocks as bf16 [slot][Hkv][16][D], a warp for each
// (slot, head).  Exact: a code has 4 significant bits, its scale is a power of two.
template <int D>
__global__ void __launch_bounds__(256)
    widen_kernel(const uint8_t* k8, const uint8_t* v8, const float4* scales,
                 const int32_t* uniq, int n_uniq, int Hkv, int64_t num_blocks,
                 __nv_bfloat16* k, __nv_bfloat16* v, DeviceStatus* status) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int w = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (w >= n_uniq * Hkv) return;
  const int phys = uniq[w / Hkv];
  if (phys < 0 || phys >= num_blocks) {
    if (lane == 0) record_status(status, KV_ERR_DEVICE, phys);
    return;
  }
  const int64_t src = (int64_t)phys * Hkv + w % Hkv;
  const float4 scale = scales[src];
  constexpr int kChunks = D / 16;  // 16-byte chunks of a row of K
#pragma unroll
  for (int i = 0; i < kChunks / 2; ++i) {
    const int n = i * 32 + lane, t = n / kChunks, c = n % kChunks;
    const int at = D == 128 ? t * 128 + ((c ^ (t & 7)) << 4) : n * 16;
    const uint4 x = *reinterpret_cast<const uint4*>(k8 + src * (16 * D) + at);
    const uint32_t in[4] = {x.x, x.y, x.z, x.w};
    uint32_t y[8];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      uint32_t h[2];
      e4m3x4_to_f16x2x2(in[b], h[0], h[1]);
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const float2 f = __half22float2(*reinterpret_cast<__half2*>(&h[z]));
        y[2 * b + z] = pack_bf16(f.x * scale.x, f.y * scale.x);
      }
    }
    uint4* dst = reinterpret_cast<uint4*>(k + ((int64_t)w * 16 + t) * D + c * 16);
    dst[0] = make_uint4(y[0], y[1], y[2], y[3]);
    dst[1] = make_uint4(y[4], y[5], y[6], y[7]);
  }
  // V: a row of 16 tokens per dimension; two dimensions a lane.
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    const int c = i * 64 + lane * 2;
    float f[2][16];
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const uint4 x =
          *reinterpret_cast<const uint4*>(v8 + src * (16 * D) + (c + z) * 16);
      const uint32_t in[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        uint32_t h[2];
        e4m3x4_to_f16x2x2(in[b], h[0], h[1]);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float2 y = __half22float2(*reinterpret_cast<__half2*>(&h[u]));
          f[z][4 * b + 2 * u] = y.x * scale.y;
          f[z][4 * b + 2 * u + 1] = y.y * scale.y;
        }
      }
    }
#pragma unroll
    for (int t = 0; t < 16; ++t)
      *reinterpret_cast<uint32_t*>(v + ((int64_t)w * 16 + t) * D + c) =
          pack_bf16(f[0][t], f[1][t]);
  }
}

// ---- host side ------------------------------------------------------------------

__global__ void clear_kernel(DeviceStatus* status, int* next) {
  if (threadIdx.x != 0) return;
  *status = DeviceStatus{};
  *next = 0;
}

// Queries [total][Hq][D], `stride` values between tokens: boxes of the G heads of
// a kv-head for the tokens of a CTA, 64 values wide.
kv_status make_query_map(CUtensorMap* tm, const void* q, int64_t stride,
                         int64_t total, int Hq, int G, int d) {
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)Hq, (cuuint64_t)total};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)(kM / G)};
  return encode_bf16_map(tm, q, 3, dims, strides, box);
}

// A pool's (block, head) tiles [16][128] (decode.cu's view): all of a tile's
// columns (halves = 2, four atoms of 8 rows x 64 columns: rows 0-7 half 0, half 1,
// rows 8-15) or one half of them (rows 0-7, 8-15).
kv_status make_tile_map(CUtensorMap* tm, const void* pool, int64_t tiles, int halves) {
  const cuuint64_t dims[5] = {64, 8, 2, 2, (cuuint64_t)tiles};
  const cuuint64_t strides[4] = {256, 128, 2048, 4096};
  const cuuint32_t box[5] = {64, 8, (cuuint32_t)halves, 2, 1};
  return encode_bf16_map(tm, pool, 5, dims, strides, box);
}

// Tiles [16][64]: boxes of 16 rows, all columns or half of them.
kv_status make_row_map(CUtensorMap* tm, const void* pool, int64_t tiles, int width) {
  const cuuint64_t dims[2] = {64, (cuuint64_t)tiles * 16};
  const cuuint64_t strides[1] = {128};
  const cuuint32_t box[2] = {(cuuint32_t)width, 16};
  return encode_bf16_map(
      tm, pool, 2, dims, strides, box,
      width == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

template <int D>
cudaError_t launch(const CUtensorMap& tq, const CUtensorMap& tk,
                   const CUtensorMap& tv, const Params& p, const ChunkMerge* merges,
                   int n_merges, int pairs, cudaStream_t st) {
  static std::atomic<uint64_t> opted{0};
  cudaError_t e = opt_in_smem(attention_kernel<D>, smem_bytes<D>(), opted);
  if (e != cudaSuccess) return e;
  e = launch_early(attention_kernel<D>, 2 * pairs, kThreads, smem_bytes<D>(), st, tq,
                   tk, tv, p);
  if (e != cudaSuccess || n_merges == 0) return e;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)n_merges,
                     (unsigned)((2 * (kM / p.G) * (int64_t)p.Hq + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<D>, merges, p);
}

kv_status run(const void* q, int64_t q_stride, const void* k_pool,
              const void* v_pool, const void* kv_scales, bool e4m3,
              int64_t num_blocks, int32_t total, int32_t nb, int32_t Hq,
              int32_t Hkv, int32_t d, int32_t block_size, float scale, void* out,
              const int32_t* plan, const kv_decode_plan_info* info,
              void* workspace, size_t ws_bytes, void* stream) {
  // A step without queries may have empty tensors, which have no address.
  if (!info || !plan || !workspace || !k_pool || !v_pool || (e4m3 && !kv_scales) ||
      (total != 0 && (!q || !out)))
    return fail(KV_ERR_INVALID_ARG, "null argument");
  if (kv_status s = chunk_heads_ok(Hq, Hkv, d)) return s;
  if (nb < 1 || total < 0) return fail(KV_ERR_INVALID_ARG, "bad nb/total");
  if (block_size != 16) return fail(KV_ERR_INVALID_ARG, "block_size must be 16");
  if (num_blocks < 1 || num_blocks > (int64_t)INT32_MAX / 16 / Hkv)
    return fail(KV_ERR_INVALID_ARG, "num_blocks out of range");
  if (((uintptr_t)q | (uintptr_t)k_pool | (uintptr_t)v_pool | (uintptr_t)kv_scales |
       (uintptr_t)out) & 15)
    return fail(KV_ERR_INVALID_ARG, "q, pools, scales and out must be 16-byte "
                                    "aligned");
  if (total > 0 && (q_stride < (int64_t)Hq * d || q_stride % 8 != 0 ||
                    q_stride >= (1ll << 38)))
    return fail(KV_ERR_INVALID_ARG, "q_stride must be a multiple of 8 and no less "
                                    "than a token's row");
  if ((uintptr_t)workspace & 255)
    return fail(KV_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if (!std::isfinite(scale) || !(scale > 0.f))
    return fail(KV_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (info->flags != (kChunkPlan | (e4m3 ? KV_PLAN_KV_E4M3 : 0)))
    return fail(KV_ERR_INVALID_ARG, "the plan is not one of paged_chunk_plan for "
                                    "%s pool", e4m3 ? "an e4m3" : "a bf16");
  if (info->latent_rows != chunk_mark(Hq, Hkv, d) || info->n_merge_rows != total ||
      info->n_row_items < 0 || info->n_tile_items < 0 || info->n_row_warp_items < 0 ||
      info->n_tile_wide_items < 0 || info->partial_rows < 0 ||
      info->partial_rows > INT32_MAX || (total > 0) != (info->n_tile_items > 0) ||
      (e4m3 && total > 0) != (info->n_row_items > 0) ||
      (int64_t)info->n_tile_items * Hkv > INT32_MAX / 2 ||
      (int64_t)info->n_row_items * Hkv > INT32_MAX / 16 ||
      (info->n_tile_wide_items > 0) != (info->partial_rows > 0))
    return fail(KV_ERR_INVALID_ARG, "plan info does not match the step");
  const size_t need = chunk_workspace(info->partial_rows, info->n_row_items, Hkv, d);
  if (ws_bytes < need || (size_t)info->workspace_bytes != need)
    return fail(KV_ERR_INVALID_ARG, "workspace %zu bytes < %zu needed", ws_bytes,
                need);
  auto* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t st = (cudaStream_t)stream;
  Params p;
  p.status = reinterpret_cast<DeviceStatus*>(ws);
  p.next = reinterpret_cast<int*>(ws + sizeof(DeviceStatus));
  CUtensorMap tq, tk, tv;
  const int U = info->n_row_items;
  auto* wide = ws + ws_total(info->partial_rows, d);
  const void* k = e4m3 ? wide : k_pool;
  const void* v = e4m3 ? wide + chunk_half(U, Hkv, d) : v_pool;
  p.blocks = e4m3 ? U : num_blocks;
  if (total > 0) {
    if (kv_status s = make_query_map(&tq, q, q_stride, total, Hq, Hq / Hkv, d))
      return s;
    const int64_t tiles = p.blocks * Hkv;
    if (kv_status s = d == 128 ? make_tile_map(&tk, k, tiles, 2)
                               : make_row_map(&tk, k, tiles, 64))
      return s;
    if (kv_status s = d == 128 ? make_tile_map(&tv, v, tiles, 1)
                               : make_row_map(&tv, v, tiles, 32))
      return s;
  }
  int dev = 0, sms = 152;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess)
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess)
    return fail(KV_ERR_CUDA, "chunk attention: %s", cudaGetErrorString(e));
  clear_kernel<<<1, 32, 0, st>>>(p.status, p.next);
  e = cudaGetLastError();
  if (e != cudaSuccess)
    return fail(KV_ERR_CUDA, "chunk attention: %s", cudaGetErrorString(e));
  if (total == 0) return KV_OK;
  p.slots = plan + kPlanHeaderInts + U;
  p.n_slots = info->n_row_warp_items;
  p.items = reinterpret_cast<const ChunkItem*>(p.slots + p.n_slots);
  p.n_items = info->n_tile_items;
  const auto* merges = reinterpret_cast<const ChunkMerge*>(p.items + p.n_items);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.ml = reinterpret_cast<float2*>(ws + ws_ml_offset());
  p.o = reinterpret_cast<float*>(ws + ws_o_offset(info->partial_rows));
  p.partial_rows = info->partial_rows;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.total = total;
  p.scale_log2 = scale * 1.4426950408889634f;
  // Heads whose keys and values the pairs share L2 for (shared blocks count as
  // often as branches hold them).
  p.heads = (int)std::clamp<int64_t>((48ll << 20) / ((int64_t)p.n_slots * 16 * d * 4),
                                     1, Hkv);
  if (e4m3) {
    const int ctas = (U * Hkv + 7) / 8;
    auto* k8 = static_cast<const uint8_t*>(k_pool);
    auto* v8 = static_cast<const uint8_t*>(v_pool);
    auto* sc = static_cast<const float4*>(kv_scales);
    const int32_t* uniq = plan + kPlanHeaderInts;
    auto* kw = reinterpret_cast<__nv_bfloat16*>(wide);
    auto* vw = const_cast<__nv_bfloat16*>(p.v);
    e = d == 128 ? launch_early(widen_kernel<128>, ctas, 256, 0, st, k8, v8, sc, uniq,
                                U, Hkv, num_blocks, kw, vw, p.status)
                 : launch_early(widen_kernel<64>, ctas, 256, 0, st, k8, v8, sc, uniq,
                                U, Hkv, num_blocks, kw, vw, p.status);
    if (e != cudaSuccess)
      return fail(KV_ERR_CUDA, "widening kernel: %s", cudaGetErrorString(e));
  }
  const int pairs = (int)std::min<int64_t>((int64_t)p.n_items * Hkv,
                                           std::max(sms / 2, 1));
  e = d == 128 ? launch<128>(tq, tk, tv, p, merges, info->n_tile_wide_items, pairs, st)
               : launch<64>(tq, tk, tv, p, merges, info->n_tile_wide_items, pairs, st);
  if (e != cudaSuccess)
    return fail(KV_ERR_CUDA, "chunk attention: %s", cudaGetErrorString(e));
  return KV_OK;
}

}  // namespace chunk
}  // namespace pkv

extern "C" kv_status paged_chunk_attn(
    const void* q, int64_t q_stride, const void* k_pool, const void* v_pool,
    int64_t num_blocks, int32_t total, int32_t nb, int32_t Hq, int32_t Hkv,
    int32_t head_dim, int32_t block_size, float scale, void* out,
    const int32_t* plan, const kv_decode_plan_info* info, void* workspace,
    size_t ws_bytes, void* stream) {
  pkv::clear_error();
  return pkv::chunk::run(q, q_stride, k_pool, v_pool, nullptr, false, num_blocks,
                         total, nb, Hq, Hkv, head_dim, block_size, scale, out, plan,
                         info, workspace, ws_bytes, stream);
}

extern "C" kv_status paged_chunk_attn_e4m3(
    const void* q, int64_t q_stride, const void* k_pool, const void* v_pool,
    const void* kv_scales, int64_t num_blocks, int32_t total, int32_t nb, int32_t Hq,
    int32_t Hkv, int32_t head_dim, int32_t block_size, float scale, void* out,
    const int32_t* plan, const kv_decode_plan_info* info, void* workspace,
    size_t ws_bytes, void* stream) {
  pkv::clear_error();
  return pkv::chunk::run(q, q_stride, k_pool, v_pool, kv_scales, true, num_blocks,
                         total, nb, Hq, Hkv, head_dim, block_size, scale, out, plan,
                         info, workspace, ws_bytes, stream);
}
