// Chunk attention (paged_chunk_attn): new tokens attend causally to all cached
// tokens of their branch,
//   out[i][h] = sum_{t <= pos(i)} softmax_t(scale q[i][h] . K[t][h / G]) V[t][h / G],
// K and V in the paged pool.  4 D flops for each query head and visible token; a
// prompt or a chunk is bound by the products, a few drafted tokens on long
// branches by the K and V bytes.
//
// Persistent CTAs take work items as they come: a tile of query tokens with the G
// heads of a kv-head, and a range of key tiles.  Rows are packed (token, head), so
// that a kv-head's keys are loaded once for all of its heads and single tokens fill G
// rows: a CTA has floor(128 / G) tokens.  Items of more tokens than that run on pairs
// of CTAs (cta_group::2), one on every two SMs, that each load half of every key tile
// of 128 tokens (64 tokens of K, half of V's columns); items of no more, on which
// the second CTA would have nothing to do, on single CTAs.  A step with both kinds
// has the second kernel fill the SMs that the first leaves.  K and V tiles come in
// through TMA as they lie in the pool, a box per block, and land in the layouts the
// products take.
//
// The rows' two warpgroups take the key tiles in turn.  TMEM: S of the two (2 x 128
// columns), P of the two (2 x 64, bf16 pairs), O (D).  Both add to one O, relative to
// one lazy maximum a row, which they hand each other tile by tile; O is rescaled
// where it grows by more than 8 (log2 units), after the product before.  The softmax
// of a tile (a thread a row, base 2, two columns to an instruction) takes about two
// tiles' time, beside the other warpgroup's.  (With an O and a maximum for each
// warpgroup there was room for one S alone, and QK(j + 1) waited for S(j) to be
// read: 1430 cycles a tile of 256 rows, 1024 of them products.)
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
  int* next;              // work items handed out past the first ones
  int n_slots, n_items, Hq, Hkv, G, total, heads;  // heads of a group
  bool beside;            // single CTAs that run beside the pairs
  int64_t blocks;         // blocks the slots may name
  int64_t partial_rows;
  float scale_log2;
};

constexpr int kT = kChunkKeys, kTB = kT / 16;  // tokens and blocks of a key tile
constexpr int kM = kChunkRows;                 // query rows of a CTA
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColP = 256, kColO = 384;   // TMEM: S (2), P (2), O
constexpr float kRescale = 8.f;                // lazy-max threshold (log2 units)

// Warps 0 scores, 1 O, 2, 3 and 14 loads, 4-11 rows, 12 work items (of the odd CTA), 13
// values that are masked.  Scores and O are issued by a warp each: few products fit
// between a warp and the tensor unit, so that one warp's waits for K, V, S and P (some
// 130 cycles each beside the rows' exponentials, when they are there already) leave the
// unit idle: 1550 cycles a tile of 128 rows a CTA, 1024 of them products.  The rows
// take registers from the others: 256 x 184 and 256 x 72 are the 512 x 128 of the
// launch.
constexpr int kThreads = 16 * 32;
constexpr int kRowRegs = 184, kOtherRegs = 72;

// kCtas: CTAs of an item.
template <int D, int kCtas>
struct Cfg {
  static constexpr int kQ = D / 64 * kM * 128;   // Q: 64-wide parts, double-buffered
  static constexpr int kQs = kCtas == 2 || D == 64 ? 2 : 1;
  static constexpr int kBlkK = 16 * D * 2;       // a block's keys of a head
  static constexpr int kK = kTB / kCtas * kBlkK; // a K stage
  static constexpr int kBlkV = 16 * D * 2 / kCtas;  // a block's values, a CTA's columns
  static constexpr int kV = kTB * kBlkV;         // a V stage
  static constexpr int kRowV = D * 2 / kCtas;    // bytes of a token in it
  static constexpr int kNK = D == 64 ? (kCtas == 2 ? 8 : 6) : (kCtas == 2 ? 5 : 3);
  static constexpr int kNV = kNK;
  // Load warps.  A warp has waited for the stage of the tile kLoads before its own
  // to be empty; with no fewer stages than warps, a wait is never two phases ahead of
  // its barrier, whose parity would then pass for the one waited for.
  static constexpr int kLoads = kNV < 3 ? kNV : 3;
  static constexpr int kOffK = kQs * kQ;
  static constexpr int kOffV = kOffK + kNK * kK;
  static constexpr int kTiles = kOffV + kNV * kV;
  // A row of V's 16 bytes, in the swizzle's order: block, 8 tokens, (half of the
  // columns,) token.
  __device__ static __forceinline__ int v_at(int row, int c) {
    return kRowV == 256
               ? (row >> 3) * 2048 + (c >> 3) * 1024 + (row & 7) * 128 + (c & 7) * 16
               : row * kRowV + c * 16;
  }
};

static_assert(Cfg<128, 1>::kLoads <= Cfg<128, 1>::kNK, "stages of K and load warps");

template <typename C>
struct Small {
  // Pairs: q_full, k_full, v_full and o_empty are used in the even CTA alone,
  // item_empty in the odd one; v_raw and m_full are the CTA's own.  k_full: K has
  // landed and the rows have read what is in its S; v_full: V has landed and the rows
  // have written P.
  uint64_t q_full[2], q_empty[2], k_full[C::kNK], k_empty[C::kNK], v_full[C::kNV],
      v_empty[C::kNV], s_full[2], p_empty[2], o_ready, o_empty, item_full[2],
      item_empty[2], v_raw[C::kNV], m_full[2][4], drain[2];
  int4 item[2][2];       // ChunkItem, its pad the head (-1: no more)
  float top[2][kM];      // the rows' maximum after a tile of each warpgroup
  float sum[2][kM];      // and at an item's end the sum relative to it
  uint32_t tmem_base;
  int aborted;
  int odd_values;        // a masked tile held a value that is not finite
};

template <int D, int kCtas>
constexpr int smem_bytes() {
  return Cfg<D, kCtas>::kTiles + (int)sizeof(Small<Cfg<D, kCtas>>);
}
static_assert(smem_bytes<128, 2>() <= 227 * 1024, "shared memory of a CTA");
static_assert(smem_bytes<64, 2>() <= 227 * 1024, "shared memory of a CTA");
static_assert(smem_bytes<128, 1>() <= 227 * 1024, "shared memory of a CTA");
static_assert(smem_bytes<64, 1>() <= 227 * 1024, "shared memory of a CTA");

// V as an MN-major operand, eight tokens an atom.  A CTA's 128 columns: two atoms of
// 64 side by side; 64: rows of 128 bytes with 128-byte swizzle; 32: rows of 64 bytes
// with 64-byte swizzle (layout type 4).
template <int kRowV>
__device__ __forceinline__ uint64_t vdesc(uint32_t addr) {
  if (kRowV == 256) return sdesc(addr, 1024, 2048);
  if (kRowV == 128) return sdesc(addr, 1024, 1024);
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

// The forms of one CTA and of a pair.
template <int kCtas>
__device__ __forceinline__ void commit(uint32_t bar) {
  if (kCtas == 2) tc::umma2_commit(bar); else tc::umma_commit(bar);
}
template <int kCtas>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id,
                                       uint32_t acc) {
  if (kCtas == 2) tc::umma2_ss(d, a, b, id, acc); else tc::umma_ss(d, a, b, id, acc);
}
template <int kCtas>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id,
                                       uint32_t acc) {
  if (kCtas == 2) tc::umma2_ts(d, a, b, id, acc); else tc::umma_ts(d, a, b, id, acc);
}
template <int kCtas>
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap* tm, int x,
                                        int y, uint32_t bar) {
  if (kCtas == 2) tc::tma2_load_2d(dst, tm, x, y, bar);
  else tma_load_2d(dst, tm, x, y, bar);
}
template <int kCtas>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* tm, int half,
                                          int tile, uint32_t bar) {
  if (kCtas == 2) tc::tma2_load_5d_at(dst, tm, half, tile, bar);
  else tc::tma_load_5d_at(dst, tm, half, tile, bar);
}
template <int kCtas>
__device__ __forceinline__ void load_3d(uint32_t dst, const CUtensorMap* tm, int x,
                                        int y, int z, uint32_t bar) {
  if (kCtas == 2) {
    tc::tma2_load_3d(dst, tm, x, y, z, bar);
  } else {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::"
        "bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(tm), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
  }
}

// Whether the phase with the given parity has completed.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Warp-wide wait for one barrier, and where `second` for another, asked together.
__device__ __forceinline__ bool both_wait(uint32_t bar0, uint32_t parity0,
                                          uint32_t bar1, uint32_t parity1,
                                          bool second) {
  const bool a = mbar_test(bar0, parity0);
  const bool b = !second || mbar_test(bar1, parity1);
  if (__all_sync(0xffffffffu, a && b)) return true;
  return all_wait(bar0, parity0) && (!second || all_wait(bar1, parity1));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// A place of shared memory in CTA `rank` of the item's.
template <int kCtas>
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
  return kCtas == 2 ? tc::map_rank(addr, rank) : addr;
}

template <int D, int kCtas>
__global__ void __launch_bounds__(kThreads, 1)
    attention_kernel(const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const Params p) {
  using C = Cfg<D, kCtas>;
  constexpr int kLoads = C::kLoads, kNK = C::kNK, kNV = C::kNV, kQs = C::kQs;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  Small<C>& sh = *reinterpret_cast<Small<C>*>(smem + C::kTiles);
  volatile int* aborted = &sh.aborted;
  volatile int* odd_values = &sh.odd_values;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (base & 1023) {  // never, with no static shared memory
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (threadIdx.x == 0) record_status(p.status, KV_ERR_INTERNAL, (int)base);
    return;
  }
  const int rank = kCtas == 2 ? (int)tc::cluster_rank() : 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh.q_full[i]), kCtas);
      mbar_init(smem_u32(&sh.q_empty[i]), 1);
      mbar_init(smem_u32(&sh.s_full[i]), 1);
      mbar_init(smem_u32(&sh.p_empty[i]), 1);
      mbar_init(smem_u32(&sh.drain[i]), 1);
      mbar_init(smem_u32(&sh.item_full[i]), 1);
      mbar_init(smem_u32(&sh.item_empty[i]), kCtas * (8 + kLoads + 1) + 2);
      for (int w = 0; w < 4; ++w) mbar_init(smem_u32(&sh.m_full[i][w]), 1);
    }
    for (int s = 0; s < kNK; ++s) {
      mbar_init(smem_u32(&sh.k_full[s]), 5 * kCtas);
      mbar_init(smem_u32(&sh.k_empty[s]), 1);
    }
    for (int s = 0; s < kNV; ++s) {
      mbar_init(smem_u32(&sh.v_full[s]), 5 * kCtas);
      mbar_init(smem_u32(&sh.v_empty[s]), 1);
      mbar_init(smem_u32(&sh.v_raw[s]), 1);
    }
    mbar_init(smem_u32(&sh.o_ready), 1);
    mbar_init(smem_u32(&sh.o_empty), 8 * kCtas);
    sh.aborted = 0;
    sh.odd_values = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  __syncwarp();
  if (warp == 0) {
    if (kCtas == 2) {
      tc::tmem_alloc2(smem_u32(&sh.tmem_base), kTmemCols);
    } else {
      asm volatile(
          "tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
              smem_u32(&sh.tmem_base)),
          "r"(kTmemCols)
          : "memory");
      asm volatile(
          "tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
  }
  fence_before_sync();
  tc::cluster_sync();
  fence_after_sync();
  const uint32_t tmem = sh.tmem_base;
  // Launched while the kernel before runs: nothing of global memory before this.
  // (A single CTA beside the pairs needs nothing of theirs, and starts after what
  // they have waited for: it waits for them at its end.)
  if (!p.beside) asm volatile("griddepcontrol.wait;" ::: "memory");
  if (kCtas == 2) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  auto timed_out = [&](int site) {
    if (!*aborted) record_status(p.status, KV_ERR_TIMEOUT, site);
    atomicExch(&sh.aborted, 1);
    if (kCtas == 2)
      tc::cluster_store4(in_cta<kCtas>(smem_u32(&sh.aborted), rank ^ 1), 1u);
  };
  const int G = p.G, ctok = kM / G;  // tokens of a CTA

  // The items in turn; `tiles0` key tiles came before the item, and its j-th key tile
  // is tile tiles0 + j of the stream, which the stages, barriers and the warpgroups'
  // turns go by.
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
      tc::remote_arrive(in_cta<kCtas>(smem_u32(&sh.item_empty[slot]), kCtas - 1));
    ++it.n;
    it.nblk = (it.t.pos0 + it.t.ntok + 15) / 16;  // blocks the last row sees
    it.nt = it.t.key_end - it.t.key_begin;
    return it.h >= 0;
  };

  if (warp >= 4 && warp < 12) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRowRegs));
    // ---- rows: thread = row r, every second key tile ----------------------------
    const int g = (warp >> 2) - 1, w4 = warp & 3;
    const int r = w4 * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)(w4 * 32) << 16);
    const uint32_t srow = lane_base + g * kT;
    const uint32_t prow = lane_base + kColP + g * 64;
    const uint32_t orow = lane_base + kColO;
    const uint32_t k_full = in_cta<kCtas>(smem_u32(&sh.k_full[0]), 0);
    const uint32_t v_full = in_cta<kCtas>(smem_u32(&sh.v_full[0]), 0);
    const uint32_t o_empty = in_cta<kCtas>(smem_u32(&sh.o_empty), 0);
    const int tok = rank * ctok + r / G;              // token of the tile
    const int tok_lo = rank * ctok + w4 * 32 / G;     // the warp's first
    bool ok = true;
    // S holds nothing yet.
    if (lane == 0) tc::remote_arrive(k_full + g * 8);
    // All or none go on: they meet at the item's end.
    while (tc::bar_and(1, 256, next_item(ok))) {
      const ChunkItem t = it.t;
      const int nt = it.nt, h = it.h;
      const int pos = t.pos0 + tok;  // this row's position
      const int pos_lo = t.pos0 + tok_lo;
      // Rows of this warp: the CTA's rows are (token, head), tokens first.
      const int rows = min(max(t.ntok - rank * ctok, 0), ctok) * G;
      const int n = rows - w4 * 32;
      float m_own = -INFINITY, l = 0.f;  // the sum, relative to this maximum
      for (int j = (it.tiles0 ^ g) & 1; j < nt; j += 2) {
        const uint32_t q = it.tiles0 + j;
        // S, and the row's maximum after the tile before, from the other warpgroup.
        ok = both_wait(smem_u32(&sh.s_full[g]), (q >> 1) & 1,
                       smem_u32(&sh.m_full[g ^ 1][w4]), ((q - 1) >> 1) & 1,
                       j > 0 && n > 0);
        if (!ok) break;
        fence_after_sync();
        if (n <= 0) {
          // None: their P is whatever lies there, and goes to rows nobody stores.
          if (j > 1) ok = all_wait(smem_u32(&sh.p_empty[g]), ((q - 2) >> 1) & 1);
          if (!ok) break;
          if (lane == 0) {
            tc::remote_arrive(k_full + (q + 2) % kNK * 8);
            mbar_arrive(smem_u32(&sh.m_full[g][w4]));
            tc::remote_arrive(v_full + q % kNV * 8);
          }
          continue;
        }
        uint32_t u[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(srow + c * 32, u[c]);
        const float m_prev = j > 0 ? sh.top[g ^ 1][r] : -INFINITY;
        // PV(j - 2) done: P may be overwritten.  Asked early, known when needed.
        const bool p_free =
            j < 2 || mbar_test(smem_u32(&sh.p_empty[g]), ((q - 2) >> 1) & 1);
        tmem_wait_ld();
        fence_before_sync();
        __syncwarp();
        // S may be overwritten, by QK(q + 2).
        if (lane == 0) tc::remote_arrive(k_full + (q + 2) % kNK * 8);
        const int key0 = (t.key_begin + j) * kT;
        const int seen = pos - key0 + 1;        // tokens of the tile this row sees
        if (pos_lo - key0 + 1 < kT) {           // not all for every row of the warp
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (c * 32 + i >= seen) u[c][i] = 0xff800000u;  // -inf
        }
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 32; i += 2)
            m4[(i >> 1) & 3] = max3(m4[(i >> 1) & 3], __uint_as_float(u[c][i]),
                                    __uint_as_float(u[c][i + 1]));
        const float m_tile =
            fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * p.scale_log2;
        const bool need = m_tile > m_prev + kRescale;
        const float m = need ? m_tile : m_prev;
        sh.top[g][r] = m;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.m_full[g][w4]));
        if (m != m_own) {
          l *= ex2(m_own - m);
          m_own = m;
        }
        const float neg_m = m == -INFINITY ? 0.f : -m;
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
            ok = __all_sync(0xffffffffu, p_free) ||
                 all_wait(smem_u32(&sh.p_empty[g]), ((q - 2) >> 1) & 1);
            if (!ok) break;
            fence_after_sync();
          }
          tmem_st32(prow + c2 * 32, pk);
        }
        if (!ok) break;
        float s_even, s_odd;
        unpack2(add2(s2[0], s2[1]), s_even, s_odd);
        l += s_even + s_odd;
        if (__any_sync(0xffffffffu, need) && j > 0) {
          // O is what PV(j - 1) leaves, and PV(j) waits for this warp.
          ok = all_wait(smem_u32(&sh.p_empty[g ^ 1]), ((q - 1) >> 1) & 1);
          if (!ok) break;
          fence_after_sync();
          rescale_row<D>(orow, need ? ex2(m_prev - m) : 1.f);
        }
        tmem_wait_st();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::remote_arrive(v_full + q % kNV * 8);
      }
      ok = ok && all_wait(smem_u32(&sh.o_ready), (it.n - 1) & 1);
      sh.top[g][r] = m_own;  // (a warpgroup may have had no tile)
      sh.sum[g][r] = l;
      ok = tc::bar_and(1, 256, ok && !*aborted);
      if (!ok) break;
      fence_after_sync();
      if (n <= 0) {
        if (lane == 0) tc::remote_arrive(o_empty);
        continue;
      }
      // The two warpgroups' sums joined, in an order that does not depend on which
      // had the item's first tile; the larger maximum is O's.  Each warp D / 2
      // columns.
      const int a = it.tiles0 & 1;  // the warpgroup of the first tile
      const float m0 = sh.top[a][r], m1 = sh.top[a ^ 1][r];
      const float top = fmaxf(m0, m1);
      // A row may see nothing of a cut range: no weight, and a sum of 0.
      const float e0 = m0 == -INFINITY ? 0.f : ex2(m0 - top);
      const float e1 = m1 == -INFINITY ? 0.f : ex2(m1 - top);
      const float sum = e0 * sh.sum[a][r] + e1 * sh.sum[a ^ 1][r];
      const bool cut = t.partial >= 0;
      const float inv = cut ? 1.f : 1.f / sum;
      // This row: of the item's partial rows, or as a (token, head) of the batch.
      const int64_t prow = (int64_t)t.partial + (int64_t)h * t.ntok * G +
                           rank * ctok * G + r;
      const int64_t orow_at =
          (int64_t)(t.row0 + tok) * p.Hq + h * G + (r - (tok - rank * ctok) * G);
      if (cut && g == 0 && lane < n) p.ml[prow] = make_float2(top, sum);
      const bool odd = *odd_values != 0;
#pragma unroll 1
      for (int c = g * (D / 2); c < (g + 1) * (D / 2); c += 32) {
        uint32_t v[32];
        tmem_ld32(orow + c, v);
        tmem_wait_ld();
        if (c + 32 == (g + 1) * (D / 2)) {  // O has been read
          fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::remote_arrive(o_empty);
        }
        float x[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) x[k] = __uint_as_float(v[k]) * inv;
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
        // Each lane its row: whole sectors in two stores (turning 32 rows through
        // shared memory for wider runs took 1650 cycles here, with no product running).
        if (lane < n && cut) {
          float4* dst = reinterpret_cast<float4*>(p.o + prow * D + c);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            dst[k] = make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
        } else if (lane < n) {
          uint4* dst = reinterpret_cast<uint4*>(p.out + orow_at * D + c);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            dst[k] = make_uint4(pack_bf16(x[8 * k], x[8 * k + 1]),
                                pack_bf16(x[8 * k + 2], x[8 * k + 3]),
                                pack_bf16(x[8 * k + 4], x[8 * k + 5]),
                                pack_bf16(x[8 * k + 6], x[8 * k + 7]));
        }
        __syncwarp();
      }
    }
    if (!ok && lane == 0) timed_out(70);
  } else {
   asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
   if (warp == 0 && rank == 0) {
    // ---- scores: QK(q) once K is there and S(q - 2) has been read (uniform warp,
    // one lane issues) -----------------------------------------------------------------
    constexpr uint32_t id = idesc(128 * kCtas, kT, false);
    const bool lead = elect_one();
    bool ok = true;
    while (next_item(ok)) {
      const int nt = uniform(it.nt);
      const uint32_t item = uniform(it.n) - 1, t0 = uniform(it.tiles0);
      const uint32_t qs = item % kQs;
      const uint64_t qd = sdesc(base + qs * C::kQ, 16, 1024);
      ok = all_wait(smem_u32(&sh.q_full[qs]), (item / kQs) & 1);
      for (int j = 0; j < nt && ok; ++j) {
        const uint32_t q = t0 + j, st = q % kNK;
        const uint64_t kd =
            sdesc(base + C::kOffK + st * C::kK, 16, D == 128 ? 2048 : 1024);
        ok = all_wait(smem_u32(&sh.k_full[st]), (q / kNK) & 1);
        if (!ok) break;
        fence_after_sync();
        if (lead) {
#pragma unroll
          for (int x = 0; x < D / 16; ++x)
            mma_ss<kCtas>(tmem + (q & 1) * kT,
                          qd + (((x >> 2) * 16384 + (x & 3) * 32) >> 4),
                          kd + (((x >> 2) * 1024 + (x & 3) * 32) >> 4), id,
                          x > 0 ? 1u : 0u);
          commit<kCtas>(smem_u32(&sh.s_full[q & 1]));
          commit<kCtas>(smem_u32(&sh.k_empty[st]));
          if (j == nt - 1) commit<kCtas>(smem_u32(&sh.q_empty[qs]));
        }
        __syncwarp();
      }
    }
    if (!ok && lead) {
      timed_out(71);
      // Every product issued has finished once this lands, or a time has passed.
      commit<kCtas>(smem_u32(&sh.drain[0]));
      mbar_wait(smem_u32(&sh.drain[0]), 0);
    }
   } else if (warp == 1 && rank == 0) {
    // ---- O: PV(q) once V is there and P(q) has been written ---------------------------
    constexpr uint32_t id = idesc(128 * kCtas, D, true);
    const bool lead = elect_one();
    bool ok = true;
    while (next_item(ok)) {
      const int nt = uniform(it.nt), first = uniform(it.t.key_begin);
      const int blocks = uniform(it.nblk) - first * kTB;
      const int whole = uniform(it.t.pos0) + 1 - first * kT;
      const uint32_t item = uniform(it.n) - 1, t0 = uniform(it.tiles0);
      // O of the item before has been read.
      ok = all_wait(smem_u32(&sh.o_empty), (item & 1) ^ 1);
      for (int j = 0; j < nt && ok; ++j) {
        const uint32_t q = t0 + j, st = q % kNV;
        ok = all_wait(smem_u32(&sh.v_full[st]), (q / kNV) & 1);
        // Where values have been written over: the writes, of both CTAs.
        if (ok && (j + 1) * kT > whole)
          ok = tc::all_wait_cluster(smem_u32(&sh.v_full[st]), (q / kNV) & 1);
        if (!ok) break;
        fence_after_sync();
        if (lead) {
          const uint32_t pcol = tmem + kColP + (q & 1) * 64;
          const uint64_t vd = vdesc<C::kRowV>(base + C::kOffV + st * C::kV);
#pragma unroll
          for (int x = 0; x < kTB; ++x)
            if (x < blocks - j * kTB)
              mma_ts<kCtas>(tmem + kColO, pcol + x * 8, vd + x * (C::kBlkV >> 4), id,
                            j > 0 || x > 0 ? 1u : 0u);
          commit<kCtas>(smem_u32(&sh.p_empty[q & 1]));
          commit<kCtas>(smem_u32(&sh.v_empty[st]));
          if (j == nt - 1) commit<kCtas>(smem_u32(&sh.o_ready));
        }
        __syncwarp();
      }
    }
    if (!ok && lead) {
      timed_out(74);
      commit<kCtas>(smem_u32(&sh.drain[1]));
      mbar_wait(smem_u32(&sh.drain[1]), 0);
    }
  } else if (warp == 12 && rank == kCtas - 1) {
    // ---- the work items: the first by its place in the grid, then as they come.
    // Head groups in turn (what is read at a time stays in L2), in a group the
    // longest items first.
    bool ok = true;
    const int n_work = p.n_items * p.Hkv, units = gridDim.x / kCtas;
    auto next_index = [&] {
      int i = 0;
      if (lane == 0) i = units + atomicAdd(p.next, 1);
      return __shfl_sync(0xffffffffu, i, 0);
    };
    int i = blockIdx.x / kCtas;
    for (uint32_t n = 0;; ++n) {
      const uint32_t slot = n & 1;
      if (n >= 2) ok = all_wait(smem_u32(&sh.item_empty[slot]), ((n >> 1) - 1) & 1);
      ok = __all_sync(0xffffffffu, ok && !*aborted);
      if (!ok) break;
      ChunkItem t{0, 1, 0, 0, 0, 1, -1, 0};
      int h = -1;
      for (; i < n_work; i = next_index()) {
        const int group = i / (p.n_items * p.heads);
        const int heads = min(p.heads, p.Hkv - group * p.heads);
        const int rest = i - group * p.n_items * p.heads;
        t = p.items[rest / heads];
        h = group * p.heads + rest % heads;
        if (t.ntok >= 1 && t.ntok <= kCtas * ctok && t.pos0 >= 0 &&
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
      if (lane < kCtas) {
        const uint32_t bar = in_cta<kCtas>(smem_u32(&sh.item_full[slot]), lane);
        const uint32_t to = in_cta<kCtas>(smem_u32(&sh.item[slot]), lane);
        tc::remote_expect_tx(bar, 32);
        tc::remote_store16(to, t.row0, t.ntok, t.pos0, t.table, bar);
        tc::remote_store16(to + 16, t.key_begin, t.key_end, t.partial, h, bar);
      }
      __syncwarp();
      if (h < 0) break;
      i = next_index();
    }
    if (!ok && lane == 0) timed_out(75);
  } else if (warp == 2 || warp == 3 || (warp == 14 && kLoads == 3)) {
    // ---- loads of this CTA's part: its rows of Q, its keys, its columns of the
    // values; the load warps take the key tiles in turn ----------------------------
    const int me = warp == 14 ? 2 : warp - 2;
    bool ok = true;
    // Widened blocks were stored by a kernel before, read by bulk copies here.
    asm volatile("fence.proxy.async;" ::: "memory");
    // Lanes 0-7 (pairs: 0-3) keys, 8-15 values.
    constexpr int kKeyLanes = kTB / kCtas;
    const int bi = lane < 8 ? rank * kKeyLanes + (lane & (kKeyLanes - 1)) : lane & 7;
    while (next_item(ok)) {
      const int nt = it.nt, h = it.h;
      const uint32_t item = it.n - 1;
      if (me == 0) {
        const uint32_t qb = item % kQs;
        if (item >= kQs)
          ok = all_wait(smem_u32(&sh.q_empty[qb]), (item / kQs - 1) & 1);
        ok = __all_sync(0xffffffffu, ok && !*aborted);
        if (!ok) break;
        const uint32_t bar = in_cta<kCtas>(smem_u32(&sh.q_full[qb]), 0);
        if (lane == 0) tc::remote_expect_tx(bar, D / 64 * ctok * G * 128);
        __syncwarp();
        if (lane < D / 64)
          load_3d<kCtas>(base + qb * C::kQ + lane * 16384, &tmQ, lane * 64, h * G,
                         it.t.row0 + rank * ctok, bar);
        __syncwarp();
      }
      auto slot_of = [&](int tile) {
        const int blk = (it.t.key_begin + tile) * kTB + bi;
        if ((lane >= kKeyLanes && lane < 8) || lane >= 16 || tile >= nt ||
            blk >= it.nblk)
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
        const uint32_t q = it.tiles0 + j, ks = q % kNK, vs = q % kNV;
        const uint32_t kbar = in_cta<kCtas>(smem_u32(&sh.k_full[ks]), 0);
        const uint32_t vbar = in_cta<kCtas>(smem_u32(&sh.v_full[vs]), 0);
        if (q >= kNK) ok = all_wait(smem_u32(&sh.k_empty[ks]), (q / kNK - 1) & 1);
        ok = __all_sync(0xffffffffu, ok && !*aborted);
        if (!ok) break;
        if (lane == 0) tc::remote_expect_tx(kbar, __popc(act & 0xff) * C::kBlkK);
        __syncwarp();
        if (load && lane < 8) {
          const uint32_t dst = base + C::kOffK + ks * C::kK + lane * C::kBlkK;
          if (D == 128)
            load_tile<kCtas>(dst, &tmK, 0, slot * p.Hkv + h, kbar);
          else
            load_2d<kCtas>(dst, &tmK, 0, (slot * p.Hkv + h) * 16, kbar);
        }
        __syncwarp();
        if (q >= kNV) ok = all_wait(smem_u32(&sh.v_empty[vs]), (q / kNV - 1) & 1);
        ok = __all_sync(0xffffffffu, ok && !*aborted);
        if (!ok) break;
        // Not all of the tile's tokens are seen by every row of the item: by way of the
        // warp for those.
        const bool masked = (it.t.key_begin + j + 1) * kT > it.t.pos0 + 1;
        const uint32_t bar =
            masked ? in_cta<kCtas>(smem_u32(&sh.v_raw[vs]), rank) : vbar;
        if (lane == 0) tc::remote_expect_tx(bar, __popc(act >> 8) * C::kBlkV);
        __syncwarp();
        const int vst = C::kOffV + vs * C::kV;
        if (load && lane >= 8) {
          const uint32_t dst = base + vst + bi * C::kBlkV;
          if (D == 128)
            load_tile<kCtas>(dst, &tmV, rank, slot * p.Hkv + h, bar);
          else
            load_2d<kCtas>(dst, &tmV, rank * 32, (slot * p.Hkv + h) * 16, bar);
        }
        __syncwarp();
      }
      if (!ok) break;
    }
    if (!ok && lane == 0) timed_out(72);
  } else if (warp == 13) {
    // ---- values that some row of the item does not see: zeros over what no row sees
    // and over what is not finite -----------------------------------------------------
    uint32_t raws = 0;  // parities of v_raw
    bool ok = true;
    while (next_item(ok)) {
      for (int j = max(it.t.pos0 + 1 - it.t.key_begin * kT, 0) / kT; j < it.nt; ++j) {
        const uint32_t q = it.tiles0 + j, vs = q % kNV;
        ok = all_wait(smem_u32(&sh.v_raw[vs]), raws >> vs & 1);
        if (!ok) break;
        raws ^= 1u << vs;
        constexpr int kChunks = C::kRowV / 16;         // of a token
        const int key0 = (it.t.key_begin + j) * kT;
        const int rows = min(kTB, it.nblk - key0 / 16) * 16;
        const int len = it.t.pos0 + it.t.ntok - key0;  // tokens that a row sees
        uint8_t* v = smem + C::kOffV + vs * C::kV;
        bool odd = false;
        const int end = min(rows, len) * kChunks;
        for (int k0 = max(it.t.pos0 + 1 - key0, 0) * kChunks + lane; k0 < end;
             k0 += 4 * 32) {
          uint4 y[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int k = min(k0 + x * 32, end - 1);
            y[x] = *reinterpret_cast<uint4*>(v + C::v_at(k / kChunks, k % kChunks));
          }
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            bool here = drop_odd(y[x].x);
            here |= drop_odd(y[x].y);
            here |= drop_odd(y[x].z);
            here |= drop_odd(y[x].w);
            const int k = min(k0 + x * 32, end - 1);
            if (here)
              *reinterpret_cast<uint4*>(v + C::v_at(k / kChunks, k % kChunks)) = y[x];
            odd |= here;
          }
        }
        for (int k = end + lane; k < rows * kChunks; k += 32)
          *reinterpret_cast<uint4*>(v + C::v_at(k / kChunks, k % kChunks)) =
              make_uint4(0, 0, 0, 0);
        odd = __any_sync(0xffffffffu, odd);
        if (odd && lane < kCtas)
          tc::cluster_store4(in_cta<kCtas>(smem_u32(&sh.odd_values), lane), 1u);
        const uint32_t bar = in_cta<kCtas>(smem_u32(&sh.v_full[vs]), 0);
        if (odd || len < rows) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) remote_arrive_release(bar);
        } else if (lane == 0) {
          tc::remote_arrive(bar);  // nothing was written
        }
      }
      if (!ok) break;
    }
    if (!ok && lane == 0) timed_out(73);
  }
  }
  __syncwarp();
  fence_before_sync();
  __syncthreads();
  if (*aborted) tc::wait_for_copies();
  __syncwarp();
  tc::cluster_sync();
  fence_after_sync();
  if (warp == 0) {
    if (kCtas == 2)
      tc::tmem_free2(tmem, kTmemCols);
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                   "r"(kTmemCols)
                   : "memory");
  }
  tc::cluster_sync();  // neither CTA leaves before both have given it back
  if (p.beside) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Joins the partial rows of cut tiles: a warp for each (token, head), in turn.  Eight
// pieces are fetched at a time, then joined in order: one at a time each waited for the
// one before (1 token with 8 heads on 60000 cached ones 46 us, now 25; with 64 heads on
// 4000 16.7, now 13.3).
template <int D>
__global__ void __launch_bounds__(256) join_kernel(const ChunkMerge* merges,
                                                   const Params p) {
  constexpr int V = D / 32;  // values per lane
  constexpr int kAhead = 8;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const ChunkMerge m = merges[blockIdx.x];
  const int lane = threadIdx.x & 31;
  const int first = blockIdx.y * 8 + (threadIdx.x >> 5);  // (head, token, head of G)
  const int64_t stride = (int64_t)m.ntok * p.Hq;
  if (m.ntok < 1 || m.row0 < 0 || m.row0 > p.total - m.ntok || m.pieces < 1 ||
      m.partial < 0 || m.partial + stride * m.pieces > p.partial_rows) {
    if (first == 0 && lane == 0) record_status(p.status, KV_ERR_DEVICE, m.partial);
    return;
  }
  for (int row = first; row < stride; row += gridDim.y * 8) {
    const int h = row / (m.ntok * p.G), rest = row % (m.ntok * p.G);
    float top = -INFINITY, sum = 0.f, acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    for (int k0 = 0; k0 < m.pieces; k0 += kAhead) {
      float2 ml[kAhead];
      float v[kAhead][V];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (k0 + k >= m.pieces) break;
        const int64_t at = m.partial + (k0 + k) * stride + row;
        ml[k] = p.ml[at];
#pragma unroll
        for (int i = 0; i < V; i += 2)
          *reinterpret_cast<float2*>(v[k] + i) =
              *reinterpret_cast<const float2*>(p.o + at * D + lane * V + i);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (k0 + k >= m.pieces) break;
        const float m_new = fmaxf(top, ml[k].x);
        const float a = top == -INFINITY ? 0.f : ex2(top - m_new);
        const float w = ml[k].x == -INFINITY ? 0.f : ex2(ml[k].x - m_new);
        sum = sum * a + w * ml[k].y;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = acc[i] * a + w * v[k][i];
        top = m_new;
      }
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
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (threadIdx.x != 0) return;
  *status = DeviceStatus{};
  next[0] = next[1] = 0;
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

// All columns of a CTA's part of the values are in one box.
template <int D, int kCtas>
kv_status make_maps(CUtensorMap* tk, CUtensorMap* tv, const void* k, const void* v,
                    int64_t tiles) {
  if (D == 128) {
    if (kv_status s = make_tile_map(tk, k, tiles, 2)) return s;
    return make_tile_map(tv, v, tiles, 2 / kCtas);
  }
  if (kv_status s = make_row_map(tk, k, tiles, 64)) return s;
  return make_row_map(tv, v, tiles, 64 / kCtas);
}

// Persistent CTAs (pairs) for `work` items on `sms` SMs.
template <int D, int kCtas>
kv_status launch(const CUtensorMap& tq, const void* k, const void* v, const Params& p,
                 int64_t work, int sms, cudaStream_t st) {
  CUtensorMap tk, tv;
  if (kv_status s = make_maps<D, kCtas>(&tk, &tv, k, v, p.blocks * p.Hkv)) return s;
  static std::atomic<uint64_t> opted{0};
  cudaError_t e =
      opt_in_smem(attention_kernel<D, kCtas>, smem_bytes<D, kCtas>(), opted);
  cudaLaunchAttribute attrs[2]{};
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim = {kCtas, 1, 1};
  cudaLaunchConfig_t cfg{};
  cfg.gridDim =
      dim3((unsigned)(kCtas * std::min<int64_t>(work, std::max(sms / kCtas, 1))));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)smem_bytes<D, kCtas>();
  cfg.stream = st;
  cfg.attrs = attrs;
  cfg.numAttrs = 2;
  if (e == cudaSuccess)
    e = cudaLaunchKernelEx(&cfg, attention_kernel<D, kCtas>, tq, tk, tv, p);
  if (e != cudaSuccess)
    return fail(KV_ERR_CUDA, "chunk attention: %s", cudaGetErrorString(e));
  return KV_OK;
}

// The step's items: those of more than a CTA's tokens (n_wide, first in the list) on
// pairs, the others beside them on single CTAs; then the cut tiles joined.
template <int D>
kv_status launch_all(const CUtensorMap& tq, const void* k, const void* v, Params p,
                     int n_wide, const ChunkMerge* merges, int n_merges, int sms,
                     cudaStream_t st) {
  const int n_narrow = p.n_items - n_wide;
  p.beside = false;
  if (n_wide > 0) {
    p.n_items = n_wide;
    if (kv_status s =
            launch<D, 2>(tq, k, v, p, (int64_t)n_wide * p.Hkv, sms, st))
      return s;
  }
  if (n_narrow > 0) {
    p.beside = n_wide > 0;
    p.items += n_wide;
    p.n_items = n_narrow;
    p.next += 1;
    if (kv_status s =
            launch<D, 1>(tq, k, v, p, (int64_t)n_narrow * p.Hkv, sms, st))
      return s;
  }
  if (n_merges == 0) return KV_OK;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  // No more CTAs than run at once: most tiles have fewer rows than they could.
  const int64_t most = (2 * (kM / p.G) * (int64_t)p.Hq + 7) / 8;
  cfg.gridDim = dim3((unsigned)n_merges,
                     (unsigned)std::clamp<int64_t>(4 * 152 / n_merges, 1, most));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, join_kernel<D>, merges, p);
  if (e != cudaSuccess)
    return fail(KV_ERR_CUDA, "chunk attention: %s", cudaGetErrorString(e));
  return KV_OK;
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
  const int64_t n_slots = info->plan_ints - kPlanHeaderInts - info->n_row_items -
                          8ll * info->n_tile_items - 4ll * info->n_row_warp_items;
  if (info->latent_rows != chunk_mark(Hq, Hkv, d) || info->n_merge_rows != total ||
      info->n_row_items < 0 || info->n_tile_items < 0 || info->n_tile_wide_items < 0 ||
      info->n_tile_wide_items > info->n_tile_items || info->n_row_warp_items < 0 ||
      n_slots < 0 || n_slots > INT32_MAX || info->partial_rows < 0 ||
      info->partial_rows > INT32_MAX || (total > 0) != (info->n_tile_items > 0) ||
      (e4m3 && total > 0) != (info->n_row_items > 0) ||
      (int64_t)info->n_tile_items * Hkv > INT32_MAX / 2 ||
      (int64_t)info->n_row_items * Hkv > INT32_MAX / 16 ||
      (info->n_row_warp_items > 0) != (info->partial_rows > 0))
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
  CUtensorMap tq;
  const int U = info->n_row_items;
  auto* wide = ws + ws_total(info->partial_rows, d);
  const void* k = e4m3 ? wide : k_pool;
  const void* v = e4m3 ? wide + chunk_half(U, Hkv, d) : v_pool;
  p.blocks = e4m3 ? U : num_blocks;
  if (total > 0)
    if (kv_status s = make_query_map(&tq, q, q_stride, total, Hq, Hq / Hkv, d))
      return s;
  int dev = 0, sms = 152;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess)
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess)
    return fail(KV_ERR_CUDA, "chunk attention: %s", cudaGetErrorString(e));
  e = launch_early(clear_kernel, 1, 32, 0, st, p.status, p.next);
  if (e != cudaSuccess)
    return fail(KV_ERR_CUDA, "chunk attention: %s", cudaGetErrorString(e));
  if (total == 0) return KV_OK;
  p.slots = plan + kPlanHeaderInts + U;
  p.n_slots = (int)n_slots;
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
  // Heads whose items run at a time: all of them where their keys and values fit L2
  // together (then the longest items of all heads come first), else as many as do
  // (shared blocks count as often as branches hold them).
  const int64_t head_bytes = (int64_t)p.n_slots * 16 * d * 4;
  p.heads = head_bytes * Hkv <= (96ll << 20)
                ? Hkv
                : (int)std::clamp<int64_t>((48ll << 20) / head_bytes, 1, Hkv);
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
  return d == 128 ? launch_all<128>(tq, k, v, p, info->n_tile_wide_items, merges,
                                    info->n_row_warp_items, sms, st)
                  : launch_all<64>(tq, k, v, p, info->n_tile_wide_items, merges,
                                   info->n_row_warp_items, sms, st);
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
