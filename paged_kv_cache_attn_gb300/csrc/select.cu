// Blocks that a cheap score selects for each query: bounds of the blocks' keys
// (paged_key_bounds), scores and selection (paged_select_blocks), and the decode
// step over what was selected (paged_selected_plan, paged_selected_attn).
//
// Bounds.  A block's keys of a kv-head lie in a box; its corners are kept as whole
// numbers of 8 bits times one power of two 2^e, rounded outward, e the smallest with
// max|k| <= 127 x 2^e.  2 D + 4 bytes against the 32 D (bf16) of the keys.
//
// Scores.  A query head as whole numbers q_c of at most 127 times a power of two has
// with every key of the block a product of at most
//   sum_c max(q_c lo_c, q_c hi_c) = sum_c (min(q_c, 0) lo_c + max(q_c, 0) hi_c)
// (times the two powers), a product of 2 D whole numbers below 2^24 in total: exact
// in fp32 in any order, so that the selection does not depend on how it is computed.
// It runs on f16 mma.sync (whole numbers up to 2048 are exact there): bytes become
// f16 by one byte permutation and one subtraction a pair.
//
// Attention.  A (branch, kv-head) with its list of blocks is a branch with one
// kv-head in the pool seen as [num_blocks x Hkv][1][16][D], which the split-KV
// kernels read as they are: the selection writes their tables.

#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include <cuda_fp16.h>

#include "device_common.cuh"
#include "e4m3.cuh"
#include "tensor_map.h"

namespace pkv {
namespace sel {

constexpr int kEMin = -60, kEMax = 40;  // exponents of bounds and queries
constexpr int kMaxG = 128;              // query heads of a kv-head

// Smallest e in [-60, 40] with amax <= 127 x 2^e, from the bits of amax:
// amax = (1 + M / 2^23) 2^(E - 127) and 127 = 1.984375 x 2^6, so e = E - 133 where
// M / 2^23 <= 0.984375 (0x7e0000), else E - 132.
__device__ __forceinline__ int bound_exponent(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int e = (int)(bits >> 23) - ((bits & 0x7fffffu) <= 0x7e0000u ? 133 : 132);
  return min(max(e, kEMin), kEMax);
}

// ---- bounds -----------------------------------------------------------------------

struct BoundsParams {
  const uint8_t* k;          // this layer's K pool
  const float4* scales;      // e4m3: records
  const int32_t* tables;
  const int32_t* seq_lens;
  const int32_t* row_offsets;
  int8_t* bounds;            // [num_blocks][Hkv][2][D]
  float* bound_scales;       // [num_blocks][Hkv]
  DeviceStatus* status;
  int64_t num_blocks;
  int total, nb, max_blocks, Hkv;
};

__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t min2h(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max2h(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// A warp's part of a tile's keys: a lane has kPer dimensions (16 bytes) of every
// kRows-th row.
template <int D, bool E4M3>
struct TileKeys {
  static constexpr int kPer = E4M3 ? 16 : 8;
  static constexpr int kChunks = D / kPer;      // 16-byte chunks of a row
  static constexpr int kRows = 32 / kChunks;    // rows of a load
  static constexpr int kLoads = 16 / kRows;
  uint4 x[kLoads];
  float scale;

  __device__ __forceinline__ void load(const BoundsParams& p, int64_t tile, int valid,
                                       int lane) {
    const int c = lane % kChunks, r0 = lane / kChunks;
    const uint8_t* src = p.k + tile * (16 * D * (E4M3 ? 1 : 2));
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      // Slots past the branch's length: its last token again.
      const int t = min(i * kRows + r0, valid - 1);
      const int at = E4M3 ? t * D + ((D == 128 ? c ^ (t & 7) : c) << 4)
                          : (t * kChunks + c) * 16;
      x[i] = *reinterpret_cast<const uint4*>(src + at);
    }
    scale = E4M3 ? p.scales[tile].x : 1.f;
  }
};

// Bounds of one (block, head) tile, by one warp.
template <int D, bool E4M3>
__device__ __forceinline__ void tile_bounds(const BoundsParams& p, int64_t tile,
                                            const TileKeys<D, E4M3>& keys, int lane) {
  using K = TileKeys<D, E4M3>;
  constexpr int kPer = K::kPer, kChunks = K::kChunks, kRows = K::kRows,
                kLoads = K::kLoads;
  const int c = lane % kChunks;
  const auto& x = keys.x;
  const float scale = keys.scale;
  // Pairs of dimensions, least and largest.
  constexpr int kPairs = kPer / 2;
  uint32_t lo[kPairs], hi[kPairs];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    uint32_t y[kPairs];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (E4M3)
        e4m3x4_to_f16x2x2(w[k], y[(2 * k) % kPairs], y[(2 * k + 1) % kPairs]);
      else
        y[k] = w[k];
    }
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
      if (i == 0) {
        lo[k] = hi[k] = y[k];
      } else {
        lo[k] = E4M3 ? min2h(lo[k], y[k]) : min2(lo[k], y[k]);
        hi[k] = E4M3 ? max2h(hi[k], y[k]) : max2(hi[k], y[k]);
      }
    }
  }
  // Joined over the rows' lanes, each step leaving a lane half of its pairs: those of
  // its chunk from pair `at` on.
  int at = 0;
#pragma unroll
  for (int o = kChunks, n = kPairs / 2; o < 32; o <<= 1, n >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int k = 0; k < n; ++k) {
      const uint32_t a = __shfl_xor_sync(0xffffffffu, up ? lo[k] : lo[k + n], o);
      const uint32_t b = __shfl_xor_sync(0xffffffffu, up ? hi[k] : hi[k + n], o);
      lo[k] = E4M3 ? min2h(up ? lo[k + n] : lo[k], a) : min2(up ? lo[k + n] : lo[k], a);
      hi[k] = E4M3 ? max2h(up ? hi[k + n] : hi[k], b) : max2(up ? hi[k + n] : hi[k], b);
    }
    at += up ? n : 0;
  }
  constexpr int kLeft = kPairs / kRows;
  auto value = [&](uint32_t w, int half) {
    if (E4M3) {
      const float2 f = __half22float2(*reinterpret_cast<__half2*>(&w));
      return (half ? f.y : f.x) * scale;
    }
    return __uint_as_float(half ? w & 0xffff0000u : w << 16);
  };
  float amax = 0.f;
  bool odd = false;
#pragma unroll
  for (int k = 0; k < kLeft; ++k)
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const float a = fabsf(value(lo[k], z)), b = fabsf(value(hi[k], z));
      odd |= !(a < INFINITY) || !(b < INFINITY);
      amax = fmaxf(amax, fmaxf(a, b));
    }
  // (Not negative: ordered as whole numbers.)
  amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
  odd = __any_sync(0xffffffffu, odd);
  const int e = bound_exponent(amax);
  const float inv = pow2f(-e);
  uint32_t out[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < 2 * kLeft; ++k) {
    const float l = fmaxf(floorf(value(lo[k / 2], k & 1) * inv), -127.f);
    const float u = fminf(ceilf(value(hi[k / 2], k & 1) * inv), 127.f);
    // (Above -127 and below 127 too, where keys are beyond the exponents.)
    out[0] |= (uint32_t)((int)fminf(l, 127.f) & 0xff) << (8 * k);
    out[1] |= (uint32_t)((int)fmaxf(u, -127.f) & 0xff) << (8 * k);
  }
  if (odd) out[0] = out[1] = 0;
  int8_t* dst = p.bounds + tile * (2 * D) + c * kPer + 2 * at;
#pragma unroll
  for (int z = 0; z < 2; ++z) {
    if constexpr (kLeft == 2)
      *reinterpret_cast<uint32_t*>(dst + z * D) = out[z];
    else
      *reinterpret_cast<uint16_t*>(dst + z * D) = (uint16_t)out[z];
  }
  // A block with a value that is not finite has a score above all others.
  if (lane == 0) p.bound_scales[tile] = odd ? INFINITY : pow2f(e);
}

// A warp for each (run of new tokens, kHeads kv-heads): every block that a token of the
// run is the first new one of.  run: tokens of a run (steps of one token a branch: 1).
// Finding a block takes four reads that wait for one another; with more tiles than warps
// that run at once, a warp has four heads of each block, whose keys are in flight
// together.
template <int D, bool E4M3, int kHeads>
__global__ void __launch_bounds__(256) bounds_kernel(const BoundsParams p, int run) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int per_run = (p.Hkv + kHeads - 1) / kHeads;
  const int64_t tok0 = w / per_run * run;
  const int h = (int)(w % per_run) * kHeads;
  if (tok0 >= p.total) return;
  const int end = (int)min(tok0 + run, (int64_t)p.total);
  int tok = (int)tok0, b = tok;
  if (p.row_offsets) {
    // The last branch that starts at or before the token.
    int lo = 0, hi = p.nb;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.row_offsets[mid] <= tok) lo = mid; else hi = mid;
    }
    b = lo;
  }
  while (tok < end) {
    int first = tok, next = tok + 1;  // the branch's new tokens
    if (p.row_offsets) {
      while (b + 1 < p.nb && p.row_offsets[b + 1] <= tok) ++b;
      first = p.row_offsets[b];
      next = p.row_offsets[b + 1];
      if (first > tok || next <= tok) return;  // malformed
    }
    const int L = p.seq_lens[b];
    const int64_t pos = (int64_t)L - (next - first) + (tok - first);
    if (pos < 0 || L > (int64_t)p.max_blocks * 16) {
      if (lane == 0) record_status(p.status, KV_ERR_DEVICE, (int)pos);
    } else if (tok == first || (pos & 15) == 0) {
      const int phys = p.tables[(int64_t)b * p.max_blocks + (pos >> 4)];
      if (phys < 0 || phys >= p.num_blocks) {
        if (lane == 0) record_status(p.status, KV_ERR_DEVICE, phys);
      } else {
        const int64_t tile = (int64_t)phys * p.Hkv + h;
        const int valid = min(16, L - (int)(pos & ~15ll));
        TileKeys<D, E4M3> keys[kHeads];
#pragma unroll
        for (int i = 0; i < kHeads; ++i)
          if (i == 0 || h + i < p.Hkv) keys[i].load(p, tile + i, valid, lane);
#pragma unroll
        for (int i = 0; i < kHeads; ++i)
          if (i == 0 || h + i < p.Hkv) tile_bounds<D, E4M3>(p, tile + i, keys[i], lane);
      }
    }
    if (!p.row_offsets) {
      ++tok;
      ++b;
    } else {
      tok = min(next, tok + 16 - (int)(pos & 15));
    }
  }
}

// ---- scores -----------------------------------------------------------------------

struct SelectParams {
  const __nv_bfloat16* q;      // [nb][Hq][D]
  const int8_t* bounds;
  const float* bound_scales;
  const int32_t* tables;
  const int32_t* seq_lens;
  float* scores;               // [nb * Hkv][stride]
  int32_t* sel;                // [nb][Hkv][n_sel], logical blocks (may be null)
  int32_t* sel_tables;         // [nb * Hkv][n_sel], block * Hkv + head
  int32_t* sel_lens;           // [nb * Hkv]
  DeviceStatus* status;
  int64_t num_blocks;
  int nb, max_blocks, stride, Hq, Hkv, G, n_sel, n_first, n_last;
  int heads;                   // of a CTA of the scores (G <= 8; else 1)
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4],
                                        uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four signed bytes as f16 pairs, exactly: v + 128 in the low bits of 1024 (f16
// 0x6400 + u is 1024 + u), less 1152.
__device__ __forceinline__ void bytes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  uint32_t a, b;
  asm("prmt.b32 %0, %1, %2, 0x5140;" : "=r"(a) : "r"(u), "r"(0x64646464u));
  asm("prmt.b32 %0, %1, %2, 0x7362;" : "=r"(b) : "r"(u), "r"(0x64646464u));
  const uint32_t bias = 0x64806480u;  // 1152
  asm("sub.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(bias));
  asm("sub.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(bias));
}

constexpr int kWarps = 8;

// Eight query heads (those from G on are zeros) as whole numbers of at most 127 times a
// power of two, four lanes a head: their f16 values to dst, the powers to e (-1: no such
// head).
template <int D>
__device__ __forceinline__ void quantise8(const __nv_bfloat16* q, int G, __half* dst,
                                          int row, float* e, int lane) {
  constexpr int V = D / 32;  // 16-byte pieces of a lane
  const int g = lane >> 2, part = lane & 3;
  uint4 w[V];
  float amax = 0.f;
  bool odd = false;
  auto value = [](uint32_t pair, int half) {
    return __uint_as_float(half ? pair & 0xffff0000u : pair << 16);
  };
#pragma unroll
  for (int i = 0; i < V; ++i) {
    w[i] = make_uint4(0, 0, 0, 0);
    if (g < G) w[i] = *reinterpret_cast<const uint4*>(q + g * D + (i * 4 + part) * 8);
    const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float a = fabsf(value(x[k / 2], k & 1));
      odd |= !(a < INFINITY);
      amax = fmaxf(amax, a);
    }
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    odd |= __shfl_xor_sync(0xffffffffu, (int)odd, o) != 0;
  }
  const int ex = bound_exponent(amax);
  const float inv = pow2f(-ex);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
    uint32_t y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float f[2];
#pragma unroll
      for (int z = 0; z < 2; ++z)
        f[z] = odd ? 0.f
                   : fminf(fmaxf(rintf(value(x[k], z) * inv), -127.f), 127.f);
      const __half2 h = __floats2half2_rn(f[0], f[1]);
      y[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(dst + g * row + (i * 4 + part) * 8) =
        make_uint4(y[0], y[1], y[2], y[3]);
  }
  if (part == 0) e[g] = g < G ? (odd ? 0.f : pow2f(ex)) : -1.f;
}

// grid (block ranges, groups of p.heads kv-heads, nb); a warp has a head and kSteps x 16
// consecutive blocks.  Up to 16 query heads are the rows of the products, eight blocks
// their columns; lane 4 n + t has bytes [16 t + 64 j, + 16) of block n's record, which
// are its columns of four products in any order that the queries' fragments share.  The
// records of 16 blocks (4 KB at D = 128) are in flight while those before are used, the
// first while the queries are quantised.
// kFew: at most 8 query heads a kv-head, kept in registers (the rows after them are
// zeros), and a CTA's warps have several kv-heads of the same blocks, whose records lie
// side by side.  Else 16 query heads at a time from shared memory, one kv-head a CTA.
// 32 x ~32000 tokens, 133 MB: 35 us; the reads alone 28, the products alone 26, with 16
// warps an SM to run them beside each other.  (Through bulk copies to shared memory 37
// us, 16-byte ones 39; 24 warps with one buffer and the queries in shared memory 32, but
// 48 mixed branches 15 instead of 12.)
template <int D, bool kFew, int kSteps>
__global__ void __launch_bounds__(32 * kWarps, kFew ? 2 : 1)
    score_kernel(const SelectParams p) {
  constexpr int kWarpBlocks = 16 * kSteps;
  constexpr int kRow = D + 8;  // a head's f16 values in shared memory
  __shared__ __align__(16) __half qs[(kFew ? kWarps * 8 : kMaxG) * kRow];
  __shared__ float qe_all[kFew ? kWarps * 8 : kMaxG];
  // (Both kernels of a selection may start early; the second reads the tables at once.)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int b = blockIdx.z, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && b == 0 && blockIdx.y == 0 && threadIdx.x == 0)
    *p.status = DeviceStatus{};  // the next kernel records
  const int L = p.seq_lens[b];
  const int nblk = L < 1 || L > (int64_t)p.max_blocks * 16 ? 0 : (L + 15) / 16;
  const int heads = kFew ? p.heads : 1, ranges = kWarps / heads;
  const int64_t cta_blocks = (int64_t)ranges * kWarpBlocks;
  // A branch of few blocks has them all.
  if (nblk <= p.n_sel || blockIdx.x * cta_blocks >= nblk) return;
  const int h = blockIdx.y * heads + warp % heads;
  const int blk0 = (int)(blockIdx.x * cta_blocks) + warp / heads * kWarpBlocks;
  // (No barrier follows where kFew.)
  if (kFew && (h >= p.Hkv || warp >= ranges * heads || blk0 >= nblk)) return;
  const int32_t* table = p.tables + (int64_t)b * p.max_blocks;
  // A block id outside the pool (recorded by the next kernel) has no score.
  constexpr int kIds = (kSteps + 1) / 2;
  int phys[kIds];
#pragma unroll
  for (int i = 0; i < kIds; ++i) {
    phys[i] = -1;
    if (blk0 + i * 32 + lane < nblk) phys[i] = table[blk0 + i * 32 + lane];
    if (phys[i] >= p.num_blocks) phys[i] = -1;
  }
  const int n = lane >> 2, t = lane & 3;
  constexpr int kJ = 2 * D / 64;  // 64-byte parts of a record
  uint4 rec[2][2][kJ];
  auto fetch = [&](int step) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int ph =
          __shfl_sync(0xffffffffu, phys[step / 2], (step & 1) * 16 + i * 8 + n);
      const uint4* src = reinterpret_cast<const uint4*>(
          p.bounds + ((int64_t)max(ph, 0) * p.Hkv + h) * (2 * D));
#pragma unroll
      for (int j = 0; j < kJ; ++j) rec[step & 1][i][j] = src[j * 4 + t];
    }
  };
  fetch(0);
  float scales[kIds];
#pragma unroll
  for (int i = 0; i < kIds; ++i)
    scales[i] = phys[i] >= 0 ? p.bound_scales[(int64_t)phys[i] * p.Hkv + h] : 0.f;
  const int G = p.G, rows = kFew ? 8 : (G + 15) & ~15;
  const __nv_bfloat16* q = p.q + ((int64_t)b * p.Hq + (int64_t)h * G) * D;
  __half* const own = qs + (kFew ? warp * 8 * kRow : 0);
  float* const qe = qe_all + (kFew ? warp * 8 : 0);
  if constexpr (kFew) {
    quantise8<D>(q, G, own, kRow, qe, lane);
    __syncwarp();
  } else {
    for (int g = 8 * warp; g < rows; g += 8 * kWarps)
      quantise8<D>(q + (int64_t)g * D, G - g, own + g * kRow, kRow, qe + g, lane);
    __syncthreads();
    if (blk0 >= nblk) return;
  }
  // The least values meet the queries' negative numbers, the largest the positive
  // ones.
  auto fragment = [&](int g, int j, uint32_t (&f)[8]) {
    const __half* src = own + g * kRow + (j * 64) % D + t * 16;
    const uint4 v0 = *reinterpret_cast<const uint4*>(src);
    const uint4 v1 = *reinterpret_cast<const uint4*>(src + 8);
    const uint32_t v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
    for (int k = 0; k < 8; ++k)
      f[k] = j < kJ / 2 ? min2h(v[k], 0u) : max2h(v[k], 0u);
  };
  uint32_t few[kFew ? kJ : 1][8];
  if constexpr (kFew) {
#pragma unroll
    for (int j = 0; j < kJ; ++j) fragment(n, j, few[j]);
  }
  float* dst = p.scores + ((int64_t)b * p.Hkv + h) * p.stride;
#pragma unroll
  for (int step = 0; step < kSteps; ++step) {
    if (blk0 + step * 16 >= nblk) break;
    if (step + 1 < kSteps) fetch(step + 1);
    float best[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) best[i][0] = best[i][1] = -INFINITY;
#pragma unroll 1
    for (int g0 = 0; g0 < rows; g0 += 16) {
      float acc[2][4] = {};
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        uint32_t f[2][8];
        if constexpr (!kFew) {
          fragment(g0 + n, j, f[0]);
          fragment(g0 + 8 + n, j, f[1]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4 x = rec[step & 1][i][j];
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            uint32_t b0, b1;
            bytes_to_f16(w[s], b0, b1);
            const uint32_t a[4] = {kFew ? few[kFew ? j : 0][2 * s] : f[0][2 * s],
                                   kFew ? 0u : f[1][2 * s],
                                   kFew ? few[kFew ? j : 0][2 * s + 1] : f[0][2 * s + 1],
                                   kFew ? 0u : f[1][2 * s + 1]};
            mma_f16(acc[i], a, b0, b1);
          }
        }
      }
      const float e0 = qe[g0 + n], e1 = kFew ? -1.f : qe[g0 + 8 + n];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const float s0 = e0 < 0.f ? -INFINITY : acc[i][z] * e0;
          const float s1 = e1 < 0.f ? -INFINITY : acc[i][2 + z] * e1;
          best[i][z] = fmaxf(best[i][z], fmaxf(s0, s1));
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        float s = best[i][z];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1)
          s = fmaxf(s, __shfl_xor_sync(0xffffffffu, s, o));
        const int at = step * 16 + i * 8 + 2 * t + z;
        const float sc = __shfl_sync(0xffffffffu, scales[step / 2], at & 31);
        // (+ 0 makes a zero positive.)
        if (n == 0 && blk0 + at < nblk)
          dst[blk0 + at] = sc == INFINITY ? INFINITY : s * sc + 0.f;
      }
  }
}

// ---- selection --------------------------------------------------------------------

__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

constexpr int kBuckets = 1024;

// Inclusive sums over the CTA's threads; `sh`: 32 entries.
template <int T>
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  __syncthreads();  // sh may still be read
  if (lane == 31) sh[warp] = v;
  __syncthreads();
  uint32_t w = lane < T / 32 ? sh[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  return v + (warp > 0 ? __shfl_sync(0xffffffffu, w, warp - 1) : 0);
}

// A CTA for each (branch, kv-head): which blocks are among the n_sel.  A thread has
// eight blocks' keys at a time (a branch of up to 8 T blocks in registers).  The keys'
// range is cut into 1024 buckets and the one that holds the last key wanted becomes
// the range, until it is wanted whole (nearly always after two passes: scores spread
// over their range) or holds one key, of whose blocks the first are taken.
template <int T>
__global__ void __launch_bounds__(T) pick_kernel(const SelectParams p) {
  __shared__ uint32_t hist[kBuckets], sums[32];
  __shared__ uint32_t sh_lo, sh_hi, sh_bucket, sh_left, sh_count;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int row = blockIdx.x, b = row / p.Hkv, h = row % p.Hkv, tid = threadIdx.x;
  const int L = p.seq_lens[b];
  const int32_t* table = p.tables + (int64_t)b * p.max_blocks;
  int32_t* sel = p.sel ? p.sel + (int64_t)row * p.n_sel : nullptr;
  int32_t* out = p.sel_tables + (int64_t)row * p.n_sel;
  const bool bad = L < 1 || L > (int64_t)p.max_blocks * 16;
  const int nblk = bad ? 0 : (L + 15) / 16;
  const int count = min(nblk, p.n_sel);
  if (tid == 0) {
    sh_lo = 0xffffffffu;
    sh_hi = 0;
  }
  // This thread's blocks' ids, of the first 8 T (older than the kernel before).
  int ids[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) ids[i] = 8 * tid + i < nblk ? table[8 * tid + i] : 0;
  // Scores, and a cleared status word.  (The scores' kernel lets this one start beside
  // it.)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (bad && tid == 0) record_status(p.status, KV_ERR_DEVICE, L);
  // Ids outside the pool (as unsigned numbers no less than its blocks): recorded, -1.
  auto check = [&](int (&id)[8]) {
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) most = max(most, (uint32_t)id[i]);
    if (most < (uint32_t)p.num_blocks) return;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((uint32_t)id[i] >= (uint32_t)p.num_blocks) {
        if (h == 0) record_status(p.status, KV_ERR_DEVICE, id[i]);
        id[i] = -1;
      }
  };
  check(ids);
  auto put_id = [&](int at, int blk, int phys) {
    if (sel) sel[at] = blk;
    out[at] = phys >= 0 ? (int)(phys * (int64_t)p.Hkv + h) : -1;
  };
  if (tid == 0)
    p.sel_lens[row] = count > 0 ? 16 * (count - 1) + (L - 16 * (nblk - 1)) : 0;
  for (int i = count + tid; i < p.n_sel; i += T) {
    if (sel) sel[i] = -1;
    out[i] = -1;
  }
  auto load_ids = [&](int base, int (&id)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = base + 8 * tid + i;
      id[i] = at < nblk ? table[at] : 0;
    }
    check(id);
  };
  if (nblk <= p.n_sel) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (8 * tid + i < nblk) put_id(8 * tid + i, 8 * tid + i, ids[i]);
    for (int base = 8 * T; base < nblk; base += 8 * T) {
      load_ids(base, ids);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int at = base + 8 * tid + i;
        if (at < nblk) put_id(at, at, ids[i]);
      }
    }
    return;
  }
  const float* scores = p.scores + (int64_t)row * p.stride;
  // Keys of blocks base + 8 tid ..; 0 where there is none, all ones where the block
  // is taken in any case.
  auto load = [&](int base, uint32_t (&k)[8]) {
    const int i0 = base + 8 * tid;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i0 + i < nblk) y = *reinterpret_cast<const float4*>(scores + i0 + i);
      x[i] = y.x; x[i + 1] = y.y; x[i + 2] = y.z; x[i + 3] = y.w;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) k[i] = ordered(x[i]);
    if (i0 >= p.n_first && i0 + 8 <= nblk - p.n_last) return;  // nearly all threads
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i0 + i >= nblk)
        k[i] = 0;
      else if (i0 + i < p.n_first || i0 + i >= nblk - p.n_last)
        k[i] = 0xffffffffu;
  };
  uint32_t first[8];
  load(0, first);
  // f(key, block) for all blocks.
  auto each = [&](auto&& f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f(first[i], 8 * tid + i);
    for (int base = 8 * T; base < nblk; base += 8 * T) {
      uint32_t k[8];
      load(base, k);
#pragma unroll
      for (int i = 0; i < 8; ++i) f(k[i], base + 8 * tid + i);
    }
  };
  // [lo, hi]: where the last key wanted is; left: how many of its keys are wanted.
  uint32_t lo = 0xffffffffu, hi = 0, left = (uint32_t)(p.n_sel - p.n_first - p.n_last);
  bool whole = left == 0;  // the range is wanted whole (or nothing of it)
  if (whole) {
    lo = 0xffffffffu;
    hi = 0xffffffffu;
  } else {
    uint32_t a = 0xffffffffu, z = 0;
    each([&](uint32_t k, int) {
      if (k != 0 && k != 0xffffffffu) {
        a = min(a, k);
        z = max(z, k);
      }
    });
    a = __reduce_min_sync(0xffffffffu, a);
    z = __reduce_max_sync(0xffffffffu, z);
    __syncthreads();
    if ((tid & 31) == 0) {
      atomicMin(&sh_lo, a);
      atomicMax(&sh_hi, z);
    }
    __syncthreads();
    lo = sh_lo;
    hi = sh_hi;
  }
  while (!whole && lo < hi) {
    // Keys (of finite scores and infinity) span less than 2^32.
    const int shift = max(0, 32 - __clz(hi - lo) - 10);
    for (int i = tid; i < kBuckets; i += T) hist[i] = 0;
    __syncthreads();
    each([&](uint32_t k, int) {
      if (k >= lo && k <= hi) atomicAdd(&hist[(k - lo) >> shift], 1u);
    });
    __syncthreads();
    // Thread t: buckets from the top.
    constexpr int kPer = kBuckets / T;
    uint32_t mine[kPer], all = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      mine[i] = hist[kBuckets - 1 - (tid * kPer + i)];
      all += mine[i];
    }
    uint32_t above = block_scan<T>(all, sums) - all;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (above < left && above + mine[i] >= left) {
        sh_bucket = kBuckets - 1 - (tid * kPer + i);
        sh_left = left - above;
        sh_count = mine[i];
      }
      above += mine[i];
    }
    __syncthreads();
    lo += sh_bucket << shift;
    hi = min(hi, lo + ((1u << shift) - 1));
    left = sh_left;
    whole = sh_count == left;
  }
  // Blocks above the range, and of the range's all or the first `left`.
  uint32_t n_above = 0, n_equal = 0;  // before this thread's
  // (Keys that are taken in any case lie above every score.)
  const uint32_t from = whole ? lo : hi + 1;
  auto place = [&](const uint32_t (&k)[8], const int (&id)[8], int base) {
    uint32_t up = 0, in = 0;  // the thread's blocks that are taken, and of the range
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      up |= (k[i] >= from ? 1u : 0u) << i;
      in |= (k[i] >= lo ? 1u : 0u) << i;
    }
    in &= ~up;
    const uint32_t mine = __popc(up) + (__popc(in) << 16);
    const uint32_t sum = block_scan<T>(mine, sums);
    uint32_t a = n_above + (sum & 0xffffu) - (mine & 0xffffu);
    uint32_t e = n_equal + (sum >> 16) - (mine >> 16);
    // Few lanes have any, and those one or two, as a rule.
    for (uint32_t rest = up | in; rest; rest &= rest - 1) {
      const int i = __ffs(rest) - 1;
      int phys = id[0];
#pragma unroll
      for (int z = 1; z < 8; ++z) phys = z == i ? id[z] : phys;
      if (up >> i & 1) {
        put_id((int)(a + min(e, left)), base + 8 * tid + i, phys);
        ++a;
      } else {
        if (e < left) put_id((int)(a + e), base + 8 * tid + i, phys);
        ++e;
      }
    }
    if (nblk <= 8 * T) return;
    // The CTA's total, for the blocks after these.
    __syncthreads();
    if (tid == T - 1) {
      sh_lo = n_above + (sum & 0xffffu);
      sh_hi = n_equal + (sum >> 16);
    }
    __syncthreads();
    n_above = sh_lo;
    n_equal = sh_hi;
  };
  if (whole) left = 0;
  place(first, ids, 0);
  for (int base = 8 * T; base < nblk; base += 8 * T) {
    uint32_t k[8];
    load(base, k);
    load_ids(base, ids);
    place(k, ids, base);
  }
}

__global__ void clear_kernel(DeviceStatus* status) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) *status = DeviceStatus{};
}

// ---- host side --------------------------------------------------------------------

// Longer runs of blocks a warp where there are still two rounds of CTAs (two run at
// once on an SM).
template <int D>
cudaError_t launch_scores(SelectParams p, cudaStream_t st) {
  const int64_t ctas = (int64_t)((p.max_blocks + 511) / 512) * p.Hkv * p.nb;
  const int steps = ctas >= 2 * 2 * 152 ? 4 : 2;
  const int groups = (p.Hkv + kWarps - 1) / kWarps;
  p.heads = p.G <= 8 ? (p.Hkv + groups - 1) / groups : 1;
  const int blocks = kWarps / p.heads * 16 * steps;
  const dim3 grid((unsigned)((p.max_blocks + blocks - 1) / blocks),
                  (unsigned)((p.Hkv + p.heads - 1) / p.heads), (unsigned)p.nb);
  auto launch = [&](auto kernel) { return launch_early(kernel, grid, 32 * kWarps, 0, st, p); };
  if (p.G <= 8)
    return launch(steps == 4 ? score_kernel<D, true, 4> : score_kernel<D, true, 2>);
  return launch(steps == 4 ? score_kernel<D, false, 4> : score_kernel<D, false, 2>);
}

int score_stride(int max_blocks) { return (max_blocks + 31) & ~31; }

size_t select_workspace(int64_t nb, int max_blocks, int Hkv) {
  return kStatusBytes + (size_t)nb * Hkv * score_stride(max_blocks) * 4;
}

kv_status shapes_ok(int32_t nb, int32_t max_blocks, int64_t num_blocks, int32_t Hkv,
                    int32_t d, int32_t block_size) {
  if (nb < 1 || max_blocks < 1 || Hkv < 1)
    return fail(KV_ERR_INVALID_ARG, "bad nb/max_blocks/Hkv (%d/%d/%d)", nb,
                max_blocks, Hkv);
  if (d != 64 && d != 128) return fail(KV_ERR_INVALID_ARG, "head_dim must be 64 or 128");
  if (block_size != 16) return fail(KV_ERR_INVALID_ARG, "block_size must be 16");
  if (max_blocks > INT32_MAX / 16)
    return fail(KV_ERR_INVALID_ARG, "max_blocks out of range");
  if (num_blocks < 1 || num_blocks > (int64_t)INT32_MAX / 16 / Hkv)
    return fail(KV_ERR_INVALID_ARG, "num_blocks out of range");
  return KV_OK;
}

kv_status run_bounds(const void* k_pool, const void* kv_scales, bool e4m3,
                     int64_t num_blocks, const int32_t* tables,
                     const int32_t* seq_lens, const int32_t* row_offsets,
                     int32_t total, int32_t nb, int32_t max_blocks, int32_t Hkv,
                     int32_t d, int32_t block_size, void* bounds,
                     float* bound_scales, void* workspace, size_t ws_bytes,
                     void* stream) {
  if (!k_pool || !tables || !seq_lens || !bounds || !bound_scales || !workspace ||
      (e4m3 && !kv_scales))
    return fail(KV_ERR_INVALID_ARG, "null argument");
  if (kv_status s = shapes_ok(nb, max_blocks, num_blocks, Hkv, d, block_size)) return s;
  if (total < 0 || (!row_offsets && total != nb))
    return fail(KV_ERR_INVALID_ARG, "total must be nb without row_offsets");
  if (((uintptr_t)k_pool | (uintptr_t)kv_scales | (uintptr_t)bounds) & 15 ||
      (uintptr_t)bound_scales & 3)
    return fail(KV_ERR_INVALID_ARG, "pool, scales and bounds must be 16-byte aligned");
  if ((uintptr_t)workspace & 255 || ws_bytes < kStatusBytes)
    return fail(KV_ERR_INVALID_ARG, "workspace: 256-byte aligned, >= 256 bytes");
  if (total == 0) return KV_OK;
  BoundsParams p;
  p.k = static_cast<const uint8_t*>(k_pool);
  p.scales = static_cast<const float4*>(kv_scales);
  p.tables = tables;
  p.seq_lens = seq_lens;
  p.row_offsets = row_offsets;
  p.bounds = static_cast<int8_t*>(bounds);
  p.bound_scales = bound_scales;
  p.status = static_cast<DeviceStatus*>(workspace);
  p.num_blocks = num_blocks;
  p.total = total;
  p.nb = nb;
  p.max_blocks = max_blocks;
  p.Hkv = Hkv;
  const int run = row_offsets ? 16 : 1;
  const int64_t runs = ((int64_t)total + run - 1) / run;
  // Measured, of 8 kv-heads: 30000 tiles of 2 KB 20 -> 17 us (d = 128 e4m3), 14 -> 12
  // (d = 64), 15.6 -> 11.3 (d = 64 e4m3); 12000 of them 9.7 -> 10.7.  Tiles of 4 KB are
  // better one a warp (27 us, two at a time 32).
  const int heads =
      runs * Hkv > 64 * 152 * 2 && Hkv >= 4 && (d == 64 || e4m3) ? 4 : 1;
  const int64_t ctas = (runs * ((Hkv + heads - 1) / heads) + 7) / 8;
  if (ctas > INT32_MAX) return fail(KV_ERR_INVALID_ARG, "too many tokens");
  cudaStream_t st = (cudaStream_t)stream;
  auto launch = [&](auto kernel) {
    return launch_early(kernel, (unsigned)ctas, 256, 0, st, p, run);
  };
  const cudaError_t e =
      d == 128 && e4m3
          ? launch(heads == 1 ? bounds_kernel<128, true, 1> : bounds_kernel<128, true, 4>)
      : d == 128 ? launch(bounds_kernel<128, false, 1>)
      : e4m3     ? launch(heads == 1 ? bounds_kernel<64, true, 1> : bounds_kernel<64, true, 4>)
                 : launch(heads == 1 ? bounds_kernel<64, false, 1> : bounds_kernel<64, false, 4>);
  if (e != cudaSuccess)
    return fail(KV_ERR_CUDA, "bounds kernel: %s", cudaGetErrorString(e));
  return KV_OK;
}

kv_status heads_ok(int32_t Hq, int32_t Hkv) {
  if (Hq < 1 || Hkv < 1 || Hq % Hkv != 0)
    return fail(KV_ERR_INVALID_ARG, "bad Hq/Hkv (%d/%d)", Hq, Hkv);
  if (Hq / Hkv > kMaxG)
    return fail(KV_ERR_INVALID_ARG, "more than %d query heads a kv-head", kMaxG);
  return KV_OK;
}

// The selected blocks of every (branch, kv-head) as a decode batch of its own.
kv_status virtual_batch(int32_t nb, int32_t Hq, int32_t Hkv, int64_t num_blocks) {
  if (kv_status s = heads_ok(Hq, Hkv)) return s;
  if (nb < 1 || (int64_t)nb * Hkv > INT32_MAX / 64)
    return fail(KV_ERR_INVALID_ARG, "nb x Hkv out of range");
  if (num_blocks < 1 || num_blocks > (int64_t)INT32_MAX / 16 / Hkv)
    return fail(KV_ERR_INVALID_ARG, "num_blocks out of range");
  return KV_OK;
}

// Blocks of a split-KV item.  Nothing is cut, and there is no merge, where that leaves
// work for the SMs: one item for most of them, of the e4m3 kernel, which needs more
// warps, three for two (128 blocks each, 256 items bf16 45 us, cut in three 53; 192
// items e4m3 44 us, in two 32), fewer of short ones (32 blocks, 80 items 10.1 us, cut in
// four 12.4).  A little more than the CTAs that run at once are halved (480 items bf16
// 99 -> 91 us, e4m3 86 -> 79).  Else all branches are about as long as the selection, so
// that items go by rounds of the CTAs that run at once.  An item costs about as much as
// kItem more blocks (its table entries and first loads), a piece of a branch kPiece (the
// merge's).
int32_t pick_cut(const std::vector<int32_t>& lens, int32_t G, bool e4m3,
                 int32_t num_sms) {
  constexpr double kItem = 14, kPiece = 1;
  const int64_t slots = (int64_t)kSplitCtasPerSm * num_sms;
  int32_t longest = 1, best = 1;
  for (const int32_t L : lens) longest = std::max(longest, (L + 15) / 16);
  const int64_t whole = (int64_t)lens.size() * ((G + kRowTile - 1) / kRowTile);
  const double few = longest <= 32 ? 0.5 : e4m3 ? 1.6 : 0.8;
  if (whole > slots && whole < slots + slots / 3) return (longest + 1) / 2;
  if ((double)whole >= few * num_sms) return longest;
  double least = 1e300;
  // From items of a whole branch (at most 256 blocks) down.
  for (int32_t cut = std::min(longest, 256); cut >= 8 || cut == std::min(longest, 256);
       cut = cut * 3 / 4) {
    int64_t n = 0;
    double total = 0;
    for (const int32_t L : lens) {
      const int64_t blocks = (L + 15) / 16;
      const int64_t pieces = (blocks + cut - 1) / cut * ((G + kRowTile - 1) / kRowTile);
      n += pieces;
      total += blocks * ((G + kRowTile - 1) / kRowTile) + pieces * kItem;
    }
    const double rounds = (double)((n + slots - 1) / slots);
    const double cost = std::max(std::min<double>(cut, longest) + kItem,
                                 n < 6 * slots ? rounds * (total / n) : total / slots) +
                        kPiece * ((longest + cut - 1) / cut);
    if (cost < least) {
      least = cost;
      best = cut;
    }
  }
  return best;
}

}  // namespace sel
}  // namespace pkv

using pkv::fail;

extern "C" kv_status paged_key_bounds(
    const void* k_pool, int64_t num_blocks, const int32_t* block_tables,
    const int32_t* seq_lens, const int32_t* row_offsets, int32_t total, int32_t nb,
    int32_t max_blocks, int32_t Hkv, int32_t head_dim, int32_t block_size,
    void* bounds, float* bound_scales, void* workspace, size_t ws_bytes,
    void* stream) {
  pkv::clear_error();
  return pkv::sel::run_bounds(k_pool, nullptr, false, num_blocks, block_tables,
                              seq_lens, row_offsets, total, nb, max_blocks, Hkv,
                              head_dim, block_size, bounds, bound_scales, workspace,
                              ws_bytes, stream);
}

extern "C" kv_status paged_key_bounds_e4m3(
    const void* k_pool, const void* kv_scales, int64_t num_blocks,
    const int32_t* block_tables, const int32_t* seq_lens, const int32_t* row_offsets,
    int32_t total, int32_t nb, int32_t max_blocks, int32_t Hkv, int32_t head_dim,
    int32_t block_size, void* bounds, float* bound_scales, void* workspace,
    size_t ws_bytes, void* stream) {
  pkv::clear_error();
  return pkv::sel::run_bounds(k_pool, kv_scales, true, num_blocks, block_tables,
                              seq_lens, row_offsets, total, nb, max_blocks, Hkv,
                              head_dim, block_size, bounds, bound_scales, workspace,
                              ws_bytes, stream);
}

extern "C" kv_status paged_select_blocks_workspace_size(int32_t nb,
                                                        int32_t max_blocks,
                                                        int32_t Hkv,
                                                        size_t* out_bytes) {
  pkv::clear_error();
  if (!out_bytes) return fail(KV_ERR_INVALID_ARG, "null argument");
  if (nb < 1 || max_blocks < 1 || max_blocks > INT32_MAX / 16 || Hkv < 1)
    return fail(KV_ERR_INVALID_ARG, "bad nb/max_blocks/Hkv (%d/%d/%d)", nb,
                max_blocks, Hkv);
  *out_bytes = pkv::sel::select_workspace(nb, max_blocks, Hkv);
  return KV_OK;
}

extern "C" kv_status paged_select_blocks(
    const void* q, const void* bounds, const float* bound_scales, int64_t num_blocks,
    const int32_t* block_tables, const int32_t* seq_lens, int32_t nb,
    int32_t max_blocks, int32_t Hq, int32_t Hkv, int32_t head_dim, int32_t block_size,
    int32_t n_sel, int32_t n_first, int32_t n_last, int32_t* sel, int32_t* sel_tables,
    int32_t* sel_lens, void* workspace, size_t ws_bytes, void* stream) {
  namespace S = pkv::sel;
  pkv::clear_error();
  if (!q || !bounds || !bound_scales || !block_tables || !seq_lens || !sel_tables ||
      !sel_lens || !workspace)
    return fail(KV_ERR_INVALID_ARG, "null argument");
  if (kv_status s =
          S::shapes_ok(nb, max_blocks, num_blocks, Hkv, head_dim, block_size))
    return s;
  if (kv_status s = S::heads_ok(Hq, Hkv)) return s;
  if (nb > 65535 || Hkv > 65535 || (int64_t)nb * Hkv > INT32_MAX / 64)
    return fail(KV_ERR_INVALID_ARG, "nb or Hkv out of range");
  if (n_first < 0 || n_last < 1 || n_sel < 1 || n_first > n_sel - n_last)
    return fail(KV_ERR_INVALID_ARG, "n_sel %d must hold n_first %d and n_last %d >= 1",
                n_sel, n_first, n_last);
  if (((uintptr_t)q | (uintptr_t)bounds) & 15 ||
      ((uintptr_t)bound_scales | (uintptr_t)sel | (uintptr_t)sel_tables |
       (uintptr_t)sel_lens) & 3)
    return fail(KV_ERR_INVALID_ARG, "q and bounds must be 16-byte aligned");
  const size_t need = S::select_workspace(nb, max_blocks, Hkv);
  if ((uintptr_t)workspace & 255 || ws_bytes < need)
    return fail(KV_ERR_INVALID_ARG, "workspace: 256-byte aligned, %zu bytes < %zu "
                "needed", ws_bytes, need);
  auto* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t st = (cudaStream_t)stream;
  S::SelectParams p;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.bounds = static_cast<const int8_t*>(bounds);
  p.bound_scales = bound_scales;
  p.tables = block_tables;
  p.seq_lens = seq_lens;
  p.status = reinterpret_cast<pkv::DeviceStatus*>(ws);
  p.scores = reinterpret_cast<float*>(ws + pkv::kStatusBytes);
  p.sel = sel;
  p.sel_tables = sel_tables;
  p.sel_lens = sel_lens;
  p.num_blocks = num_blocks;
  p.nb = nb;
  p.max_blocks = max_blocks;
  p.stride = S::score_stride(max_blocks);
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.n_sel = n_sel;
  p.n_first = n_first;
  p.n_last = n_last;
  cudaError_t e = max_blocks <= n_sel
                      ? pkv::launch_early(S::clear_kernel, 1, 32, 0, st, p.status)
                  : head_dim == 128 ? S::launch_scores<128>(p, st)
                                    : S::launch_scores<64>(p, st);
  // As many threads as hold a branch's keys at once.
  if (e == cudaSuccess)
    e = max_blocks <= 2048
            ? pkv::launch_early(S::pick_kernel<256>, nb * Hkv, 256, 0, st, p)
        : max_blocks <= 4096
            ? pkv::launch_early(S::pick_kernel<512>, nb * Hkv, 512, 0, st, p)
            : pkv::launch_early(S::pick_kernel<1024>, nb * Hkv, 1024, 0, st, p);
  if (e != cudaSuccess)
    return fail(KV_ERR_CUDA, "block selection: %s", cudaGetErrorString(e));
  return KV_OK;
}

extern "C" kv_status paged_selected_plan(int32_t nb, int32_t Hq, int32_t Hkv,
                                         int32_t head_dim, int32_t block_size,
                                         int32_t max_blocks, const int32_t* seq_lens,
                                         int32_t n_sel, int32_t num_sms,
                                         int32_t flags, int32_t* plan,
                                         int64_t plan_cap,
                                         kv_decode_plan_info* info) {
  pkv::clear_error();
  if (!info || !seq_lens) return fail(KV_ERR_INVALID_ARG, "null argument");
  if (kv_status s = pkv::sel::virtual_batch(nb, Hq, Hkv, 1)) return s;
  if (n_sel < 1 || n_sel > INT32_MAX / 16 || max_blocks < 1)
    return fail(KV_ERR_INVALID_ARG, "bad n_sel/max_blocks (%d/%d)", n_sel, max_blocks);
  if (block_size != 16) return fail(KV_ERR_INVALID_ARG, "block_size must be 16");
  if (flags & ~KV_PLAN_KV_E4M3)
    return fail(KV_ERR_INVALID_ARG, "unknown plan flags 0x%x", flags);
  try {
    std::vector<int32_t> lens((size_t)nb * Hkv);
    for (int32_t b = 0; b < nb; ++b) {
      const int32_t L = seq_lens[b];
      if (L < 1 || (int64_t)L > (int64_t)max_blocks * 16)
        return fail(KV_ERR_INVALID_ARG, "seq_lens[%d] = %d outside [1, %lld]", b, L,
                    (long long)max_blocks * 16);
      const int32_t nblk = (L - 1) / 16 + 1;
      const int32_t cut = nblk > n_sel ? (nblk - n_sel) * 16 : 0;
      std::fill_n(lens.begin() + (size_t)b * Hkv, Hkv, L - cut);
    }
    return pkv::decode_plan_of_rows(
        nb * Hkv, Hq / Hkv, head_dim, n_sel, lens.data(), num_sms, flags,
        pkv::sel::pick_cut(lens, Hq / Hkv, flags & KV_PLAN_KV_E4M3,
                           num_sms > 0 ? num_sms : 152),
        plan, plan_cap, info);
  } catch (const std::bad_alloc&) {
    return fail(KV_ERR_OOM, "no host memory for the plan");
  }
}

extern "C" kv_status paged_selected_attn(
    const void* q, const void* k_pool, const void* v_pool, int64_t num_blocks,
    const int32_t* sel_tables, const int32_t* sel_lens, int32_t nb, int32_t Hq,
    int32_t Hkv, int32_t head_dim, int32_t block_size, int32_t n_sel, float scale,
    void* out, const int32_t* plan, const kv_decode_plan_info* info, void* workspace,
    size_t ws_bytes, void* stream) {
  pkv::clear_error();
  if (kv_status s = pkv::sel::virtual_batch(nb, Hq, Hkv, num_blocks)) return s;
  return pkv::decode_selected(q, k_pool, v_pool, nullptr, num_blocks * Hkv, sel_tables,
                              sel_lens, nb * Hkv, n_sel, Hq / Hkv, head_dim, block_size,
                              scale, out, plan, info, workspace, ws_bytes, stream);
}

extern "C" kv_status paged_selected_attn_e4m3(
    const void* q, const void* k_pool, const void* v_pool, const void* kv_scales,
    int64_t num_blocks, const int32_t* sel_tables, const int32_t* sel_lens,
    int32_t nb, int32_t Hq, int32_t Hkv, int32_t head_dim, int32_t block_size,
    int32_t n_sel, float scale, void* out, const int32_t* plan,
    const kv_decode_plan_info* info, void* workspace, size_t ws_bytes, void* stream) {
  pkv::clear_error();
  if (kv_status s = pkv::sel::virtual_batch(nb, Hq, Hkv, num_blocks)) return s;
  if (!kv_scales) return fail(KV_ERR_INVALID_ARG, "kv_scales required");
  return pkv::decode_selected(q, k_pool, v_pool, kv_scales, num_blocks * Hkv,
                              sel_tables, sel_lens, nb * Hkv, n_sel, Hq / Hkv,
                              head_dim, block_size, scale, out, plan, info, workspace,
                              ws_bytes, stream);
}
