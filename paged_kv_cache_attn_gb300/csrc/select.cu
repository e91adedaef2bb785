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

// Bounds of the first `valid` slots of one (block, head) tile, by one warp.  A lane
// has kPer dimensions (16 bytes) of every kRows-th row.
template <int D, bool E4M3>
__device__ __forceinline__ void tile_bounds(const BoundsParams& p, int64_t tile,
                                            int valid, int lane) {
  constexpr int kPer = E4M3 ? 16 : 8;
  constexpr int kChunks = D / kPer;      // 16-byte chunks of a row
  constexpr int kRows = 32 / kChunks;    // rows of a load
  constexpr int kLoads = 16 / kRows;
  const int c = lane % kChunks, r0 = lane / kChunks;
  const uint8_t* src = p.k + tile * (16 * D * (E4M3 ? 1 : 2));
  uint4 x[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    // Slots past the branch's length: its last token again.
    const int t = min(i * kRows + r0, valid - 1);
    const int at = E4M3 ? t * D + ((D == 128 ? c ^ (t & 7) : c) << 4)
                        : (t * kChunks + c) * 16;
    x[i] = *reinterpret_cast<const uint4*>(src + at);
  }
  float scale = 1.f;
  if (E4M3) scale = p.scales[tile].x;
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
#pragma unroll
  for (int o = kChunks; o < 32; o <<= 1) {
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
      const uint32_t a = __shfl_xor_sync(0xffffffffu, lo[k], o);
      const uint32_t b = __shfl_xor_sync(0xffffffffu, hi[k], o);
      lo[k] = E4M3 ? min2h(lo[k], a) : min2(lo[k], a);
      hi[k] = E4M3 ? max2h(hi[k], b) : max2(hi[k], b);
    }
  }
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
  for (int k = 0; k < kPairs; ++k)
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const float a = fabsf(value(lo[k], z)), b = fabsf(value(hi[k], z));
      odd |= !(a < INFINITY) || !(b < INFINITY);
      amax = fmaxf(amax, fmaxf(a, b));
    }
#pragma unroll
  for (int o = 1; o < kChunks; o <<= 1)
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  odd = __any_sync(0xffffffffu, odd);
  const int e = bound_exponent(amax);
  const float inv = pow2f(-e);
  // The first lanes of a row's chunks write the least, the next the largest.
  const bool upper = r0 == 1;
  uint32_t out[kPer / 4];
#pragma unroll
  for (int k = 0; k < kPer / 4; ++k) {
    uint32_t w = 0;
#pragma unroll
    for (int z = 0; z < 4; ++z) {
      const float v = value((upper ? hi : lo)[2 * k + z / 2], z & 1) * inv;
      float n = upper ? ceilf(v) : floorf(v);
      n = odd ? 0.f : fminf(fmaxf(n, -127.f), 127.f);
      w |= (uint32_t)((int)n & 0xff) << (8 * z);
    }
    out[k] = w;
  }
  if (r0 < 2) {
    int8_t* dst = p.bounds + tile * (2 * D) + r0 * D + c * kPer;
    if constexpr (E4M3)
      *reinterpret_cast<uint4*>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
    else
      *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
  }
  // A block with a value that is not finite has a score above all others.
  if (lane == 0) p.bound_scales[tile] = odd ? INFINITY : pow2f(e);
}

// A warp for each (run of new tokens, kv-head): every block that a token of the run
// is the first new one of.  kRun: tokens of a run (steps of one token a branch: 1).
template <int D, bool E4M3>
__global__ void __launch_bounds__(256) bounds_kernel(const BoundsParams p, int run) {
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int64_t tok0 = w / p.Hkv * run;
  const int h = (int)(w % p.Hkv);
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
        tile_bounds<D, E4M3>(p, (int64_t)phys * p.Hkv + h,
                             min(16, L - (int)(pos & ~15ll)), lane);
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
constexpr int kWarpBlocks = 32;                       // blocks a warp scores
constexpr int kCtaBlocks = kWarps * kWarpBlocks;

// grid (block ranges, Hkv, nb).  The heads are the 16 rows of the products, eight
// blocks their columns; lane 4 n + t has bytes [16 t + 64 j, + 16) of block n's
// record, which are its columns of four products in any order that the queries'
// fragments share.
template <int D>
__global__ void __launch_bounds__(256) score_kernel(const SelectParams p) {
  constexpr int kRow = D + 8;  // a head's f16 values in shared memory
  __shared__ __align__(16) __half qs[kMaxG * kRow];
  __shared__ float qe[kMaxG];
  const int b = blockIdx.z, h = blockIdx.y;
  const int L = p.seq_lens[b];
  const int nblk = L < 1 || L > (int64_t)p.max_blocks * 16 ? 0 : (L + 15) / 16;
  // A branch of few blocks has them all.
  if (nblk <= p.n_sel || blockIdx.x * kCtaBlocks >= nblk) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int blk0 = blockIdx.x * kCtaBlocks + warp * kWarpBlocks;
  const int32_t* table = p.tables + (int64_t)b * p.max_blocks;
  int phys = -1;
  if (blk0 + lane < nblk) {
    phys = table[blk0 + lane];
    if (phys < 0 || phys >= p.num_blocks) {
      record_status(p.status, KV_ERR_DEVICE, phys);
      phys = -1;
    }
  }
  // Queries: a warp quantises a head at a time; heads of the last 16 that there
  // are not are zeros.
  const int G = p.G, rows = (G + 15) & ~15;
  for (int g = warp; g < rows; g += kWarps) {
    constexpr int V = D / 32;
    float x[V], amax = 0.f;
    bool odd = false;
    const __nv_bfloat16* src =
        p.q + ((int64_t)b * p.Hq + (int64_t)h * G + min(g, G - 1)) * D + lane * V;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      x[i] = g < G ? __bfloat162float(src[i]) : 0.f;
      odd |= !(fabsf(x[i]) < INFINITY);
      amax = fmaxf(amax, fabsf(x[i]));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    odd = __any_sync(0xffffffffu, odd);
    const int e = bound_exponent(amax);
    const float inv = pow2f(-e);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float n = odd ? 0.f : fminf(fmaxf(rintf(x[i] * inv), -127.f), 127.f);
      qs[g * kRow + lane * V + i] = __float2half_rn(n);
    }
    if (lane == 0) qe[g] = g < G ? (odd ? 0.f : pow2f(e)) : -1.f;
  }
  __syncthreads();
  if (blk0 >= nblk) return;
  const int n = lane >> 2, t = lane & 3;
  constexpr int kJ = 2 * D / 64;  // 64-byte parts of a record
  uint4 rec[4][kJ];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int ph = __shfl_sync(0xffffffffu, phys, i * 8 + n);
    const uint4* src = reinterpret_cast<const uint4*>(
        p.bounds + ((int64_t)max(ph, 0) * p.Hkv + h) * (2 * D));
#pragma unroll
    for (int j = 0; j < kJ; ++j) rec[i][j] = src[j * 4 + t];
  }
  const float my_scale =
      phys >= 0 ? p.bound_scales[(int64_t)phys * p.Hkv + h] : 0.f;
  float best[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) best[i][0] = best[i][1] = -INFINITY;
  for (int g0 = 0; g0 < rows; g0 += 16) {
    float acc[4][4] = {};
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      // The least values meet the queries' negative numbers, the largest the
      // positive ones.
      const int col = (j * 64) % D + t * 16;
      const bool neg = j < kJ / 2;
      uint32_t f[2][8];
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const __half* src = qs + (g0 + z * 8 + n) * kRow + col;
        const uint4 v0 = *reinterpret_cast<const uint4*>(src);
        const uint4 v1 = *reinterpret_cast<const uint4*>(src + 8);
        const uint32_t v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
        for (int k = 0; k < 8; ++k) f[z][k] = neg ? min2h(v[k], 0u) : max2h(v[k], 0u);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w[4] = {rec[i][j].x, rec[i][j].y, rec[i][j].z, rec[i][j].w};
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          uint32_t b0, b1;
          bytes_to_f16(w[s], b0, b1);
          const uint32_t a[4] = {f[0][2 * s], f[1][2 * s], f[0][2 * s + 1],
                                 f[1][2 * s + 1]};
          mma_f16(acc[i], a, b0, b1);
        }
      }
    }
    const float e0 = qe[g0 + n], e1 = qe[g0 + 8 + n];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const float s0 = e0 < 0.f ? -INFINITY : acc[i][z] * e0;
        const float s1 = e1 < 0.f ? -INFINITY : acc[i][2 + z] * e1;
        best[i][z] = fmaxf(best[i][z], fmaxf(s0, s1));
      }
  }
  float* dst = p.scores + ((int64_t)b * p.Hkv + h) * p.stride;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      float s = best[i][z];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1)
        s = fmaxf(s, __shfl_xor_sync(0xffffffffu, s, o));
      const float sc = __shfl_sync(0xffffffffu, my_scale, i * 8 + 2 * t + z);
      const int blk = blk0 + i * 8 + 2 * t + z;
      // (+ 0 makes a zero positive.)
      if (n == 0 && blk < nblk)
        dst[blk] = sc == INFINITY ? INFINITY : s * sc + 0.f;
    }
}

// ---- selection --------------------------------------------------------------------

__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

constexpr int kPickThreads = 256, kPickWarps = 8;

// A CTA for each (branch, kv-head): the n_sel-th largest key digit by digit (8
// bits), then the blocks above it and the first of those equal to it, in order.
__global__ void __launch_bounds__(kPickThreads) pick_kernel(const SelectParams p) {
  __shared__ uint32_t hist[kPickWarps][256];
  __shared__ uint32_t sh_digit, sh_left;
  __shared__ int above[kPickWarps], equal[kPickWarps];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int row = blockIdx.x, b = row / p.Hkv, h = row % p.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int L = p.seq_lens[b];
  const int32_t* table = p.tables + (int64_t)b * p.max_blocks;
  int32_t* sel = p.sel ? p.sel + (int64_t)row * p.n_sel : nullptr;
  int32_t* out = p.sel_tables + (int64_t)row * p.n_sel;
  const bool bad = L < 1 || L > (int64_t)p.max_blocks * 16;
  if (bad && threadIdx.x == 0) record_status(p.status, KV_ERR_DEVICE, L);
  const int nblk = bad ? 0 : (L + 15) / 16;
  const int count = min(nblk, p.n_sel);
  auto put = [&](int at, int blk) {
    const int phys = table[blk];
    const bool in = phys >= 0 && phys < p.num_blocks;
    if (!in) record_status(p.status, KV_ERR_DEVICE, phys);
    if (sel) sel[at] = blk;
    out[at] = in ? (int)(phys * (int64_t)p.Hkv + h) : -1;
  };
  if (threadIdx.x == 0)
    p.sel_lens[row] = count > 0 ? 16 * (count - 1) + (L - 16 * (nblk - 1)) : 0;
  for (int i = count + threadIdx.x; i < p.n_sel; i += kPickThreads) {
    if (sel) sel[i] = -1;
    out[i] = -1;
  }
  if (nblk <= p.n_sel) {
    for (int i = threadIdx.x; i < nblk; i += kPickThreads) put(i, i);
    return;
  }
  const float* scores = p.scores + (int64_t)row * p.stride;
  auto key = [&](int i) -> uint32_t {
    if (i < p.n_first || i >= nblk - p.n_last) return 0xffffffffu;
    return ordered(scores[i]);
  };
  // The digits of the n_sel-th largest key; `left`: how many of the keys that begin
  // with the digits so far are wanted.
  uint32_t prefix = 0, left = (uint32_t)p.n_sel;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < kPickWarps * 256; i += kPickThreads)
      (&hist[0][0])[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < nblk; i += kPickThreads) {
      const uint32_t k = key(i);
      if (shift == 24 || (k >> (shift + 8)) == prefix)
        atomicAdd(&hist[warp][(k >> shift) & 255], 1u);
    }
    __syncthreads();
    // Thread t: keys of digit 255 - t, and of all above it.
    uint32_t n = 0;
    for (int w = 0; w < kPickWarps; ++w) n += hist[w][255 - threadIdx.x];
    uint32_t sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    if (lane == 31) above[warp] = (int)sum;
    __syncthreads();
    for (int w = 0; w < warp; ++w) sum += (uint32_t)above[w];
    if (sum >= left && sum - n < left) {
      sh_digit = 255 - threadIdx.x;
      sh_left = left - (sum - n);
    }
    __syncthreads();
    prefix = prefix << 8 | sh_digit;
    left = sh_left;
    __syncthreads();
  }
  // Each warp a run of blocks: counts, then places.
  const int run = ((nblk + kPickWarps - 1) / kPickWarps + 31) & ~31;
  const int i0 = warp * run, i1 = min(i0 + run, nblk);
  int n_above = 0, n_equal = 0;
  for (int i = i0; i < i1; i += 32) {
    const uint32_t k = i + lane < i1 ? key(i + lane) : 0;
    n_above += __popc(__ballot_sync(0xffffffffu, i + lane < i1 && k > prefix));
    n_equal += __popc(__ballot_sync(0xffffffffu, i + lane < i1 && k == prefix));
  }
  if (lane == 0) {
    above[warp] = n_above;
    equal[warp] = n_equal;
  }
  __syncthreads();
  n_above = n_equal = 0;
  for (int w = 0; w < warp; ++w) {
    n_above += above[w];
    n_equal += equal[w];
  }
  const uint32_t below = (1u << lane) - 1;
  for (int i = i0; i < i1; i += 32) {
    const uint32_t k = i + lane < i1 ? key(i + lane) : 0;
    const uint32_t m1 = __ballot_sync(0xffffffffu, i + lane < i1 && k > prefix);
    const uint32_t m2 = __ballot_sync(0xffffffffu, i + lane < i1 && k == prefix);
    const int a = n_above + __popc(m1 & below), e = n_equal + __popc(m2 & below);
    const bool mine = (m1 >> lane & 1) || ((m2 >> lane & 1) && e < (int)left);
    if (mine) put(a + min(e, (int)left), i + lane);
    n_above += __popc(m1);
    n_equal += __popc(m2);
  }
}

__global__ void clear_kernel(DeviceStatus* status) {
  if (threadIdx.x == 0) *status = DeviceStatus{};
}

// ---- host side --------------------------------------------------------------------

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
  const int64_t ctas = (((int64_t)total + run - 1) / run * Hkv + 7) / 8;
  if (ctas > INT32_MAX) return fail(KV_ERR_INVALID_ARG, "too many tokens");
  cudaStream_t st = (cudaStream_t)stream;
  if (d == 128 && e4m3)
    bounds_kernel<128, true><<<(unsigned)ctas, 256, 0, st>>>(p, run);
  else if (d == 128)
    bounds_kernel<128, false><<<(unsigned)ctas, 256, 0, st>>>(p, run);
  else if (e4m3)
    bounds_kernel<64, true><<<(unsigned)ctas, 256, 0, st>>>(p, run);
  else
    bounds_kernel<64, false><<<(unsigned)ctas, 256, 0, st>>>(p, run);
  const cudaError_t e = cudaGetLastError();
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
  S::clear_kernel<<<1, 32, 0, st>>>(p.status);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && max_blocks > n_sel) {
    const dim3 grid((unsigned)((max_blocks + S::kCtaBlocks - 1) / S::kCtaBlocks),
                    (unsigned)Hkv, (unsigned)nb);
    if (head_dim == 128)
      S::score_kernel<128><<<grid, 256, 0, st>>>(p);
    else
      S::score_kernel<64><<<grid, 256, 0, st>>>(p);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess)
    e = pkv::launch_early(S::pick_kernel, nb * Hkv, S::kPickThreads, 0, st, p);
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
    return paged_decode_plan(nb * Hkv, Hq / Hkv, 1, head_dim, block_size, n_sel,
                             lens.data(), nullptr, 0, num_sms,
                             flags | KV_PLAN_IGNORE_GROUPS, plan, plan_cap, info);
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
  return paged_decode_attn(q, k_pool, v_pool, num_blocks * Hkv, sel_tables, sel_lens,
                           nullptr, 0, nb * Hkv, n_sel, Hq / Hkv, 1, head_dim,
                           block_size, scale, out, plan, info, workspace, ws_bytes,
                           stream);
}

extern "C" kv_status paged_selected_attn_e4m3(
    const void* q, const void* k_pool, const void* v_pool, const void* kv_scales,
    int64_t num_blocks, const int32_t* sel_tables, const int32_t* sel_lens,
    int32_t nb, int32_t Hq, int32_t Hkv, int32_t head_dim, int32_t block_size,
    int32_t n_sel, float scale, void* out, const int32_t* plan,
    const kv_decode_plan_info* info, void* workspace, size_t ws_bytes, void* stream) {
  pkv::clear_error();
  if (kv_status s = pkv::sel::virtual_batch(nb, Hq, Hkv, num_blocks)) return s;
  return paged_decode_attn_e4m3(q, k_pool, v_pool, kv_scales, num_blocks * Hkv,
                                sel_tables, sel_lens, nullptr, 0, nb * Hkv, n_sel,
                                Hq / Hkv, 1, head_dim, block_size, scale, out, plan,
                                info, workspace, ws_bytes, stream);
}
