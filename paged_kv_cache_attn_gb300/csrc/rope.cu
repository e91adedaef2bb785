// Position rotation on the way into a paged cache: paged_rope_append,
// paged_rope_append_e4m3 and paged_latent_append.
//
// A layer's projections give unrotated queries and keys of the new tokens.
// Token i of branch b's new tokens sits at position p = seq_lens[b] - n_b + i
// (its slot was reserved beforehand), and each pair of dimensions (a, b) is
// turned by the angle whose (cos, sin) is row p of the caller's table:
//   y_a = x_a cos - x_b sin,   y_b = x_b cos + x_a sin,
// computed in fp32 and rounded once, to bf16 or to the e4m3 code of the
// block's scale.  Queries go to q_out, keys and values to their slots.
//
// Every value is read once and written once, so the calls are bound by HBM on
// prompts and by the launch and one chain of dependent loads (offsets, length,
// table entry, table row) on a decode step.  Measured: 4 prompts of 4096 tokens
// with 64 + 8 + 8 heads of 128 in 118 us (5.7 TB/s), five of about 2000 latent
// tokens with 16 heads' queries in 18.5 us (3.7 TB/s: 1279 CTAs, three an SM at 80
// registers, are 2.8 waves, and every warp of each goes through that chain for its
// token), steps of 64 (bf16) and of 128 branches (latent) in 6.2 us, a step of 64
// branches into an e4m3 pool in 8.3 us (the chain, then a warp's maximum, the block's
// scale and the codes).

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "device_common.cuh"
#include "e4m3.cuh"
#include "tensor_map.h"

namespace pkv {
namespace rope {

// Where a token of a batch lives.
struct TokenMap {
  const int32_t* tables;
  const int32_t* seq_lens;
  const int32_t* off;  // [nb + 1] first new token of each branch; null: one each
  DeviceStatus* status;
  int64_t num_blocks;
  int nb, total, max_blocks, rope_len;
};

struct Token {
  int pos, phys, first, n;  // position, block, branch's first token, its count
  bool ok;
};

// Warp-wide: the last branch whose first token is <= t, 32 candidates at a time.
__device__ __forceinline__ int find_branch(const TokenMap& m, int t, int lane) {
  int lo = 0, hi = m.nb;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int idx = lo + lane * step;
    const bool le = idx < hi && m.off[idx] <= t;
    const int cnt = __popc(__ballot_sync(0xffffffffu, le));
    lo += max(cnt - 1, 0) * step;
    hi = min(lo + step, hi);
  }
  return lo;
}

// Position and block of token t of branch b.  A token whose branch, position
// or block is out of range is recorded (by the calling threads with `tell`) and
// not ok.
__device__ __forceinline__ Token place(const TokenMap& m, int t, int b,
                                       bool tell) {
  Token k;
  k.first = m.off ? m.off[b] : t;
  k.n = m.off ? m.off[b + 1] - k.first : 1;
  k.pos = m.seq_lens[b] - k.n + (t - k.first);
  k.phys = -1;
  k.ok = t >= k.first && t - k.first < k.n && k.pos >= 0 && k.pos < m.rope_len &&
         (k.pos >> 4) < m.max_blocks;
  int bad = k.pos;
  if (k.ok) {
    k.phys = m.tables[(int64_t)b * m.max_blocks + (k.pos >> 4)];
    bad = k.phys;
    k.ok = k.phys >= 0 && (int64_t)k.phys < m.num_blocks;
  }
  if (!k.ok && tell) record_status(m.status, KV_ERR_DEVICE, bad);
  return k;
}

// Warp-wide, the same token for all lanes.
__device__ __forceinline__ Token locate(const TokenMap& m, int t, int lane) {
  return place(m, t, m.off ? find_branch(m, t, lane) : t, lane == 0);
}

// Rows of D values handled alike ("heads" of a token).  Destination of head
// h: dst + t * dst_token + phys * dst_block + slot * dst_slot + h * dst_head.
struct Rows {
  const __nv_bfloat16* src;
  __nv_bfloat16* dst;
  int64_t src_token, src_head;
  int64_t dst_token, dst_block, dst_slot, dst_head;
  int heads;
  int rotate;
};

struct RotateArgs {
  TokenMap map;
  Rows rows[3];  // queries, keys, values
  const float2* table;  // [rope_len][half] (cos, sin)
  int half;             // rotated pairs
  int split;            // warps a token
};

// The 8 values of this lane's vector, rotated.  HALVES: the partner of
// dimension j < half is j + half, half / 8 lanes away; PAIRS: neighbours.
template <bool PAIRS>
__device__ __forceinline__ uint4 rotate8(uint4 v, const float (&c)[8],
                                         const float (&s)[8], int half8,
                                         int vec, bool rot, int lane) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  uint32_t y[4];
  if constexpr (PAIRS) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      y[i] = pack_bf16(fmaf(x[2 * i], c[i], -(x[2 * i + 1] * s[i])),
                       fmaf(x[2 * i + 1], c[i], x[2 * i] * s[i]));
  } else {
    const bool low = vec < half8;
    const int mate = low ? lane + half8 : lane - half8;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t o = __shfl_sync(0xffffffffu, w[i], mate & 31);
      const float p0 = __uint_as_float(o << 16);
      const float p1 = __uint_as_float(o & 0xffff0000u);
      const float s0 = low ? -s[2 * i] : s[2 * i];
      const float s1 = low ? -s[2 * i + 1] : s[2 * i + 1];
      y[i] = pack_bf16(fmaf(x[2 * i], c[2 * i], p0 * s0),
                       fmaf(x[2 * i + 1], c[2 * i + 1], p1 * s1));
    }
  }
  return rot ? make_uint4(y[0], y[1], y[2], y[3]) : v;
}

// One warp's share of a token: a lane holds one 16-byte vector (8
// dimensions), a warp 256 / D heads, and the (cos, sin) of the lane's
// dimensions stay in registers over all heads.  Four vectors are loaded
// before the first is written, so that 2 KB a warp are in flight.
template <int D, bool PAIRS>
__device__ __forceinline__ void rotate_share(const RotateArgs& a, int t,
                                             int share, int lane) {
  constexpr int kVecs = D / 8, kHeads = 32 / kVecs;
  const Token k = locate(a.map, t, lane);
  if (!k.ok) return;
  const int vec = lane % kVecs, sub = lane / kVecs;
  const int half8 = a.half / 8;
  const bool rot = vec * 8 < 2 * a.half;
  float c[8], s[8];
  {
    const float2* row = a.table + (int64_t)k.pos * a.half;
    const int j0 = PAIRS ? vec * 4 : (vec < half8 ? vec : vec - half8) * 8;
    constexpr int n = PAIRS ? 4 : 8;
#pragma unroll
    for (int i = 0; i < n; i += 2) {
      const float4 f = rot ? __ldg(reinterpret_cast<const float4*>(row + j0 + i))
                           : make_float4(1.f, 0.f, 1.f, 0.f);
      c[i] = f.x;
      s[i] = f.y;
      c[i + 1] = f.z;
      s[i + 1] = f.w;
    }
  }
  int n_it[3];
#pragma unroll
  for (int r = 0; r < 3; ++r) n_it[r] = (a.rows[r].heads + kHeads - 1) / kHeads;
  const int total = n_it[0] + n_it[1] + n_it[2];
  constexpr int U = 4;
  for (int i0 = share; i0 < total; i0 += U * a.split) {
    uint4 v[U];
    __nv_bfloat16* dst[U];
    bool rt[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      int i = i0 + u * a.split;
      const int w = i < n_it[0] ? 0 : i < n_it[0] + n_it[1] ? 1 : 2;
      const Rows& r = a.rows[w];
      const int h = (i - (w > 0 ? n_it[0] : 0) - (w > 1 ? n_it[1] : 0)) * kHeads + sub;
      dst[u] = nullptr;
      rt[u] = r.rotate && rot;
      v[u] = make_uint4(0, 0, 0, 0);
      if (i < total && h < r.heads) {
        v[u] = *reinterpret_cast<const uint4*>(r.src + t * r.src_token +
                                               h * r.src_head + vec * 8);
        dst[u] = r.dst + t * r.dst_token + k.phys * r.dst_block +
                 (k.pos & 15) * r.dst_slot + h * r.dst_head + vec * 8;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint4 y = rotate8<PAIRS>(v[u], c, s, half8, vec, rt[u], lane);
      if (dst[u]) *reinterpret_cast<uint4*>(dst[u]) = y;
    }
  }
}

template <int D, bool PAIRS>
__global__ void __launch_bounds__(256)
    rotate_kernel(const __grid_constant__ RotateArgs a) {
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t t = w / a.split;
  if (t < a.map.total)
    rotate_share<D, PAIRS>(a, (int)t, (int)(w - t * a.split), threadIdx.x & 31);
  // Beside a quantising launch (below) it runs with that one, which has to be
  // complete when this one is.
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ---- e4m3 pools ---------------------------------------------------------------

constexpr int kQuantWarps = 4;

struct QuantArgs {
  RotateArgs rot;  // queries only (rows[0])
  int q_ctas;      // CTAs of the rotation part
  int window;      // tokens a quantising CTA looks at
  const __nv_bfloat16* k_new;
  const __nv_bfloat16* v_new;
  int64_t k_token, v_token;
  uint8_t* k8;
  uint8_t* v8;
  float4* scales;
  int Hkv;
};

// Two codes, `lo` in the lower byte: nearest, ties to even, saturating (the
// conversion of e4m3_encode, two values at a time).
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t join16(uint32_t lo, uint32_t hi) {
  return __byte_perm(lo, hi, 0x5410);
}

// Where one warp's write goes and comes from.
struct QuantTile {
  uint8_t* codes;
  float* scale;
  const __nv_bfloat16* src;  // this lane's values of the first row
  int64_t stride;
  const float2* table;       // the first row's (cos, sin)
  int c0;                    // this lane's first dimension
  bool is_v, rot, low;
};

// This lane's V values of R rows (row min(r, m - 1) as the r-th), rotated for
// keys.  All the rows are asked for before the first is used, and all of their
// (cos, sin) next: taken row by row, a tile waited for memory sixteen times.
template <int D, bool PAIRS, int R>
__device__ __forceinline__ void quant_rows(const QuantTile& q, int m, int half,
                                           int lane, float (&x)[R][D / 32]) {
  constexpr int V = D / 32;
  uint32_t raw[R][V / 2];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const __nv_bfloat16* at = q.src + min(r, m - 1) * q.stride;
    if constexpr (V == 4) {
      const uint2 u = __ldg(reinterpret_cast<const uint2*>(at));
      raw[r][0] = u.x;
      raw[r][1] = u.y;
    } else {
      raw[r][0] = __ldg(reinterpret_cast<const uint32_t*>(at));
    }
  }
  auto value = [&](int r, int i) {
    return __uint_as_float(i & 1 ? raw[r][i / 2] & 0xffff0000u : raw[r][i / 2] << 16);
  };
  if (q.is_v) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < V; ++i) x[r][i] = value(r, i);
    return;
  }
  const int j0 = PAIRS ? q.c0 / 2 : q.low ? q.c0 : q.c0 - half;
  const float2* row = q.table + (q.rot ? j0 : 0);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float2* at = row + (int64_t)min(r, m - 1) * half;
    if constexpr (PAIRS) {
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const float2 f = __ldg(at + i / 2);
        const float a = value(r, i), b = value(r, i + 1);
        x[r][i] = q.rot ? fmaf(a, f.x, -(b * f.y)) : a;
        x[r][i + 1] = q.rot ? fmaf(b, f.x, a * f.y) : b;
      }
    } else {
      const int mate = (q.low ? lane + half / V : lane - half / V) & 31;
      uint32_t o[V / 2];
#pragma unroll
      for (int i = 0; i < V / 2; ++i) o[i] = __shfl_sync(0xffffffffu, raw[r][i], mate);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float2 f = __ldg(at + i);
        const float a = value(r, i);
        const float b = __uint_as_float(i & 1 ? o[i / 2] & 0xffff0000u : o[i / 2] << 16);
        x[r][i] = q.rot ? fmaf(a, f.x, b * (q.low ? -f.y : f.y)) : a;
      }
    }
  }
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// A whole block (16 rows from slot 0), nearly every write of a prompt: the
// rows stay in registers between the maximum and the codes.
template <int D, bool PAIRS>
__device__ __forceinline__ void quant_block(const QuantTile& q, int half,
                                            int lane) {
  constexpr int V = D / 32;  // values per lane and row
  float x[16][V];
  quant_rows<D, PAIRS, 16>(q, 16, half, lane, x);
  float m4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int t = 0; t < 16; ++t)
#pragma unroll
    for (int i = 0; i < V; ++i) m4[t & 3] = fmaxf(m4[t & 3], fabsf(x[t][i]));
  const int e = e4m3_exponent_for(
      warp_max(fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]))));
  const float inv = pow2f(-e);
  if (!q.is_v) {
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      uint8_t* at = q.codes + k_tile_offset(t, q.c0, D);
      const uint32_t lo = e4m3x2(x[t][0] * inv, x[t][1] * inv);
      if constexpr (V == 4)
        *reinterpret_cast<uint32_t*>(at) =
            join16(lo, e4m3x2(x[t][2] * inv, x[t][3] * inv));
      else
        *reinterpret_cast<uint16_t*>(at) = (uint16_t)lo;
    }
  } else {
    // Transposed tile: the 16 slots of a dimension are 16 contiguous bytes.
#pragma unroll
    for (int i = 0; i < V; ++i) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = join16(e4m3x2(x[4 * k][i] * inv, x[4 * k + 1][i] * inv),
                      e4m3x2(x[4 * k + 2][i] * inv, x[4 * k + 3][i] * inv));
      *reinterpret_cast<uint4*>(q.codes + v_tile_offset(0, q.c0 + i)) =
          make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  if (lane == 0) *q.scale = pow2f(e);
}

// The rows already stored, slots [0, s0), move by an exponent (a pure shift of
// their stored values).  All of a lane's codes are loaded before the first is
// written back.
template <int D>
__device__ __forceinline__ void shift_rows(const QuantTile& q, int s0, int sh) {
  constexpr int V = D / 32;
  auto moved = [&](uint32_t w, int n) {  // the n lowest codes of a word
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i >= n) break;
      const float v = ldexpf(e4m3_decode((uint8_t)(w >> (8 * i))), sh);
      w = (w & ~(0xffu << (8 * i))) | ((uint32_t)e4m3_encode(v) << (8 * i));
    }
    return w;
  };
  if (!q.is_v) {
    uint32_t w[15];
#pragma unroll
    for (int t = 0; t < 15; ++t) {
      const uint8_t* at = q.codes + k_tile_offset(t, q.c0, D);
      if (t < s0)
        w[t] = V == 4 ? *reinterpret_cast<const uint32_t*>(at)
                      : *reinterpret_cast<const uint16_t*>(at);
    }
#pragma unroll
    for (int t = 0; t < 15; ++t) {
      uint8_t* at = q.codes + k_tile_offset(t, q.c0, D);
      if (t >= s0) break;
      if constexpr (V == 4)
        *reinterpret_cast<uint32_t*>(at) = moved(w[t], 4);
      else
        *reinterpret_cast<uint16_t*>(at) = (uint16_t)moved(w[t], 2);
    }
  } else {
    uint4 v[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
      v[i] = *reinterpret_cast<const uint4*>(q.codes + v_tile_offset(0, q.c0 + i));
#pragma unroll
    for (int i = 0; i < V; ++i) {
      uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = moved(w[k], min(max(s0 - 4 * k, 0), 4));
      *reinterpret_cast<uint4*>(q.codes + v_tile_offset(0, q.c0 + i)) =
          make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// Slots [s0, s0 + m) of a block, m <= R (a decode step's token: R = 1; the ends
// of a chunk: 16).
template <int D, bool PAIRS, int R>
__device__ __forceinline__ void quant_part(const QuantTile& q, int s0, int m,
                                           int half, int lane) {
  constexpr int V = D / 32;
  float x[R][V];
  float amax = 0.f;
  quant_rows<D, PAIRS, R>(q, m, half, lane, x);  // rows past m: the last again
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < V; ++i) amax = fmaxf(amax, fabsf(x[r][i]));
  int e = e4m3_exponent_for(warp_max(amax));
  if (s0 > 0) {
    const int e_old = scale_exponent(*q.scale);
    if (e_old >= e)
      e = e_old;
    else
      shift_rows<D>(q, s0, e_old - e);
  }
  const float inv = pow2f(-e);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (r >= m) break;
    const uint32_t lo = e4m3x2(x[r][0] * inv, x[r][1] * inv);
    const uint32_t w =
        V == 4 ? join16(lo, e4m3x2(x[r][V - 2] * inv, x[r][V - 1] * inv)) : lo;
    if (!q.is_v) {
      uint8_t* at = q.codes + k_tile_offset(s0 + r, q.c0, D);
      if constexpr (V == 4)
        *reinterpret_cast<uint32_t*>(at) = w;
      else
        *reinterpret_cast<uint16_t*>(at) = (uint16_t)w;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        q.codes[v_tile_offset(s0 + r, q.c0 + i)] = (uint8_t)(w >> (8 * i));
    }
  }
  __syncwarp();  // every lane has read the old scale
  if (lane == 0) *q.scale = pow2f(e);
}

// One warp: slots from pos0's of one (block, head) tile of K or V, from the
// rows of tokens t0 .., under the block rule of kv_pool_desc; values are
// rounded once, from fp32 to e4m3.  Lane l holds dimensions l * D / 32 ..
template <int D, bool PAIRS>
__device__ __forceinline__ void quant_tile(const QuantArgs& a, bool is_v, int h,
                                           int t0, int pos0, int phys, int m,
                                           int lane) {
  constexpr int V = D / 32;
  const int half = a.rot.half;
  const int64_t tile = (int64_t)phys * a.Hkv + h;
  QuantTile q;
  q.is_v = is_v;
  q.c0 = lane * V;
  q.rot = !is_v && q.c0 < 2 * half;
  q.low = q.c0 < half;
  q.codes = (is_v ? a.v8 : a.k8) + tile * 16 * D;
  q.scale = reinterpret_cast<float*>(a.scales + tile) + (is_v ? 1 : 0);
  q.stride = is_v ? a.v_token : a.k_token;
  q.src = (is_v ? a.v_new : a.k_new) + (int64_t)t0 * q.stride + (int64_t)h * D +
          q.c0;
  q.table = a.rot.table + (int64_t)pos0 * half;
  if (m == 16)
    quant_block<D, PAIRS>(q, half, lane);
  else if (m == 1)
    quant_part<D, PAIRS, 1>(q, pos0 & 15, m, half, lane);
  else
    quant_part<D, PAIRS, 16>(q, pos0 & 15, m, half, lane);
}

// CTAs [0, q_ctas) rotate queries; each later CTA takes a window of tokens,
// finds those that begin a write (a branch's first new token, or slot 0) and
// runs one warp per (write, kv-head, K or V); the CTAs of grid.y share a
// window's units.  128 threads and four CTAs an SM: a tile's 64 values and its
// table entries stay in registers.
template <int D, bool PAIRS>
__global__ void __launch_bounds__(kQuantWarps * 32, 4)
    quant_append_kernel(const __grid_constant__ QuantArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // The queries' launch depends on nothing of this one.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if ((int)blockIdx.x < a.q_ctas) {
    if (blockIdx.y > 0) return;
    const int64_t w = (int64_t)blockIdx.x * kQuantWarps + warp;
    const int64_t t = w / a.rot.split;
    if (t < a.rot.map.total)
      rotate_share<D, PAIRS>(a.rot, (int)t, (int)(w - t * a.rot.split), lane);
    return;
  }
  __shared__ int4 write[16];
  __shared__ int n_write;
  if (threadIdx.x == 0) n_write = 0;
  __syncthreads();
  const int64_t w0 = (int64_t)((int)blockIdx.x - a.q_ctas) * a.window;
  if (warp == 0 && w0 < a.rot.map.total) {
    // A lane a token: the first one's branch, and on from there.
    const TokenMap& map = a.rot.map;
    int br = map.off ? find_branch(map, (int)w0, lane) : (int)w0;
    const int64_t t = w0 + lane;
    if (lane < a.window && t < map.total) {
      while (map.off && br + 1 < map.nb && map.off[br + 1] <= t) ++br;
      const Token k = place(map, (int)t, br, blockIdx.y == 0);
      if (k.ok && (t == k.first || (k.pos & 15) == 0)) {
        int m = min(16 - (k.pos & 15), k.n - ((int)t - k.first));
        m = min(m, map.rope_len - k.pos);
        m = min(m, map.total - (int)t);
        write[atomicAdd(&n_write, 1)] = make_int4((int)t, k.pos, k.phys, m);
      }
    }
  }
  __syncthreads();
  const int units = n_write * a.Hkv * 2;
  for (int u = blockIdx.y * kQuantWarps + warp; u < units;
       u += kQuantWarps * gridDim.y) {
    const int4 w = write[u / (2 * a.Hkv)];
    const int r = u % (2 * a.Hkv);
    quant_tile<D, PAIRS>(a, r >= a.Hkv, r % a.Hkv, w.x, w.y, w.z, w.w, lane);
  }
}

// Warps a token: enough that a decode step's few tokens still fill the SMs,
// one where there are tokens enough.
int split_for(int total, int iterations) {
  int s = 1;
  while (s < iterations && (int64_t)total * s < 152 * 16) s *= 2;
  return s;
}

template <int D>
cudaError_t launch_rotate(const RotateArgs& a, bool pairs, cudaStream_t st,
                          bool beside = false) {
  const int64_t ctas = ((int64_t)a.map.total * a.split + 7) / 8;
  if (beside)  // the launch before
    return pairs ? launch_early(rotate_kernel<D, true>, (int)ctas, 256, 0, st, a)
                 : launch_early(rotate_kernel<D, false>, (int)ctas, 256, 0, st, a);
  if (pairs)
    rotate_kernel<D, true><<<(unsigned)ctas, 256, 0, st>>>(a);
  else
    rotate_kernel<D, false><<<(unsigned)ctas, 256, 0, st>>>(a);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_quant(const QuantArgs& a, bool pairs, cudaStream_t st) {
  const int64_t ctas =
      a.q_ctas + ((int64_t)a.rot.map.total + a.window - 1) / a.window;
  // A decode step has one write a window, and CTAs to spare.
  const int share = std::max(1, std::min(a.window > 1 ? 2 : 8,
                                         2 * a.Hkv / kQuantWarps));
  const dim3 grid((unsigned)ctas, (unsigned)share);
  if (pairs)
    quant_append_kernel<D, true><<<grid, kQuantWarps * 32, 0, st>>>(a);
  else
    quant_append_kernel<D, false><<<grid, kQuantWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace rope

namespace {

// Checks shared by the three entry points; fills the token map.
kv_status check_common(rope::TokenMap* m, const void* rope, int32_t rope_len,
                       int32_t rope_style, int64_t num_blocks,
                       const int32_t* tables, const int32_t* seq_lens,
                       const int32_t* off, int32_t total, int32_t nb,
                       int32_t max_blocks, int32_t block_size, void* workspace,
                       size_t ws_bytes) {
  if (!rope || !tables || !seq_lens || !workspace)
    return fail(KV_ERR_INVALID_ARG, "null argument");
  if (rope_style != KV_ROPE_HALVES && rope_style != KV_ROPE_PAIRS)
    return fail(KV_ERR_INVALID_ARG, "unknown rope_style %d", rope_style);
  if (rope_len < 1) return fail(KV_ERR_INVALID_ARG, "rope_len must be >= 1");
  if ((uintptr_t)rope & 15)
    return fail(KV_ERR_INVALID_ARG, "rope must be 16-byte aligned");
  if (block_size != 16)
    return fail(KV_ERR_INVALID_ARG, "block_size must be 16");
  if (nb < 1 || total < 0 || max_blocks < 1)
    return fail(KV_ERR_INVALID_ARG, "bad nb/total/max_blocks");
  if (total > (1 << 27))
    return fail(KV_ERR_INVALID_ARG, "total %d above 2^27 tokens", total);
  if (!off && total != nb)
    return fail(KV_ERR_INVALID_ARG, "without row_offsets total (%d) must be nb "
                                    "(%d)", total, nb);
  if (((uintptr_t)workspace & 255) || ws_bytes < kStatusBytes)
    return fail(KV_ERR_INVALID_ARG, "workspace: 256-byte aligned, >= 256 bytes");
  m->tables = tables;
  m->seq_lens = seq_lens;
  m->off = off;
  m->status = static_cast<DeviceStatus*>(workspace);
  m->num_blocks = num_blocks;
  m->nb = nb;
  m->total = total;
  m->max_blocks = max_blocks;
  m->rope_len = rope_len;
  return KV_OK;
}

bool bad_rows(const void* p, int64_t token_stride, int64_t width) {
  return ((uintptr_t)p & 15) || token_stride < width || token_stride % 8 != 0;
}

kv_status rope_append_impl(
    const void* q, int64_t q_stride, const void* k_new, int64_t k_stride,
    const void* v_new, int64_t v_stride, const float* rope, int32_t rope_len,
    int32_t rot_dim, int32_t rope_style, void* q_out, int64_t q_out_stride,
    void* k_pool, void* v_pool, void* kv_scales, int64_t num_blocks,
    const int32_t* tables, const int32_t* seq_lens, const int32_t* off,
    int32_t total, int32_t nb, int32_t max_blocks, int32_t Hq, int32_t Hkv,
    int32_t d, int32_t block_size, void* workspace, size_t ws_bytes,
    void* stream) {
  // A step without new tokens may have empty tensors, which have no address.
  if (!k_pool || !v_pool || (total != 0 && (!k_new || !v_new)))
    return fail(KV_ERR_INVALID_ARG, "null argument");
  if (total != 0 && (q == nullptr) != (q_out == nullptr))
    return fail(KV_ERR_INVALID_ARG, "q and q_out both set or both NULL");
  if (d != 64 && d != 128) return fail(KV_ERR_INVALID_ARG, "head_dim 64 or 128");
  if (Hkv < 1 || Hq < 0 || (q && Hq < 1) || Hq > 65536 || Hkv > 65536)
    return fail(KV_ERR_INVALID_ARG, "bad Hq/Hkv (%d/%d)", Hq, Hkv);
  if (rot_dim < 16 || rot_dim > d || rot_dim % 16 != 0)
    return fail(KV_ERR_INVALID_ARG, "rot_dim %d: a multiple of 16 in [16, "
                                    "head_dim]", rot_dim);
  if (num_blocks < 1 || num_blocks > (int64_t)INT32_MAX / (16 * (int64_t)Hkv))
    return fail(KV_ERR_INVALID_ARG, "num_blocks out of range");
  if (((uintptr_t)k_pool | (uintptr_t)v_pool | (uintptr_t)kv_scales) & 15)
    return fail(KV_ERR_INVALID_ARG, "pools must be 16-byte aligned");
  if (bad_rows(k_new, k_stride, (int64_t)Hkv * d) ||
      bad_rows(v_new, v_stride, (int64_t)Hkv * d) ||
      (q && (bad_rows(q, q_stride, (int64_t)Hq * d) ||
             bad_rows(q_out, q_out_stride, (int64_t)Hq * d))))
    return fail(KV_ERR_INVALID_ARG, "q, k_new, v_new, q_out: 16-byte aligned, "
                "token strides multiples of 8 and no less than a token's row");
  rope::QuantArgs a{};
  rope::RotateArgs& r = a.rot;
  if (kv_status s = check_common(&r.map, rope, rope_len, rope_style, num_blocks,
                                 tables, seq_lens, off, total, nb, max_blocks,
                                 block_size, workspace, ws_bytes))
    return s;
  if (total == 0) return KV_OK;
  const bool pairs = rope_style == KV_ROPE_PAIRS;
  const bool e4m3 = kv_scales != nullptr;
  cudaStream_t st = (cudaStream_t)stream;
  r.table = reinterpret_cast<const float2*>(rope);
  r.half = rot_dim / 2;
  const int per_warp = 256 / d;
  if (q)
    r.rows[0] = {static_cast<const __nv_bfloat16*>(q),
                 static_cast<__nv_bfloat16*>(q_out), q_stride, d, q_out_stride,
                 0, 0, d, Hq, 1};
  int its = q ? (Hq + per_warp - 1) / per_warp : 0;
  cudaError_t e;
  if (!e4m3) {
    const int64_t blk = (int64_t)Hkv * 16 * d;
    r.rows[1] = {static_cast<const __nv_bfloat16*>(k_new),
                 static_cast<__nv_bfloat16*>(k_pool), k_stride, d, 0, blk, d,
                 16 * d, Hkv, 1};
    r.rows[2] = {static_cast<const __nv_bfloat16*>(v_new),
                 static_cast<__nv_bfloat16*>(v_pool), v_stride, d, 0, blk, d,
                 16 * d, Hkv, 0};
    its += 2 * ((Hkv + per_warp - 1) / per_warp);
    r.split = rope::split_for(total, its);
    e = d == 128 ? rope::launch_rotate<128>(r, pairs, st)
                 : rope::launch_rotate<64>(r, pairs, st);
  } else {
    r.split = rope::split_for(total, std::max(its, 1));
    // A decode step's tokens each begin a write: one CTA a token, and the
    // queries in the same launch.  In a chunk about every sixteenth does; the
    // queries are most of the bytes then and take a launch of their own, which
    // keeps twice the warps on an SM and may start before the other has ended (24
    // chunks of 37 to 701 tokens: 73 us in one launch, 58 us one after the other,
    // 50.5 so).  The two take 30.0 and 27.6 us alone, so they overlap by 7 us only:
    // four CTAs of 128 threads at 128 registers are an SM's whole register file, and
    // the queries' CTAs find room when the last of those leave.
    a.window = off ? 16 : 1;
    const bool own_launch = off != nullptr && q != nullptr;
    a.q_ctas = q && !own_launch
                   ? (int)(((int64_t)total * r.split + rope::kQuantWarps - 1) /
                           rope::kQuantWarps)
                   : 0;
    a.k_new = static_cast<const __nv_bfloat16*>(k_new);
    a.v_new = static_cast<const __nv_bfloat16*>(v_new);
    a.k_token = k_stride;
    a.v_token = v_stride;
    a.k8 = static_cast<uint8_t*>(k_pool);
    a.v8 = static_cast<uint8_t*>(v_pool);
    a.scales = static_cast<float4*>(kv_scales);
    a.Hkv = Hkv;
    e = d == 128 ? rope::launch_quant<128>(a, pairs, st)
                 : rope::launch_quant<64>(a, pairs, st);
    if (e == cudaSuccess && own_launch)
      e = d == 128 ? rope::launch_rotate<128>(r, pairs, st, true)
                   : rope::launch_rotate<64>(r, pairs, st, true);
  }
  if (e != cudaSuccess)
    return fail(KV_ERR_CUDA, "rope append launch: %s", cudaGetErrorString(e));
  return KV_OK;
}

}  // namespace
}  // namespace pkv

using pkv::fail;

extern "C" kv_status paged_rope_append(
    const void* q, int64_t q_stride, const void* k_new, int64_t k_stride,
    const void* v_new, int64_t v_stride, const float* rope, int32_t rope_len,
    int32_t rot_dim, int32_t rope_style, void* q_out, int64_t q_out_stride,
    void* k_pool, void* v_pool, int64_t num_blocks,
    const int32_t* block_tables, const int32_t* seq_lens,
    const int32_t* row_offsets, int32_t total, int32_t nb, int32_t max_blocks,
    int32_t Hq, int32_t Hkv, int32_t d, int32_t block_size, void* workspace,
    size_t ws_bytes, void* stream) {
  pkv::clear_error();
  return pkv::rope_append_impl(
      q, q_stride, k_new, k_stride, v_new, v_stride, rope, rope_len, rot_dim,
      rope_style, q_out, q_out_stride, k_pool, v_pool, nullptr, num_blocks,
      block_tables, seq_lens, row_offsets, total, nb, max_blocks, Hq, Hkv, d,
      block_size, workspace, ws_bytes, stream);
}

extern "C" kv_status paged_rope_append_e4m3(
    const void* q, int64_t q_stride, const void* k_new, int64_t k_stride,
    const void* v_new, int64_t v_stride, const float* rope, int32_t rope_len,
    int32_t rot_dim, int32_t rope_style, void* q_out, int64_t q_out_stride,
    void* k_pool, void* v_pool, void* kv_scales, int64_t num_blocks,
    const int32_t* block_tables, const int32_t* seq_lens,
    const int32_t* row_offsets, int32_t total, int32_t nb, int32_t max_blocks,
    int32_t Hq, int32_t Hkv, int32_t d, int32_t block_size, void* workspace,
    size_t ws_bytes, void* stream) {
  pkv::clear_error();
  if (!kv_scales) return fail(KV_ERR_INVALID_ARG, "kv_scales required");
  return pkv::rope_append_impl(
      q, q_stride, k_new, k_stride, v_new, v_stride, rope, rope_len, rot_dim,
      rope_style, q_out, q_out_stride, k_pool, v_pool, kv_scales, num_blocks,
      block_tables, seq_lens, row_offsets, total, nb, max_blocks, Hq, Hkv, d,
      block_size, workspace, ws_bytes, stream);
}

extern "C" kv_status paged_latent_append(
    const void* c_new, int64_t c_stride, const void* r_new, int64_t r_stride,
    const void* q_rope, int64_t q_stride, int64_t q_head_stride,
    const float* rope, int32_t rope_len, int32_t rope_style, void* q_rope_out,
    int64_t q_out_stride, int64_t q_out_head_stride, void* c_pool,
    void* r_pool, int64_t num_blocks, const int32_t* block_tables,
    const int32_t* seq_lens, const int32_t* row_offsets, int32_t total,
    int32_t nb, int32_t max_blocks, int32_t Hq, int32_t rank, int32_t rope_dim,
    int32_t block_size, void* workspace, size_t ws_bytes, void* stream) {
  pkv::clear_error();
  namespace rp = pkv::rope;
  // A step without new tokens may have empty tensors, which have no address.
  if (!c_pool || !r_pool || (total != 0 && (!c_new || !r_new)))
    return fail(KV_ERR_INVALID_ARG, "null argument");
  if (total != 0 && (q_rope == nullptr) != (q_rope_out == nullptr))
    return fail(KV_ERR_INVALID_ARG, "q_rope and q_rope_out both set or both NULL");
  if (rank != KV_LATENT_RANK || rope_dim != KV_LATENT_ROPE)
    return fail(KV_ERR_INVALID_ARG, "a latent cache has rank 512 and rope_dim "
                                    "64, got %d and %d", rank, rope_dim);
  if (Hq < 0 || (q_rope && Hq < 1) || Hq > 65536)
    return fail(KV_ERR_INVALID_ARG, "bad Hq %d", Hq);
  if (num_blocks < 1 || num_blocks > (int64_t)INT32_MAX / 16)
    return fail(KV_ERR_INVALID_ARG, "num_blocks out of range");
  if (((uintptr_t)c_pool | (uintptr_t)r_pool) & 15)
    return fail(KV_ERR_INVALID_ARG, "pools must be 16-byte aligned");
  // A head's 64 values are one row; rows of one token do not overlap.
  const int64_t q_min = (Hq > 0 ? (Hq - 1) * q_head_stride : 0) + rope_dim;
  const int64_t qo_min = (Hq > 0 ? (Hq - 1) * q_out_head_stride : 0) + rope_dim;
  if (pkv::bad_rows(c_new, c_stride, rank) ||
      pkv::bad_rows(r_new, r_stride, rope_dim) ||
      (q_rope && (q_head_stride < rope_dim || q_head_stride % 8 != 0 ||
                  q_out_head_stride < rope_dim || q_out_head_stride % 8 != 0 ||
                  pkv::bad_rows(q_rope, q_stride, q_min) ||
                  pkv::bad_rows(q_rope_out, q_out_stride, qo_min))))
    return fail(KV_ERR_INVALID_ARG, "c_new, r_new, q_rope, q_rope_out: 16-byte "
                "aligned, strides multiples of 8 and no less than a row");
  rp::RotateArgs a{};
  if (kv_status s = pkv::check_common(&a.map, rope, rope_len, rope_style,
                                      num_blocks, block_tables, seq_lens,
                                      row_offsets, total, nb, max_blocks,
                                      block_size, workspace, ws_bytes))
    return s;
  if (total == 0) return KV_OK;
  a.table = reinterpret_cast<const float2*>(rope);
  a.half = rope_dim / 2;
  if (q_rope)
    a.rows[0] = {static_cast<const __nv_bfloat16*>(q_rope),
                 static_cast<__nv_bfloat16*>(q_rope_out), q_stride,
                 q_head_stride, q_out_stride, 0, 0, q_out_head_stride, Hq, 1};
  a.rows[1] = {static_cast<const __nv_bfloat16*>(r_new),
               static_cast<__nv_bfloat16*>(r_pool), r_stride, 0, 0,
               16 * rope_dim, rope_dim, 0, 1, 1};
  // The latent as eight rows of 64 values.
  a.rows[2] = {static_cast<const __nv_bfloat16*>(c_new),
               static_cast<__nv_bfloat16*>(c_pool), c_stride, 64, 0, 16 * rank,
               rank, 64, rank / 64, 0};
  a.split = rp::split_for(total, (q_rope ? (Hq + 3) / 4 : 0) + 3);
  const cudaError_t e = rp::launch_rotate<64>(
      a, rope_style == KV_ROPE_PAIRS, (cudaStream_t)stream);
  if (e != cudaSuccess)
    return fail(KV_ERR_CUDA, "latent append launch: %s", cudaGetErrorString(e));
  return KV_OK;
}
