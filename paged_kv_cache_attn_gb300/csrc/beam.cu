// Beam selection (kv_beam_select): of every group of beams the n continuations
// (beam, token) with the highest
//   y = score[beam] + x[token] - log sum_t exp x[t],
// ties to the lower beam, then the lower token.  Bound by the logits' bytes: they are
// read once.
//
// First kernel: a CTA has a piece of one beam's logits in registers.  Its maximum and
// its sum of exponentials go out, and its n highest logits (of one beam the order of
// y is that of x): the n-th highest of the threads' maxima bounds them from below, is
// found to within a few by bisection over counts, and leaves a few candidates, which
// are ranked against each other.  Second kernel: a CTA per group joins the sums in
// 64 bits and picks the n highest y of the pieces' candidates the same way.
//
// y is computed in 64 bits from fp32 sums of exponentials (a thread's 8 or 32 of
// them; across threads and pieces in 64 bits), about 1e-7 from exact, so that beams
// are hardly ever ordered otherwise than exactly.

#include <algorithm>
#include <cmath>

#include "device_common.cuh"
#include "tensor_map.h"

namespace pkv {
namespace beam {

constexpr int kThreads = 256;
constexpr int kMaxOut = 128;
constexpr int kMaxBeams = 1024;
constexpr int kCand = 1024;  // candidates in shared memory; more: one at a time

struct Stat {
  double sum;  // of exponentials of logits less `top`
  float top, pad;
};

struct Params {
  const void* logits;
  const float* scores;   // [rows]
  Stat* stats;           // [rows][pieces]
  uint2* entries;        // [rows][pieces][n]: ordered logit (0: none), token
  float* out_scores;     // [groups][n]
  int32_t* out_parents;
  int32_t* out_tokens;
  int64_t stride;        // values between rows
  int vocab, pieces, n, beams;
};

// Floats as unsigned numbers of the same order; -inf is 0x007fffff.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 is 0
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

__device__ __forceinline__ uint64_t ordered(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x + 0.);
  return u ^ ((uint64_t)((int64_t)u >> 63) | 0x8000000000000000ull);
}

constexpr uint32_t kNone32 = 0x007fffffu;  // ordered(-inf): no candidate
constexpr uint64_t kNone64 = 0x000fffffffffffffull;

// A value that at least n threads' `mine` reach, and not many more; `floor` (the
// least a candidate has) where fewer do.  All threads call it; `lo` and `hi`: the
// least and largest of `mine`.
template <typename Key>
__device__ __forceinline__ Key threshold(Key mine, Key lo, Key hi, Key floor, int n) {
  if (__syncthreads_count(mine >= floor) < n) return floor;
  lo = lo < floor ? floor : lo;
  while (hi - lo > 1) {
    const Key mid = lo + (hi - lo) / 2;
    const int c = __syncthreads_count(mine >= mid);
    if (c >= n) {
      lo = mid;
      if (c <= n + n / 2 + 4) break;
    } else {
      hi = mid;
    }
  }
  return lo;
}

// Least and largest over the CTA.
template <typename Key>
__device__ __forceinline__ void range(Key mine, Key* sh, Key& lo, Key& hi) {
  lo = hi = mine;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) {
    sh[threadIdx.x >> 5] = lo;
    sh[32 + (threadIdx.x >> 5)] = hi;
  }
  __syncthreads();
  for (int w = 0; w < warps; ++w) {
    lo = min(lo, sh[w]);
    hi = max(hi, sh[32 + w]);
  }
}

template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float(float x) { return x; }
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 x) {
  return __bfloat162float(x);
}

// E: logits of a thread.
template <typename T, int E>
__global__ void __launch_bounds__(kThreads) piece_kernel(const Params p) {
  constexpr int VE = 16 / sizeof(T), NV = E / VE;
  __shared__ uint64_t cand[kCand];
  __shared__ uint32_t sh[64];
  __shared__ double sums[kThreads / 32];
  __shared__ int count;
  __shared__ unsigned long long top;
  const int row = blockIdx.y, piece = blockIdx.x, tid = threadIdx.x;
  if (!(p.scores[row] > -INFINITY)) return;  // no beam
  const T* x = static_cast<const T*>(p.logits) + (int64_t)row * p.stride;
  // Vectors start on 16-byte borders, the first at or before the row's start.
  const int off = (int)((uintptr_t)x % 16 / sizeof(T));
  const int64_t v0 = (int64_t)piece * (kThreads * NV) + tid;
  float f[NV][VE];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t e = (v0 + (int64_t)i * kThreads) * VE - off;
    if (e >= 0 && e + VE <= p.vocab) {
      const uint4 raw = __ldcs(reinterpret_cast<const uint4*>(x + e));
      const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
      for (int k = 0; k < VE; ++k) {
        if (sizeof(T) == 4)
          f[i][k] = __uint_as_float(w[k % 4]);
        else
          f[i][k] = __uint_as_float(k & 1 ? w[k / 2] & 0xffff0000u : w[k / 2] << 16);
      }
    } else {
#pragma unroll
      for (int k = 0; k < VE; ++k)
        f[i][k] = e + k >= 0 && e + k < p.vocab ? to_float(x[e + k]) : -INFINITY;
    }
  }
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < VE; ++k) {
      f[i][k] = fmaxf(f[i][k], -INFINITY);  // NaN counts as -inf
      m = fmaxf(m, f[i][k]);
    }
  const uint32_t mine = ordered(m);
  uint32_t lo, hi;
  range(mine, sh, lo, hi);
  const float top_x = unordered(hi);
  float s = 0.f;
  if (top_x > -INFINITY) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < VE; ++k) s += ex2((f[i][k] - top_x) * 1.4426950408889634f);
  }
  double sum = s;
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((tid & 31) == 0) sums[tid >> 5] = sum;
  if (tid == 0) count = 0;
  const int n = p.n;
  const uint32_t bar = threshold(mine, lo, hi, kNone32 + 1, n);
  const int64_t slot = (int64_t)row * p.pieces + piece;
  if (tid == 0) {
    double all = 0;
    for (int w = 0; w < kThreads / 32; ++w) all += sums[w];
    p.stats[slot] = Stat{all, top_x, 0.f};
  }
  auto token = [&](int i, int k) {
    return (uint32_t)((v0 + (int64_t)i * kThreads) * VE - off + k);
  };
  // Higher logits first, then lower tokens.
  auto key = [&](int i, int k) {
    return (uint64_t)ordered(f[i][k]) << 32 | (0xffffffffu - token(i, k));
  };
  if (mine >= bar) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < VE; ++k)
        if (ordered(f[i][k]) >= bar) {
          const int at = atomicAdd(&count, 1);
          if (at < kCand) cand[at] = key(i, k);
        }
  }
  __syncthreads();
  const int c = count;
  uint2* out = p.entries + slot * n;
  if (c <= kCand) {
    for (int i = tid; i < c; i += kThreads) {
      const uint64_t a = cand[i];
      int rank = 0;
      for (int j = 0; j < c; ++j) rank += cand[j] > a;
      if (rank < n) out[rank] = make_uint2((uint32_t)(a >> 32), ~(uint32_t)a);
    }
    for (int i = c + tid; i < n; i += kThreads) out[i] = make_uint2(0, 0);
    return;
  }
  // Many equal logits: one at a time (c > n of them).
  uint64_t last = ~0ull;
  for (int r = 0; r < n; ++r) {
    uint64_t best = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < VE; ++k) {
        const uint64_t a = key(i, k);
        if (a < last && a > best) best = a;
      }
    if (tid == 0) top = 0;
    __syncthreads();
#pragma unroll
    for (int o = 16; o; o >>= 1)
      best = max(best, (uint64_t)__shfl_xor_sync(0xffffffffu, best, o));
    if ((tid & 31) == 0) atomicMax(&top, (unsigned long long)best);
    __syncthreads();
    last = top;
    if (tid == 0) out[r] = make_uint2((uint32_t)(last >> 32), ~(uint32_t)last);
    __syncthreads();
  }
}

struct Cand {
  uint64_t y;    // ordered
  int64_t flat;  // beam x vocab + token
};

__device__ __forceinline__ bool before(const Cand& a, const Cand& b) {
  return a.y > b.y || (a.y == b.y && a.flat < b.flat);
}

__global__ void __launch_bounds__(kThreads) group_kernel(const Params p) {
  __shared__ Cand cand[kCand];
  // log sum exp(x - top), NaN: no continuations.  Kept apart from the highest logit,
  // so that logits of any size cancel before the score is added.
  __shared__ double log_sum[kMaxBeams];
  __shared__ float top[kMaxBeams];
  __shared__ uint64_t sh[64];
  __shared__ Cand best_of[kThreads / 32];
  __shared__ int count;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int group = blockIdx.x, tid = threadIdx.x, lane = tid & 31, n = p.n;
  for (int b = tid >> 5; b < p.beams; b += kThreads / 32) {
    const int64_t row = (int64_t)group * p.beams + b;
    const float score = p.scores[row];
    double out = NAN;
    if (score > -INFINITY) {
      const Stat* st = p.stats + row * p.pieces;
      float m = -INFINITY;
      for (int i = lane; i < p.pieces; i += 32) m = fmaxf(m, st[i].top);
#pragma unroll
      for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      double s = 0;
      if (m > -INFINITY && m < INFINITY)
        for (int i = lane; i < p.pieces; i += 32)
          if (st[i].top > -INFINITY) s += st[i].sum * exp((double)st[i].top - m);
#pragma unroll
      for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (s > 0) out = log(s);
      if (lane == 0) top[b] = m;
    }
    if (lane == 0) log_sum[b] = out;
  }
  if (tid == 0) count = 0;
  __syncthreads();
  const int per = p.pieces * n, total = p.beams * per;
  const uint2* entries = p.entries + (int64_t)group * total;
  const float* scores = p.scores + (int64_t)group * p.beams;
  auto get = [&](int i) {
    const int b = i / per;
    const double l = log_sum[b];
    if (isnan(l)) return Cand{0, 0};
    const uint2 e = entries[i];
    if (e.x == 0) return Cand{0, 0};
    const double y = (double)scores[b] + (((double)unordered(e.x) - top[b]) - l);
    if (!(y > -INFINITY)) return Cand{0, 0};
    return Cand{ordered(y), (int64_t)b * p.vocab + e.y};
  };
  uint64_t mine = 0, lo, hi;
  for (int i = tid; i < total; i += kThreads) mine = max(mine, get(i).y);
  range(mine, sh, lo, hi);
  const uint64_t bar = threshold(mine, lo, hi, kNone64 + 1, n);
  if (mine >= bar)
    for (int i = tid; i < total; i += kThreads) {
      const Cand a = get(i);
      if (a.y >= bar) {
        const int at = atomicAdd(&count, 1);
        if (at < kCand) cand[at] = a;
      }
    }
  __syncthreads();
  const int c = count;
  auto put = [&](int rank, const Cand& a) {
    const int64_t at = (int64_t)group * n + rank;
    const uint64_t u = a.y & 0x8000000000000000ull ? a.y ^ 0x8000000000000000ull : ~a.y;
    p.out_scores[at] = (float)__longlong_as_double((long long)u);
    p.out_parents[at] = (int32_t)(a.flat / p.vocab);
    p.out_tokens[at] = (int32_t)(a.flat % p.vocab);
  };
  for (int i = c + tid; i < n; i += kThreads) {
    const int64_t at = (int64_t)group * n + i;
    p.out_scores[at] = -INFINITY;
    p.out_parents[at] = p.out_tokens[at] = -1;
  }
  if (c <= kCand) {
    for (int i = tid; i < c; i += kThreads) {
      const Cand a = cand[i];
      int rank = 0;
      for (int j = 0; j < c; ++j) rank += before(cand[j], a);
      if (rank < n) put(rank, a);
    }
    return;
  }
  // Many equal sums: one at a time (c > n of them).
  Cand last{~0ull, -1};
  for (int r = 0; r < n; ++r) {
    Cand best{0, 0};
    for (int i = tid; i < total; i += kThreads) {
      const Cand a = get(i);
      if (a.y && before(last, a) && before(a, best)) best = a;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const Cand a{__shfl_xor_sync(0xffffffffu, best.y, o),
                   __shfl_xor_sync(0xffffffffu, best.flat, o)};
      if (before(a, best)) best = a;
    }
    if (lane == 0) best_of[tid >> 5] = best;
    __syncthreads();
    for (int w = 0; w < kThreads / 32; ++w)
      if (before(best_of[w], best)) best = best_of[w];
    last = best;
    if (tid == 0) put(r, best);
    __syncthreads();
  }
}

// Logits of a piece: 8192, or 2048 where those would be fewer than two waves of
// pieces (three CTAs of them an SM).
int piece_size(int64_t rows, int vocab) {
  return rows * ((vocab + 8191) / 8192) < 2 * 3 * 152 ? 2048 : 8192;
}

// Pieces of a row, with vectors that start up to 7 values before it.
int64_t n_pieces(int64_t rows, int vocab) {
  const int size = piece_size(rows, vocab);
  return ((int64_t)vocab + 7 + size - 1) / size;
}

kv_status sizes_ok(int32_t n_groups, int32_t beams, int32_t vocab, int32_t n_out) {
  if (n_groups < 1 || beams < 1 || beams > kMaxBeams || vocab < 1)
    return fail(KV_ERR_INVALID_ARG, "bad n_groups/beams/vocab (%d/%d/%d)", n_groups,
                beams, vocab);
  if (n_out < 1 || n_out > kMaxOut)
    return fail(KV_ERR_INVALID_ARG, "n_out %d outside [1, %d]", n_out, kMaxOut);
  const int64_t rows = (int64_t)n_groups * beams;
  if (rows > 65535) return fail(KV_ERR_INVALID_ARG, "more than 65535 beams");
  if (n_pieces(rows, vocab) * beams * n_out > INT32_MAX / 2)
    return fail(KV_ERR_INVALID_ARG, "vocabulary too large");
  return KV_OK;
}

size_t entries_offset(int64_t rows, int64_t pieces) {
  return align_up((size_t)rows * pieces * sizeof(Stat), 256);
}

size_t workspace(int64_t rows, int32_t vocab, int32_t n) {
  const int64_t pieces = n_pieces(rows, vocab);
  return align_up(entries_offset(rows, pieces) + (size_t)rows * pieces * n * 8, 256);
}

}  // namespace beam
}  // namespace pkv

using pkv::fail;

extern "C" kv_status kv_beam_select_workspace_size(int32_t n_groups, int32_t beams,
                                                   int32_t vocab, int32_t n_out,
                                                   size_t* out_bytes) {
  pkv::clear_error();
  if (!out_bytes) return fail(KV_ERR_INVALID_ARG, "null argument");
  if (kv_status s = pkv::beam::sizes_ok(n_groups, beams, vocab, n_out)) return s;
  *out_bytes = pkv::beam::workspace((int64_t)n_groups * beams, vocab, n_out);
  return KV_OK;
}

extern "C" kv_status kv_beam_select(const void* logits, int32_t logits_type,
                                    int64_t row_stride, const float* scores,
                                    int32_t n_groups, int32_t beams, int32_t vocab,
                                    int32_t n_out, float* out_scores,
                                    int32_t* out_parents, int32_t* out_tokens,
                                    void* workspace, size_t ws_bytes, void* stream) {
  namespace W = pkv::beam;
  pkv::clear_error();
  if (!logits || !scores || !out_scores || !out_parents || !out_tokens || !workspace)
    return fail(KV_ERR_INVALID_ARG, "null argument");
  if (kv_status s = W::sizes_ok(n_groups, beams, vocab, n_out)) return s;
  if (logits_type != KV_LOGITS_BF16 && logits_type != KV_LOGITS_F32)
    return fail(KV_ERR_INVALID_ARG, "bad logits_type %d", logits_type);
  const bool f32 = logits_type == KV_LOGITS_F32;
  if (row_stride < vocab || row_stride > ((int64_t)1 << 40))
    return fail(KV_ERR_INVALID_ARG, "row_stride must be no less than vocab");
  if ((uintptr_t)logits % (f32 ? 4 : 2) ||
      ((uintptr_t)scores | (uintptr_t)out_scores | (uintptr_t)out_parents |
       (uintptr_t)out_tokens) & 3)
    return fail(KV_ERR_INVALID_ARG, "arrays must be aligned to their values");
  const int64_t rows = (int64_t)n_groups * beams;
  const size_t need = W::workspace(rows, vocab, n_out);
  if ((uintptr_t)workspace & 255 || ws_bytes < need)
    return fail(KV_ERR_INVALID_ARG, "workspace: 256-byte aligned, %zu bytes < %zu "
                "needed", ws_bytes, need);
  W::Params p;
  p.logits = logits;
  p.scores = scores;
  p.pieces = (int)W::n_pieces(rows, vocab);
  p.stats = static_cast<W::Stat*>(workspace);
  p.entries = reinterpret_cast<uint2*>(static_cast<uint8_t*>(workspace) +
                                       W::entries_offset(rows, p.pieces));
  p.out_scores = out_scores;
  p.out_parents = out_parents;
  p.out_tokens = out_tokens;
  p.stride = row_stride;
  p.vocab = vocab;
  p.n = n_out;
  p.beams = beams;
  cudaStream_t st = (cudaStream_t)stream;
  const dim3 grid((unsigned)p.pieces, (unsigned)rows);
  const bool big = W::piece_size(rows, vocab) == 8192;
  if (f32 && big)
    W::piece_kernel<float, 32><<<grid, W::kThreads, 0, st>>>(p);
  else if (f32)
    W::piece_kernel<float, 8><<<grid, W::kThreads, 0, st>>>(p);
  else if (big)
    W::piece_kernel<__nv_bfloat16, 32><<<grid, W::kThreads, 0, st>>>(p);
  else
    W::piece_kernel<__nv_bfloat16, 8><<<grid, W::kThreads, 0, st>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess)
    e = pkv::launch_early(W::group_kernel, n_groups, W::kThreads, 0, st, p);
  if (e != cudaSuccess)
    return fail(KV_ERR_CUDA, "beam selection: %s", cudaGetErrorString(e));
  return KV_OK;
}
