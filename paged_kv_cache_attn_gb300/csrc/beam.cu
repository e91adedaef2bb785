// Beam selection (kv_beam_select): of every group of beams the n continuations
// (beam, token) with the highest
//   y = score[beam] + x[token] - log sum_t exp x[t],
// ties to the lower beam, then the lower token.  Bound by the logits' bytes: they are
// read once.
//
// First kernel: a CTA streams a piece of one beam's logits through shared memory, a step
// of up to 4096 at a time; each thread adds up its exponentials and keeps the largest
// logits of its steps, and waits for no other thread.  Of one beam the order of y is
// that of x: at the end a value that n threads' largest logits reach (and not many
// more, by bisection over counts) is a bar for the n highest, and the few groups of
// logits whose largest reaches it are read again.  (With candidates kept as they came,
// a barrier a step and a bar raised on the way, 32 x 16 beams of 128256 took 88 us, 21
// instructions a logit; this takes 58 us, 4.5 TB/s.  Of the 53 us of the first kernel
// some 6 are its ends: sums joined, the bar, groups read again from memory.)  Second
// kernel: a CTA per group joins the sums and picks the n highest y of the pieces'
// candidates.  1 x 8 beams of 32000 take 11 us, two launches of dependent steps.
//
// The sums are at most 16 exponentials in fp32, added up with what each addition rounds
// off; y is computed in 64 bits, about 1e-7 from exact, so that beams are hardly ever
// ordered otherwise than exactly.  References of the sums are whole numbers: what lies
// between two of them is, too, and its exponential comes from a table.

#include <algorithm>
#include <cfloat>
#include <cmath>

#include "prefill.cuh"
#include "tensor_map.h"

namespace pkv {
namespace beam {

constexpr int kThreads = 256;
constexpr int kMaxOut = 128;
constexpr int kMaxBeams = 1024;
constexpr int kRound = 4 * 152;                   // CTAs of the first kernel at once
constexpr int kCand = 768;   // candidates in shared memory; more: by their digits
constexpr int kGroups = 16;  // groups of a thread's steps whose largest logits are kept
constexpr int kList = 1024;  // groups to be read again, at most
constexpr float kHeadroom = 40.f;  // of logits above the reference of a sum

// Steps on their way to a CTA: 32 KB.
template <typename T>
constexpr int kRingSteps = sizeof(T) == 4 ? 2 : 4;

// (Below the 48 KB that need no opting in; the candidates fit in.)
template <typename T, int E>
constexpr int kRingBytes = std::max((2 * kCand + kMaxOut) * 8 + kList * 2,
                                    kRingSteps<T> * kThreads * E * (int)sizeof(T));

struct Stat {
  float sum, rest;  // of exponentials of logits less `top`, and what its rounding left
  float top, pad;   // a whole number
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
  int vocab, pieces, n, beams, heads;
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

// A value that at least n threads' `mine` reach, and not many more; `floor` (the
// least a candidate has) where fewer do.  All threads call it; `lo` and `hi`: the
// least and largest of `mine`.
__device__ __forceinline__ uint32_t threshold(uint32_t mine, uint32_t lo, uint32_t hi,
                                              uint32_t floor, int n) {
  if (__syncthreads_count(mine >= floor) < n) return floor;
  lo = lo < floor ? floor : lo;
  while (hi - lo > 1) {
    const uint32_t mid = lo + (hi - lo) / 2;
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

// Least and largest over the CTA's 256 threads.
__device__ __forceinline__ void range(uint32_t mine, uint32_t* sh, uint32_t& lo,
                                      uint32_t& hi) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  lo = __reduce_min_sync(0xffffffffu, mine);
  hi = __reduce_max_sync(0xffffffffu, mine);
  if (lane == 0) {
    sh[warp] = lo;
    sh[kThreads / 32 + warp] = hi;
  }
  __syncthreads();
  lo = __reduce_min_sync(0xffffffffu, sh[lane % (kThreads / 32)]);
  hi = __reduce_max_sync(0xffffffffu, sh[kThreads / 32 + lane % (kThreads / 32)]);
}

struct Digits {
  uint32_t hist[256];
  uint64_t prefix;
  int want;
};

// The n-th highest of the keys that `each` calls its argument with (whether there is
// one, the key; whole warps), by digits of 8 bits from bit `top` down, of the keys that
// begin with `prefix` (under `mask`): the least key of the n highest, or its first
// digits where all keys that begin so are among them (n: 0 then, else which of the
// keys equal to the result is the last).  All threads call it; 0 where there are fewer.
template <typename Each>
__device__ __forceinline__ uint64_t nth_key(Each each, int top, uint64_t prefix,
                                            uint64_t mask, int& n, Digits& sh) {
  const int tid = threadIdx.x;
  for (int d = top; d >= 0; d -= 8) {
    __syncthreads();
    sh.hist[tid] = 0;
    if (tid == 0) sh.want = -1;
    __syncthreads();
    each([&](bool in, uint64_t a) {
      const int digit = in && (a & mask) == prefix ? (int)(a >> d & 255) : -1;
      const uint32_t peers = __match_any_sync(0xffffffffu, digit);
      if (digit >= 0 && (tid & 31) == __ffs(peers) - 1)
        atomicAdd(&sh.hist[digit], __popc(peers));
    });
    __syncthreads();
    int above = 0;
    for (int k = tid + 1; k < 256; ++k) above += sh.hist[k];
    const int here = sh.hist[tid];
    if (above < n && above + here >= n) {
      sh.prefix = prefix | (uint64_t)tid << d;
      sh.want = above + here == n ? 0 : n - above;
    }
    __syncthreads();
    if (sh.want < 0) return 0;
    prefix = sh.prefix;
    n = sh.want;
    mask |= 255ull << d;
    if (n == 0) break;
  }
  return prefix;
}

template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float(float x) { return x; }
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 x) {
  return __bfloat162float(x);
}

// The n highest of c <= kCand keys to best, in order (0 where there are fewer).  Of
// many, a bar that n of the threads' highest keys reach leaves few to be ranked.
// `floor`: a logit that all of them reach.
__device__ __forceinline__ void pick_best(const uint64_t* cand, int c, int n, float floor,
                                          uint64_t* few, uint64_t* best, uint32_t* sh,
                                          int* count) {
  const int tid = threadIdx.x;
  const uint64_t* from = cand;
  int k = c;
  if (c > kThreads) {
    uint64_t own[kCand / kThreads], top = 0;
#pragma unroll
    for (int i = 0; i < kCand / kThreads; ++i) {
      const int at = tid + i * kThreads;
      own[i] = at < c ? cand[at] : 0;
      top = max(top, own[i]);
    }
    const uint32_t mine = (uint32_t)(top >> 32);
    uint32_t lo, hi;
    range(mine, sh, lo, hi);
    const uint32_t bar =
        threshold(mine, lo, hi, max(ordered(floor), kNone32 + 1), n);
    if (tid == 0) *count = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kCand / kThreads; ++i)
      if ((uint32_t)(own[i] >> 32) >= bar) few[atomicAdd(count, 1)] = own[i];
    __syncthreads();
    from = few;
    k = *count;
  }
  for (int i = tid; i < n; i += kThreads) best[i] = 0;
  __syncthreads();
  // Eight threads a key.
  for (int i0 = 0; i0 < k; i0 += kThreads / 8) {
    const int i = i0 + (tid >> 3);
    const uint64_t a = i < k ? from[i] : 0;
    int rank = 0;
    for (int j = tid & 7; j < k; j += 8) rank += from[j] > a;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
    if (i < k && rank < n && (tid & 7) == 0) best[rank] = a;
  }
  __syncthreads();
}

// e^x in 64 bits for x <= 0: x / ln 2 split into a whole number and at most half of one
// either way, its Taylor series to the 11th power (2e-14 relative).  64-bit operations
// take about 110 cycles each here: where a call waits for them they are few, and
// tables, made while nothing else can be done, stand for this and the logarithm.
__device__ __forceinline__ double exp_of(double x) {
  x = fmax(x, -700.);
  const double k = rint(x * 1.4426950408889634);
  const double r = fma(k, -0.6931471805599453, x);
  double y = 1. / 39916800.;
#pragma unroll
  for (int i = 10; i >= 0; --i) {
    constexpr double inv[11] = {1., 1., 1. / 2, 1. / 6, 1. / 24, 1. / 120, 1. / 720,
                                1. / 5040, 1. / 40320, 1. / 362880, 1. / 3628800};
    y = fma(y, r, inv[i]);
  }
  return y * __longlong_as_double((long long)((int)k + 1023) << 52);
}

// log s in 64 bits, from the 32-bit one by a Newton step (and the next term):
// log s = y + log(s e^-y).  s >= 1e-30.
__device__ __forceinline__ double log_of(double s) {
  // s = f 2^k, so that the exponential's argument is small.
  const long long bits = __double_as_longlong(s);
  const int k = (int)(bits >> 52) - 1023;
  const double f = __longlong_as_double((bits & 0xfffffffffffffll) | 1023ll << 52);
  const float y = logf((float)f);  // in [0, ln 2]
  const double d = fma(f, exp_of(-(double)y), -1.);
  return fma((double)k, 0.6931471805599453, (double)y + fma(-.5 * d, d, d));
}

// E: logits of a thread in a step.
template <typename T, int E>
__global__ void __launch_bounds__(kThreads, 4) piece_kernel(const Params p) {
  constexpr int VE = 16 / sizeof(T), NV = E / VE;
  constexpr int kDepth = kRingSteps<T>;
  __shared__ uint32_t sh[64];
  __shared__ Digits digits;
  __shared__ float2 sums[kThreads / 32];
  __shared__ uint16_t group_max[kGroups][kThreads];
  __shared__ int count, few_count, listed;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int row = blockIdx.y, piece = blockIdx.x, tid = threadIdx.x, n = p.n;
  if (!(p.scores[row] > -INFINITY)) return;  // no beam
  const T* x = static_cast<const T*>(p.logits) + (int64_t)row * p.stride;
  // Vectors start on 16-byte borders, the first at or before the row's start.
  const int off = (int)((uintptr_t)x % 16 / sizeof(T));
  const int64_t vectors = ((int64_t)p.vocab + off + VE - 1) / VE;
  const int64_t v_begin = vectors * piece / p.pieces;
  const int64_t v_end = vectors * (piece + 1) / p.pieces;
  constexpr int kStep = kThreads * NV;
  const int steps = (int)((v_end - v_begin + kStep - 1) / kStep);
  // Each thread's vectors of the next steps are on their way to its own places in
  // shared memory (32 KB a CTA, 128 KB an SM: with one step in registers the loads'
  // latency, 1.9 us under load, kept an SM at 29 GB/s), so that nothing of the stream
  // waits for another thread.  Vectors that reach over the row's ends are read value
  // by value.  What the candidates need lies there once the stream has ended.
  extern __shared__ __align__(16) uint4 ring[];  // [kDepth][NV][kThreads]
  uint64_t* cand = reinterpret_cast<uint64_t*>(ring);
  uint64_t* few = cand + kCand;
  uint64_t* best = few + kCand;
  uint16_t* list = reinterpret_cast<uint16_t*>(best + kMaxOut);
  auto inside = [&](int64_t v) {
    const int64_t e = v * VE - off;
    return v < v_end && e >= 0 && e + VE <= p.vocab;
  };
  // Nothing of a step reaches over the row's or the piece's ends.
  auto whole = [&](int64_t v0) {
    return v0 * VE >= off && v0 + kStep <= v_end && (v0 + kStep) * VE - off <= p.vocab;
  };
  const uint32_t mine_at = smem_u32(ring + tid);
  constexpr int kPlace = kThreads * 16;  // bytes between a thread's vectors
  auto copy = [&](uint32_t dst, const T* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src)
                 : "memory");
  };
  auto issue = [&](int64_t v0, int place) {
    const uint32_t dst = mine_at + place * (NV * kPlace);
    const T* src = x + ((v0 + tid) * VE - off);
    if (whole(v0)) {
#pragma unroll
      for (int i = 0; i < NV; ++i) copy(dst + i * kPlace, src + i * (kThreads * VE));
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (inside(v0 + tid + i * kThreads))
          copy(dst + i * kPlace, src + i * (kThreads * VE));
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto unpack = [&](const uint4& raw, float (&f)[VE]) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int k = 0; k < VE; ++k) {
      if (sizeof(T) == 4)
        f[k] = __uint_as_float(w[k % 4]);
      else
        f[k] = __uint_as_float(k & 1 ? w[k / 2] & 0xffff0000u : w[k / 2] << 16);
    }
  };
  auto one_by_one = [&](int64_t v, float (&f)[VE]) {
    const int64_t e = v * VE - off;
#pragma unroll
    for (int k = 0; k < VE; ++k)
      f[k] = v < v_end && e + k >= 0 && e + k < p.vocab ? to_float(x[e + k]) : -INFINITY;
  };
  // The sum so far of exponentials of logits less m, the whole number at the first
  // step's maximum.  It moves, in a thread alone, only where a logit lies far above.
  float m = -INFINITY, ref = -INFINITY;
  float sum_hi = 0.f, sum_lo = 0.f;  // the sum and what its additions have rounded off
  // Largest logit of this thread, and of a group of its steps.
  float most = -INFINITY, of_group = -INFINITY;
  const int width = (steps + kGroups - 1) / kGroups;  // steps of a group
  int group = 0, in_group = 0;
#pragma unroll
  for (int k = 0; k < kDepth; ++k) issue(v_begin + (int64_t)k * kStep, k);
  int place = 0;
#pragma unroll 1
  for (int step = 0; step < steps; ++step) {
    const int64_t v0 = v_begin + (int64_t)step * kStep;
    float f[NV][VE];
    asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
    {
      const uint32_t src = mine_at + place * (NV * kPlace);
      const bool all = whole(v0);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (all || inside(v0 + tid + i * kThreads))
          unpack(lds128(src + i * kPlace), f[i]);
        else
          one_by_one(v0 + tid + i * kThreads, f[i]);
      }
    }
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < VE; k += 2) mx = fmaxf(mx, fmaxf(f[i][k], f[i][k + 1]));
    // (This step's values are in registers: its place is free.)
    issue(v0 + (int64_t)kDepth * kStep, place);
    place = place + 1 == kDepth ? 0 : place + 1;
    if (step == 0) {
      uint32_t lo, hi;
      range(ordered(mx), sh, lo, hi);
      m = ref = rintf(unordered(hi));
    }
    most = fmaxf(most, mx);
    of_group = fmaxf(of_group, mx);
    if (++in_group == width) {
      group_max[group++][tid] = (uint16_t)(ordered(of_group) >> 16);
      of_group = -INFINITY;
      in_group = 0;
    }
    if (mx > m + kHeadroom) {
      const float to = rintf(mx);
      const double y = ((double)sum_hi + sum_lo) * exp_of((double)m - to);
      sum_hi = (float)y;
      sum_lo = (float)(y - sum_hi);
      m = to;
    }
    if (m > -INFINITY) {
      // Two at a time; where one is not a number, again without it.
      const uint64_t neg = tc::pack2(-m, -m);
      const uint64_t scale = tc::pack2(1.4426950408889634f, 1.4426950408889634f);
      uint64_t s2 = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < VE; k += 2) {
          float y, z;
          tc::unpack2(tc::fma2(tc::add2(tc::pack2(f[i][k], f[i][k + 1]), neg), scale, 0),
                      y, z);
          s2 = tc::add2(s2, tc::pack2(ex2(y), ex2(z)));
        }
      float y, z;
      tc::unpack2(s2, y, z);
      float s = y + z;
      if (s != s) {
        s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int k = 0; k < VE; ++k) {
            if (f[i][k] != f[i][k]) f[i][k] = -INFINITY;
            s += ex2((f[i][k] - m) * 1.4426950408889634f);
          }
      }
      const float to = sum_hi + s, part = to - sum_hi;
      sum_lo += (sum_hi - (to - part)) + (s - part);
      sum_hi = to;
    }
  }
  if (in_group > 0) group_max[group++][tid] = (uint16_t)(ordered(of_group) >> 16);
  // (Nothing is on its way to the ring any more, which is used for other things.)
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (tid == 0) count = listed = 0;
  // Threads that have moved their reference (rare): back to a common one.
  if (__syncthreads_or(m != ref)) {
    uint32_t lo, hi;
    range(ordered(m), sh, lo, hi);
    ref = unordered(hi);
    const double y =
        m > -INFINITY ? ((double)sum_hi + sum_lo) * exp_of((double)m - ref) : 0.;
    sum_hi = (float)y;
    sum_lo = (float)(y - sum_hi);
    __syncthreads();
  }
  auto join = [&](int o) {
    const float y = __shfl_xor_sync(0xffffffffu, sum_hi, o);
    sum_lo += __shfl_xor_sync(0xffffffffu, sum_lo, o);
    // (The larger first.)
    const float a = fmaxf(sum_hi, y), b = fminf(sum_hi, y);
    sum_hi = a + b;
    sum_lo += b - (sum_hi - a);
  };
#pragma unroll
  for (int o = 16; o; o >>= 1) join(o);
  if ((tid & 31) == 0) sums[tid >> 5] = make_float2(sum_hi, sum_lo);
  // Candidates: logits from a value on that n threads' largest reach.  They lie in the
  // groups whose largest reach it (compared by their upper halves), which are read
  // again.
  uint32_t lo, hi;
  range(ordered(most), sh, lo, hi);
  const uint32_t bar = threshold(ordered(most), lo, hi, kNone32 + 1, n);
  const int64_t at = (int64_t)row * p.pieces + piece;
  if (tid < 32) {
    sum_hi = sums[tid % (kThreads / 32)].x;
    sum_lo = sums[tid % (kThreads / 32)].y;
#pragma unroll
    for (int o = kThreads / 64; o; o >>= 1) join(o);
    if (tid == 0) p.stats[at] = Stat{sum_hi, sum_lo, ref, 0.f};
  }
  for (int g = 0; g < group; ++g)
    if (group_max[g][tid] >= bar >> 16) {
      const int i = atomicAdd(&listed, 1);
      if (i < kList) list[i] = (uint16_t)(g * kThreads + tid);
    }
  __syncthreads();
  auto vector = [&](int64_t v, float (&f)[VE]) {
    if (inside(v))
      unpack(__ldg(reinterpret_cast<const uint4*>(x + (v * VE - off))), f);
    else
      one_by_one(v, f);
  };
  // Higher logits first, then lower tokens.
  auto key = [&](float y, int64_t v, int k) {
    return (uint64_t)ordered(y) << 32 | (0xffffffffu - (uint32_t)(v * VE - off + k));
  };
  auto reaches = [&](float y) { return y == y && ordered(y) >= bar; };
  const int groups = listed;
  if (groups <= kList) {
    for (int i = tid; i < groups * width; i += kThreads) {
      const int e = list[i / width], step = e / kThreads * width + i % width;
      if (step >= steps) continue;
      const int64_t v = v_begin + (int64_t)step * kStep + e % kThreads;
      float f[NV][VE];
#pragma unroll
      for (int j = 0; j < NV; ++j) vector(v + j * kThreads, f[j]);
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < VE; ++k)
          if (reaches(f[j][k])) {
            const int to = atomicAdd(&count, 1);
            if (to < kCand) cand[to] = key(f[j][k], v + j * kThreads, k);
          }
    }
  }
  __syncthreads();
  int c = count;
  if (groups > kList || c > kCand) {
    // Many equal logits, or few threads with any: the n-th highest key by its digits.
    auto each = [&](auto&& f) {
      auto of_vector = [&](int64_t v, bool there) {
        float y[VE];
        vector(there ? v : v_end, y);
#pragma unroll
        for (int k = 0; k < VE; ++k) f(reaches(y[k]), key(y[k], v, k));
      };
      if (groups <= kList) {
        for (int i0 = 0; i0 < groups * width; i0 += kThreads) {
          const int i = min(i0 + tid, groups * width - 1);
          const int e = list[i / width], step = e / kThreads * width + i % width;
          for (int j = 0; j < NV; ++j)
            of_vector(v_begin + (int64_t)step * kStep + e % kThreads + j * kThreads,
                      i0 + tid == i && step < steps);
        }
      } else {
        for (int64_t v0 = v_begin; v0 < v_end; v0 += kThreads) of_vector(v0 + tid, true);
      }
    };
    // Digits that all of them share: of the logits between the bar and the highest, and
    // where those are equal, of the piece's tokens.
    const int64_t first = max(v_begin * VE - off, (int64_t)0), end = v_end * VE - off;
    const uint64_t high = (uint64_t)hi << 32 | (0xffffffffu - (uint32_t)first);
    const uint64_t low = (uint64_t)bar << 32 | (0xffffffffu - (uint32_t)end);
    const int top = (63 - __clzll((long long)(high ^ low))) & ~7;
    const uint64_t mask = top == 56 ? 0 : ~0ull << (top + 8);
    int last = n;
    const uint64_t least = nth_key(each, top, high & mask, mask, last, digits);
    if (tid == 0) count = 0;
    __syncthreads();
    each([&](bool in, uint64_t a) {
      if (in && a >= least) cand[atomicAdd(&count, 1)] = a;
    });
    __syncthreads();
    c = count;
  }
  pick_best(cand, c, n, unordered(bar), few, best, sh, &few_count);
  uint2* out = p.entries + at * n;
  for (int i = tid; i < n; i += kThreads)
    out[i] = best[i] ? make_uint2((uint32_t)(best[i] >> 32), ~(uint32_t)best[i])
                     : make_uint2(0, 0);
}

struct Cand {
  uint64_t y;   // ordered
  uint64_t at;  // beam, and token in the lower half
};

__device__ __forceinline__ double value_of(uint64_t y) {
  return __longlong_as_double(
      (long long)(y & 0x8000000000000000ull ? y ^ 0x8000000000000000ull : ~y));
}

__device__ __forceinline__ bool before(const Cand& a, const Cand& b) {
  return a.y > b.y || (a.y == b.y && a.at < b.at);
}

// A CTA for each group.  The tables are made while the pieces are still read.
__global__ void __launch_bounds__(kThreads) group_kernel(const Params p) {
  __shared__ Cand cand[kCand];
  __shared__ int which[kCand];
  // Score less log sum exp(x - top), NaN: no continuations.  The highest reference is
  // kept apart, so that logits of any size cancel before the score is added.
  __shared__ double offset[kMaxBeams];
  __shared__ float near_offset[kMaxBeams], top[kMaxBeams];
  __shared__ double e_ones[32], e_32s[24];   // e^-k, e^-32k
  __shared__ double log_at[65];              // log of c = 1 / (inverse of 1 + k / 64)
  __shared__ uint32_t largest;  // |offset| of the beams, at most
  __shared__ uint32_t sh[64];
  __shared__ Digits digits;
  __shared__ int count;
  const int group = blockIdx.x, tid = threadIdx.x, n = p.n;
  auto inverse_at = [](int k) { return (double)(1.f / (1.f + (float)k * 0.015625f)); };
  if (tid < 32) {
    e_ones[tid] = exp_of(-(double)tid);
  } else if (tid < 32 + 24) {
    e_32s[tid - 32] = exp_of(-32. * (tid - 32));
  } else if (tid >= 64 && tid < 64 + 65) {
    log_at[tid - 64] = -log_of(inverse_at(tid - 64));
  } else if (tid == 63) {
    count = 0;
    largest = 0;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t row0 = (int64_t)group * p.beams;
  const int per = p.pieces * n, total = p.beams * per;
  const uint2* entries = p.entries + (int64_t)group * total;
  const float* scores = p.scores + row0;
  const Stat* stats = p.stats + row0 * p.pieces;
  auto entry = [&](int i) { return i < total ? entries[i] : make_uint2(0, 0); };
  const int turns = (total + kThreads - 1) / kThreads;
  // A piece's entries come highest first: `1 << p.heads` of each, 2048 in all at most,
  // are looked at first.  A thread has its share of several ranks.
  constexpr int kOwn = 8;
  auto head = [&](int k) {
    const int at = k * kThreads + ((tid + 37 * k) & (kThreads - 1));
    const int rank = at & ((1 << p.heads) - 1);
    return rank < n ? min((at >> p.heads) * n + rank, total) : total;
  };
  uint2 own[kOwn];
#pragma unroll
  for (int k = 0; k < kOwn; ++k) own[k] = entry(head(k));
  __syncthreads();
  // As many lanes a beam as it has pieces (a power of two, at most a warp).
  int lanes = 1;
  while (lanes < p.pieces && lanes < 32) lanes <<= 1;
  for (int b0 = 0; b0 < p.beams; b0 += kThreads / lanes) {
    const int b = b0 + tid / lanes, l = tid % lanes;
    // (Beams that are not there have no sums.)
    const float score = b < p.beams ? scores[b] : -INFINITY;
    const Stat none{0.f, 0.f, -INFINITY, 0.f};
    Stat first = b < p.beams && l < p.pieces ? stats[b * p.pieces + l] : none;
    const bool there = score > -INFINITY;
    if (!there) first = none;
    float m = first.top;
    for (int i = l + lanes; there && i < p.pieces; i += lanes)
      m = fmaxf(m, stats[b * p.pieces + i].top);
    for (int o = lanes >> 1; o; o >>= 1)
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    // The references are whole numbers, and so is what lies between them.
    auto part = [&](const Stat& x) {
      const float d = m - x.top;
      if (!(d < 700.f)) return 0.;
      const int k = (int)d;
      const double y = (double)x.sum + x.rest;
      return k == 0 ? y : y * e_ones[k & 31] * e_32s[k >> 5];
    };
    double sum = part(first);
    for (int i = l + lanes; there && i < p.pieces; i += lanes)
      sum += part(stats[b * p.pieces + i]);
    for (int o = lanes >> 1; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (l == 0 && b < p.beams) {
      double at = NAN;
      // (A logit of +infinity: no continuations.)
      if (there && sum > 0 && m < INFINITY) {
        // sum = f 2^e, log f = log c + log(1 + r), r = f / c - 1 within 2^-7: its
        // series in fp32 is off by 2^-31.
        const long long bits = __double_as_longlong(sum);
        const double f = __longlong_as_double((bits & 0xfffffffffffffll) | 1023ll << 52);
        const int k = (int)((bits >> 45 & 127) + 1) >> 1;
        const float r = (float)fma(f, inverse_at(k), -1.);
        const float series =
            r * fmaf(r, fmaf(r, fmaf(r, fmaf(r, .2f, -.25f), 1.f / 3), -.5f), 1.f);
        at = (double)score - (fma((double)((int)(bits >> 52) - 1023), 0.6931471805599453,
                                  log_at[k]) + series);
        atomicMax(&largest, __float_as_uint(fabsf((float)at)));
      }
      offset[b] = at;
      near_offset[b] = (float)at;
      top[b] = m;
    }
  }
  __syncthreads();
  // An entry's beam: i + 1/2 is exact, and at least 1 / (2 per) of a beam from the
  // next whole number, which two roundings of at most total / per beams do not reach.
  const float inv_per = 1.f / (float)per;
  auto beam_of = [&](int i) { return (int)(((float)i + .5f) * inv_per); };
  auto get = [&](const uint2& e, int i) {
    const int b = beam_of(i);
    const double at = offset[b];
    if (e.x == 0 || isnan(at)) return Cand{0, 0};
    const double y = at + ((double)unordered(e.x) - top[b]);
    if (!(y > -INFINITY)) return Cand{0, 0};
    return Cand{ordered(y), (uint64_t)b << 32 | e.y};
  };
  // The same in fp32, off by less than 2^-21 (|offset| + |x - top| + |y|), the second at
  // most the others: a bar on these, lowered by that twice (and a half more), leaves
  // few results to be computed in 64 bits.
  auto near = [&](const uint2& e, int i) {
    const int b = beam_of(min(i, total - 1));
    const float at = near_offset[b];
    if (e.x == 0 || at != at) return -INFINITY;
    return fmaxf(at + (unordered(e.x) - top[b]), -FLT_MAX);
  };
  float near_own[kOwn], most = -INFINITY;
#pragma unroll
  for (int k = 0; k < kOwn; ++k) {
    near_own[k] = -INFINITY;
    if (k * kThreads < (p.beams * p.pieces) << p.heads)
      near_own[k] = near(own[k], head(k));
    most = fmaxf(most, near_own[k]);
  }
  uint32_t lo, hi;
  range(ordered(most), sh, lo, hi);
  auto lowered = [&](uint32_t key) {
    float bar = unordered(key);
    bar -= (fabsf(bar) + 2.f * __uint_as_float(largest)) * 0x1p-19f;
    return bar > -INFINITY ? bar : -INFINITY;  // (fewer than n, or no finite margin)
  };
  float bar = lowered(threshold(ordered(most), lo, hi, kNone32, n));
  auto add = [&](int i, float y) {
    if (y < bar || y == -INFINITY) return false;
    const int at = atomicAdd(&count, 1);
    if (at < kCand) which[at] = i;
    return true;
  };
  if (most >= bar) {
    uint32_t reached = 0;  // turns
#pragma unroll
    for (int k = 0; k < kOwn; ++k)
      if (add(head(k), near_own[k])) reached |= 1u << k;
    // The last ones looked at of a piece: on, as far as they reach the bar.
    if (1 << p.heads >= n) reached = 0;
#pragma unroll 1
    for (; reached; reached &= reached - 1) {
      const int at = head(__ffs(reached) - 1), left = n - 1 - at % n;
      if (n - left != 1 << p.heads) continue;
      bool more = true;
      for (int r = 1; more && r <= left; r += 4) {
        float y[4];
#pragma unroll
        for (int z = 0; z < 4; ++z)
          y[z] = r + z <= left ? near(entry(at + r + z), at + r + z) : -INFINITY;
#pragma unroll
        for (int z = 0; z < 4; ++z) more = more && add(at + r + z, y[z]);
      }
    }
  }
  __syncthreads();
  if (count > kCand) {
    // The bar is too low: from the n-th highest of all.
    int last = n;
    const uint32_t nth = (uint32_t)nth_key(
        [&](auto&& f) {
          for (int k = 0; k < turns; ++k) {
            const int i = k * kThreads + tid;
            const float y = near(entry(i), i);
            f(y > -INFINITY, ordered(y));
          }
        },
        24, 0, 0, last, digits);
    bar = lowered(nth);
    if (tid == 0) count = 0;
    __syncthreads();
    for (int i = tid; i < total; i += kThreads) add(i, near(entries[i], i));
    __syncthreads();
  }
  // Those in 64 bits.
  for (int i = tid; i < min(count, kCand); i += kThreads)
    cand[i] = get(entries[which[i]], which[i]);
  __syncthreads();
  const int c = count;
  auto put = [&](int rank, const Cand& a) {
    const int64_t at = (int64_t)group * n + rank;
    p.out_scores[at] = (float)value_of(a.y);
    p.out_parents[at] = (int32_t)(a.at >> 32);
    p.out_tokens[at] = (int32_t)a.at;
  };
  for (int i = c + tid; i < n; i += kThreads) {
    const int64_t at = (int64_t)group * n + i;
    p.out_scores[at] = -INFINITY;
    p.out_parents[at] = p.out_tokens[at] = -1;
  }
  auto rank_and_put = [&](int c) {
    // Eight threads a result.
    for (int i0 = 0; i0 < c; i0 += kThreads / 8) {
      const int i = i0 + (tid >> 3);
      const Cand a = i < c ? cand[i] : Cand{0, 0};
      int rank = 0;
      for (int j = tid & 7; j < c; j += 8) rank += before(cand[j], a);
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
      if (i < c && rank < n && (tid & 7) == 0) put(rank, a);
    }
  };
  if (c <= kCand) {
    rank_and_put(c);
    return;
  }
  // Many equal results (c > n of them): the n-th highest, and of its equals the first.
  auto each = [&](auto&& f) {
    for (int k = 0; k < turns; ++k) {
      const int i = k * kThreads + tid;
      const uint2 e = entry(i);
      const Cand a = near(e, i) >= bar ? get(e, min(i, total - 1)) : Cand{0, 0};
      f(a);
    }
  };
  int last = n;
  const uint64_t y = nth_key(
      [&](auto&& f) { each([&](const Cand& a) { f(a.y != 0, a.y); }); }, 56, 0, 0, last,
      digits);
  uint64_t at = 0;
  if (last > 0)
    at = nth_key(
        [&](auto&& f) {
          each([&](const Cand& a) { f(a.y == y, ~a.at & 0xffffffffffffull); });
        },
        40, 0, 0, last, digits);
  if (tid == 0) count = 0;
  __syncthreads();
  each([&](const Cand& a) {
    if (a.y > y || (a.y == y && (~a.at & 0xffffffffffffull) >= at))
      cand[atomicAdd(&count, 1)] = a;
  });
  __syncthreads();
  rank_and_put(count);
}

// Pieces of a row, of 2048 logits at least and for three rounds of CTAs (four on an SM)
// at most: those that are done first.  A round costs about 5 us (its first reads, the
// bar, the groups read again), and the logits either the time of a CTA's share, 0.15 us
// a thousand where reads' latency counts, or that of their bytes.  (By how full the
// rounds are alone, 203 beams of 19163 went in eight pieces and three rounds, 32 us;
// in two 14.6.)
int64_t n_pieces(int64_t rows, int vocab) {
  const int64_t most = std::min(((int64_t)vocab + 2047) / 2048,
                                std::max<int64_t>(3 * kRound / rows, 1));
  const double bytes_us = (double)rows * vocab * 4 / 6e6;
  int64_t best = 1;
  double least = 1e300;
  for (int64_t p = 1; p <= most; ++p) {
    const double rounds = (double)((rows * p + kRound - 1) / kRound);
    const double us =
        rounds * 5 + std::max(rounds * (double)vocab / (double)p * 0.15e-3, bytes_us);
    if (us < least * 0.98) {
      least = us;
      best = p;
    }
  }
  return best;
}

kv_status sizes_ok(int32_t n_groups, int32_t beams, int32_t vocab, int32_t n_out) {
  if (n_groups < 1 || beams < 1 || beams > kMaxBeams || vocab < 1)
    return fail(KV_ERR_INVALID_ARG, "bad n_groups/beams/vocab (%d/%d/%d)", n_groups,
                beams, vocab);
  if (n_out < 1 || n_out > kMaxOut)
    return fail(KV_ERR_INVALID_ARG, "n_out %d outside [1, %d]", n_out, kMaxOut);
  const int64_t rows = (int64_t)n_groups * beams;
  if (rows > 65535) return fail(KV_ERR_INVALID_ARG, "more than 65535 beams");
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
  for (p.heads = 0; (2 << p.heads) * p.pieces * beams <= 2048 && 1 << p.heads < n_out;)
    ++p.heads;
  cudaStream_t st = (cudaStream_t)stream;
  const dim3 grid((unsigned)p.pieces, (unsigned)rows);
  const bool big = vocab / p.pieces > 4096;  // steps of 4096 logits, else of 2048
  auto launch = [&](auto kernel, int ring) {
    return pkv::launch_early<true>(kernel, grid, W::kThreads, ring, st, p);
  };
  using bf16 = __nv_bfloat16;
  cudaError_t e = f32 && big ? launch(W::piece_kernel<float, 16>, W::kRingBytes<float, 16>)
                  : f32      ? launch(W::piece_kernel<float, 8>, W::kRingBytes<float, 8>)
                  : big      ? launch(W::piece_kernel<bf16, 16>, W::kRingBytes<bf16, 16>)
                             : launch(W::piece_kernel<bf16, 8>, W::kRingBytes<bf16, 8>);
  if (e == cudaSuccess)
    e = pkv::launch_early<true>(W::group_kernel, n_groups, W::kThreads, 0, st, p);
  if (e != cudaSuccess)
    return fail(KV_ERR_CUDA, "beam selection: %s", cudaGetErrorString(e));
  return KV_OK;
}
