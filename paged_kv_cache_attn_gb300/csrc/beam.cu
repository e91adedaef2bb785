// Beam selection (kv_beam_select): of every group of beams the n continuations
// (beam, token) with the highest
//   y = score[beam] + x[token] - log sum_t exp x[t],
// ties to the lower beam, then the lower token.  Bound by the logits' bytes: they are
// read once.
//
// First kernel: a CTA streams a piece of one beam's logits through registers, a step of
// up to 4096 at a time, and each thread adds up exponentials.
// Of one beam the order of y is that of x: the CTA keeps candidates for the n highest
// logits, and of what comes in only logits above a bar that n of those before reach.
// The bar is taken from the threads' maxima of a step (a value that at least n of them
// reach, and not many more, by bisection over counts).  Nearly all of a row lies below
// it and costs no more than its sum and one barrier a step.  Second kernel: a CTA per
// group joins the sums in 64 bits and picks the n highest y of the pieces' candidates.
//
// y is computed in 64 bits from sums of at most 16 exponentials in fp32 (added up with
// what each addition rounds off, and across threads in 64 bits: 64-bit operations are
// issued one lane pair a cycle here, and an addition a thread and step bounded the
// kernel), about 1e-7 from exact, so that beams are hardly ever ordered otherwise than
// exactly.

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
constexpr int kMaxParts = 3 * kRound;             // beams x pieces of a group
constexpr int kCand = 768;   // candidates in shared memory; more: one at a time
constexpr float kHeadroom = 40.f;  // of logits above the reference of a sum

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

// The n highest of c <= kCand keys to best, in order (0 where there are fewer).  Of
// many, a bar that n of the threads' highest keys reach leaves few to be ranked.  `floor`: a logit
// that all of them reach.
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
  for (int i = tid; i < k; i += kThreads) {
    const uint64_t a = from[i];
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < k; ++j) rank += from[j] > a;
    if (rank < n) best[rank] = a;
  }
  __syncthreads();
}

// e^x in 64 bits for x <= 0: x / ln 2 split into a whole number and at most half of one
// either way, its Taylor series to the 11th power (2e-14 relative).  Few operations:
// 64-bit ones are issued one lane pair a cycle here, and this kernel waits for each.
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
  __shared__ uint64_t cand[kCand], few[kCand], best[kMaxOut];
  __shared__ uint32_t sh[64];
  __shared__ double sums[kThreads / 32];
  __shared__ int count, few_count;
  __shared__ unsigned long long top;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int row = blockIdx.y, piece = blockIdx.x, tid = threadIdx.x, n = p.n;
  if (!(p.scores[row] > -INFINITY)) return;  // no beam
  const T* x = static_cast<const T*>(p.logits) + (int64_t)row * p.stride;
  // Vectors start on 16-byte borders, the first at or before the row's start.
  const int off = (int)((uintptr_t)x % 16 / sizeof(T));
  const int64_t vectors = ((int64_t)p.vocab + off + VE - 1) / VE;
  const int64_t v_begin = vectors * piece / p.pieces;
  const int64_t v_end = vectors * (piece + 1) / p.pieces;
  if (tid == 0) count = 0;
  __syncthreads();
  // The sum so far of exponentials of logits less m, the first step's maximum.  It
  // moves, in a thread alone, only where a logit lies far above it.
  float m = -INFINITY, ref = -INFINITY;
  float sum_hi = 0.f, sum_lo = 0.f;  // the sum and what its additions have rounded off
  float bar = -INFINITY;  // what comes in is a candidate above it
  int bound = 0;          // candidates at most
  int fresh = 0;          // threads that have brought some since the bar rose
  bool picked = false;    // `best` holds the n highest of them
  // Each thread's vectors of the next two steps are on their way to its own places in
  // shared memory (32 KB a CTA, 128 KB an SM: with one step in registers the loads'
  // latency, 1.9 us under load, kept an SM at 29 GB/s).  Vectors that reach over the
  // row's ends are read value by value.
  extern __shared__ __align__(16) uint4 ring[];  // [2][NV][kThreads]
  auto inside = [&](int64_t v) {
    const int64_t e = v * VE - off;
    return v < v_end && e >= 0 && e + VE <= p.vocab;
  };
  constexpr int kStep = kThreads * NV;
  // Nothing of a step reaches over the row's or the piece's ends.
  auto whole = [&](int64_t step) {
    return step * VE >= off && step + kStep <= v_end &&
           (step + kStep) * VE - off <= p.vocab;
  };
  const uint32_t mine_at = smem_u32(ring + tid);
  constexpr int kPlace = kThreads * 16;  // bytes between a thread's vectors
  auto copy = [&](uint32_t dst, const T* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src)
                 : "memory");
  };
  auto issue = [&](int64_t step, int slot) {
    const uint32_t dst = mine_at + slot * (NV * kPlace);
    const T* src = x + ((step + tid) * VE - off);
    if (whole(step)) {
#pragma unroll
      for (int i = 0; i < NV; ++i) copy(dst + i * kPlace, src + i * (kThreads * VE));
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (inside(step + tid + i * kThreads))
          copy(dst + i * kPlace, src + i * (kThreads * VE));
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto fetch = [&](float (&f)[NV][VE], int64_t step, int slot) {
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    const uint32_t src = mine_at + slot * (NV * kPlace);
    const bool all = whole(step);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (all || inside(step + tid + i * kThreads)) {
        const uint4 raw = lds128(src + i * kPlace);
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int k = 0; k < VE; ++k) {
          if (sizeof(T) == 4)
            f[i][k] = __uint_as_float(w[k % 4]);
          else
            f[i][k] = __uint_as_float(k & 1 ? w[k / 2] & 0xffff0000u : w[k / 2] << 16);
        }
      } else {
        const int64_t v = step + tid + i * kThreads, e = v * VE - off;
#pragma unroll
        for (int k = 0; k < VE; ++k)
          f[i][k] = v < v_end && e + k >= 0 && e + k < p.vocab ? to_float(x[e + k])
                                                              : -INFINITY;
      }
    }
  };
  auto process = [&](float (&f)[NV][VE], int64_t step, int slot) {
    const int64_t v0 = step + tid;
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < VE; ++k) {
        mx = fmaxf(mx, f[i][k]);  // (passes over NaN)
      }
    // (This step's values are in registers: its place is free.)
    const int over = __syncthreads_count(mx > bar);
    issue(step + 2 * kStep, slot);
    uint32_t lo = 0, hi = 0;  // least and largest of the threads' maxima
    // (Of a first step with logits m is -inf in every thread.)
    if (over > n || (over > 0 && bar == -INFINITY)) {
      range(ordered(mx), sh, lo, hi);
      if (m == -INFINITY) m = ref = unordered(hi);
    }
    if (mx > m + kHeadroom) {
      const double y = ((double)sum_hi + sum_lo) * exp_of((double)m - mx);
      sum_hi = (float)y;
      sum_lo = (float)(y - sum_hi);
      m = mx;
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
    if (over == 0) return;
    // Candidates: above the bar; where more than n threads have some, from a value
    // on that n of them reach, which is a bar for what comes later.
    float from = bar;
    bool equal = false;
    int before = 0;
    fresh += over;
    picked = false;
    const bool many = fresh > n || bound + over * E > kCand;
    if (many) {
      if (over > n) {
        from = unordered(threshold(ordered(mx), lo, hi, ordered(bar) + 1, n));
        equal = true;
      }
      __syncthreads();
      before = count;
      __syncthreads();
    }
    // Higher logits first, then lower tokens.
    auto key = [&](int i, int k) {
      const uint32_t token = (uint32_t)((v0 + i * kThreads) * VE - off + k);
      return (uint64_t)ordered(f[i][k]) << 32 | (0xffffffffu - token);
    };
    // Few lanes have any, and those one, as a rule: which, without branches, then
    // theirs alone.
    if (mx > from || (equal && mx == from)) {
      uint32_t mask = 0;
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const float y = f[j / VE][j % VE];
        mask |= (y > from || (equal && y == from) ? 1u : 0u) << j;
      }
      while (mask) {
        const int j = __ffs(mask) - 1;
        mask &= mask - 1;
        float y = f[0][0];
#pragma unroll
        for (int k = 1; k < E; ++k) y = j == k ? f[k / VE][k % VE] : y;
        const uint32_t token =
            (uint32_t)((v0 + j / VE * kThreads) * VE - off + j % VE);
        const int at = atomicAdd(&count, 1);
        if (at < kCand) cand[at] = (uint64_t)ordered(y) << 32 | (0xffffffffu - token);
      }
    }
    bound += over * E;
    if (equal) bar = from;
    if (!many) return;
    __syncthreads();
    int c = count;
    __syncthreads();
    if (c > kCand) {
      // Many equal logits: the n highest of this step one at a time, behind the
      // candidates there were, or the n highest of those (there are more than n).
      if (before + n > kCand) {
        pick_best(cand, before, n, bar, few, best, sh, &few_count);
        for (int i = tid; i < n; i += kThreads) cand[i] = best[i];
        before = n;
        __syncthreads();
      }
      uint64_t last = ~0ull;
      for (int r = 0; r < n; ++r) {
        uint64_t most = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int k = 0; k < VE; ++k) {
            const uint64_t a = key(i, k);
            if (a < last && a > most) most = a;
          }
        if (tid == 0) top = 0;
        __syncthreads();
#pragma unroll
        for (int o = 16; o; o >>= 1)
          most = max(most, (uint64_t)__shfl_xor_sync(0xffffffffu, most, o));
        if ((tid & 31) == 0) atomicMax(&top, (unsigned long long)most);
        __syncthreads();
        last = top;
        if (tid == 0) cand[before + r] = last;
        __syncthreads();
      }
      c = before + n;
    }
    if (c > n) {
      // The n highest so far: the lowest of them is the bar.
      pick_best(cand, c, n, bar, few, best, sh, &few_count);
      for (int i = tid; i < n; i += kThreads) cand[i] = best[i];
      bar = fmaxf(bar, unordered((uint32_t)(best[n - 1] >> 32)));
      c = n;
      picked = true;
    }
    __syncthreads();
    if (tid == 0) count = c;
    bound = c;
    fresh = 0;
    __syncthreads();
  };
  issue(v_begin, 0);
  issue(v_begin + kStep, 1);
  int slot = 0;
  for (int64_t step = v_begin; step < v_end; step += kStep, slot ^= 1) {
    float f[NV][VE];
    fetch(f, step, slot);
    process(f, step, slot);
  }
  // Threads that have moved their reference (rare): back to a common one.
  if (__syncthreads_or(m != ref)) {
    uint32_t lo, hi;
    range(ordered(m), sh, lo, hi);
    ref = unordered(hi);
    const double y =
        m > -INFINITY ? ((double)sum_hi + sum_lo) * exp_of((double)m - ref) : 0.;
    sum_hi = (float)y;
    sum_lo = (float)(y - sum_hi);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float y = __shfl_xor_sync(0xffffffffu, sum_hi, o);
    sum_lo += __shfl_xor_sync(0xffffffffu, sum_lo, o);
    // (The larger first.)
    const float a = fmaxf(sum_hi, y), b = fminf(sum_hi, y);
    sum_hi = a + b;
    sum_lo += b - (sum_hi - a);
  }
  if ((tid & 31) == 0) sums[tid >> 5] = (double)sum_hi + sum_lo;
  __syncthreads();
  const int64_t at = (int64_t)row * p.pieces + piece;
  if (tid == 0) {
    double all = 0;
    for (int w = 0; w < kThreads / 32; ++w) all += sums[w];
    p.stats[at] = Stat{all, ref, 0.f};
  }
  // (Picked already where nothing came after.)
  if (!picked) pick_best(cand, count, n, bar, few, best, sh, &few_count);
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

__global__ void __launch_bounds__(kThreads) group_kernel(const Params p) {
  __shared__ Cand cand[kCand];
  __shared__ int which[kCand];
  // log sum exp(x - top), NaN: no continuations.  Kept apart from the highest logit,
  // so that logits of any size cancel before the score is added.
  __shared__ double log_sum[kMaxBeams], parts[kMaxParts];
  __shared__ uint32_t top[kMaxBeams];  // highest logit, ordered
  __shared__ uint32_t largest;  // |score| + |log sum| of the beams, at most
  __shared__ uint32_t sh[64];
  __shared__ Cand best_of[kThreads / 32];
  __shared__ int count;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int group = blockIdx.x, tid = threadIdx.x, lane = tid & 31, n = p.n;
  const int64_t row0 = (int64_t)group * p.beams;
  const int per = p.pieces * n, total = p.beams * per;
  const uint2* entries = p.entries + (int64_t)group * total;
  const float* scores = p.scores + row0;
  // A thread's first entries, and the first of its pieces' sums, asked for together.
  constexpr int kOwn = 8;
  uint2 own[kOwn];
#pragma unroll
  for (int i = 0; i < kOwn; ++i)
    own[i] = tid + i * kThreads < total ? entries[tid + i * kThreads] : make_uint2(0, 0);
  for (int b = tid; b < p.beams; b += kThreads) top[b] = kNone32;
  if (tid == 0) {
    count = 0;
    largest = 0;
  }
  __syncthreads();
  // (Beams that are not there have no sums.)
  Stat st{0, -INFINITY, 0};
  auto sum_of = [&](int i) {
    return scores[i / p.pieces] > -INFINITY ? p.stats[row0 * p.pieces + i]
                                            : Stat{0, -INFINITY, 0};
  };
  const int sums = p.beams * p.pieces;
  if (tid < sums) st = sum_of(tid);
  for (int i = tid; i < sums; i += kThreads)
    atomicMax(&top[i / p.pieces], ordered((i == tid ? st : sum_of(i)).top));
  __syncthreads();
  for (int i = tid; i < sums; i += kThreads) {
    const Stat x = i == tid ? st : sum_of(i);
    const float m = unordered(top[i / p.pieces]);
    // A logit of +infinity: no continuations.
    parts[i] = !(x.top > -INFINITY) || m == INFINITY ? 0.
               : x.top == m                          ? x.sum
                                                     : x.sum * exp_of((double)x.top - m);
  }
  __syncthreads();
  for (int b = tid; b < p.beams; b += kThreads) {
    double s[4] = {0, 0, 0, 0};
    for (int i = 0; i < p.pieces; i += 4)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i + k < p.pieces) s[k] += parts[b * p.pieces + i + k];
    const double all = (s[0] + s[1]) + (s[2] + s[3]);
    const double l = all > 0 ? log_of(all) : NAN;
    log_sum[b] = l;
    if (all > 0) atomicMax(&largest, __float_as_uint(fabsf(scores[b]) + fabsf((float)l)));
  }
  __syncthreads();
  auto get = [&](const uint2& e, int i) {
    const int b = i / per;
    const double l = log_sum[b];
    if (e.x == 0 || isnan(l)) return Cand{0, 0};
    const double y =
        (double)scores[b] + (((double)unordered(e.x) - unordered(top[b])) - l);
    if (!(y > -INFINITY)) return Cand{0, 0};
    return Cand{ordered(y), (uint64_t)b << 32 | e.y};
  };
  // The same in fp32, off by less than 2^-21 (|score| + |log sum| + |x - top|), the
  // last at most the first two and |y|: a bar on these, lowered by that twice (and a
  // half more), leaves few results to be computed in 64 bits.
  auto near = [&](const uint2& e, int i) {
    const int b = min(i, total - 1) / per;
    const float l = (float)log_sum[b];
    if (e.x == 0 || l != l) return -INFINITY;
    return fmaxf(scores[b] + ((unordered(e.x) - unordered(top[b])) - l), -FLT_MAX);
  };
  float near_own[kOwn], most = -INFINITY;
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    near_own[i] = near(own[i], tid + i * kThreads);
    most = fmaxf(most, near_own[i]);
  }
  for (int i = tid + kOwn * kThreads; i < total; i += kThreads)
    most = fmaxf(most, near(entries[i], i));
  uint32_t lo, hi;
  range(ordered(most), sh, lo, hi);
  float bar = unordered(threshold(ordered(most), lo, hi, kNone32, n));
  bar -= (fabsf(bar) + 2.f * __uint_as_float(largest)) * 0x1p-19f;
  if (!(bar > -INFINITY)) bar = -INFINITY;  // (fewer than n, or no finite margin)
  auto add = [&](int i, float y) {
    if (y < bar || y == -INFINITY || i >= total) return;
    const int at = atomicAdd(&count, 1);
    if (at < kCand) which[at] = i;
  };
  if (most >= bar) {
#pragma unroll
    for (int i = 0; i < kOwn; ++i) add(tid + i * kThreads, near_own[i]);
    for (int i = tid + kOwn * kThreads; i < total; i += kThreads)
      add(i, near(entries[i], i));
  }
  __syncthreads();
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
  Cand last{~0ull, 0};
  for (int r = 0; r < n; ++r) {
    Cand best{0, 0};
    for (int i = tid; i < total; i += kThreads) {
      const Cand a = get(entries[i], i);
      if (a.y && before(last, a) && before(a, best)) best = a;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const Cand a{__shfl_xor_sync(0xffffffffu, best.y, o),
                   __shfl_xor_sync(0xffffffffu, best.at, o)};
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

// Pieces of a row, of 2048 logits at least: one to three rounds of CTAs (four on an
// SM), whichever is filled best.
int64_t n_pieces(int64_t rows, int vocab) {
  const int64_t most = ((int64_t)vocab + 2047) / 2048;
  int64_t best = 1;
  double filled = 0;
  for (int64_t rounds = 1; rounds <= 3; ++rounds) {
    const int64_t p = std::clamp<int64_t>(rounds * kRound / rows, 1, most);
    const int64_t r = (rows * p + kRound - 1) / kRound;
    const double f = (double)(rows * p) / (double)(r * kRound);
    if (f > filled * 1.02) {
      filled = f;
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
  cudaStream_t st = (cudaStream_t)stream;
  const dim3 grid((unsigned)p.pieces, (unsigned)rows);
  const bool big = vocab / p.pieces > 4096;  // steps of 4096 logits, else of 2048
  // (Below the 48 KB that need no opting in.)
  const int ring = 2 * W::kThreads * (big ? 16 : 8) * (f32 ? 4 : 2);
  if (f32 && big)
    W::piece_kernel<float, 16><<<grid, W::kThreads, ring, st>>>(p);
  else if (f32)
    W::piece_kernel<float, 8><<<grid, W::kThreads, ring, st>>>(p);
  else if (big)
    W::piece_kernel<__nv_bfloat16, 16><<<grid, W::kThreads, ring, st>>>(p);
  else
    W::piece_kernel<__nv_bfloat16, 8><<<grid, W::kThreads, ring, st>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess)
    e = pkv::launch_early(W::group_kernel, n_groups, W::kThreads, 0, st, p);
  if (e != cudaSuccess)
    return fail(KV_ERR_CUDA, "beam selection: %s", cudaGetErrorString(e));
  return KV_OK;
}
