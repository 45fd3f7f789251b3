// Log probabilities of given tokens under softmax(logits), with the entropy and
// the top alternatives, and their gradient.
//
//   forward   m = max x, t_v = (x_v - m) log2 e, e_v = 2^t_v, Z = sum e_v,
//             S = sum e_v t_v:  logp = x_target - m - ln Z,
//             entropy = ln Z - ln 2 S / Z
//   backward  l_v = x_v - m - ln Z, p_v = e^l_v:
//             dx_v = dlogp 1[v = target] - p_v (dlogp + dentropy (l_v + entropy))
//
// The forward reads the logits once: each thread keeps a running maximum and
// rescales its Z and S when it grows, once for 64 bytes at most.  x - m is formed
// before it is scaled, so that neither a mask of the type's lowest value nor
// large logits lose the difference.  Sums are fp32, in pairs, before they are joined
// in a tree: chains of vocab / 256 terms in a block of 128 threads, half of that in one
// of 256, of a block's part in a cluster, and of vocab / 64 (256 at most) where a warp
// takes the row.  (A batch's own sums first, for longer rows: 2 % slower at 8192 x 50257
// and 5 % at the clocks of a long run.)
//
// Bytes: 2 or 4 an element forward, twice that backward; one exponential (16 a clock
// and SM) and about 8 instructions.  32-bit logits and the gradient wait for HBM; the
// forward of 16-bit logits waits for issue slots and the exponential unit (0.72 of
// its rate) before it waits for memory, so that it follows the SM's clock.  A block takes a row, or a warp
// where rows are short; with few rows a cluster of up to 8 blocks shares one and joins
// its parts through distributed shared memory, in one launch without scratch.  In the
// gradient a warp takes a part of a row.
//
// B200, GPU time (share of the bytes at 6535 GB/s): forward with entropy 8192 x 50257
// bf16 136 us in short runs (0.93) and 164 (0.77) in a loop that lasts, where the card
// reaches its power cap and lowers its clock; 1000 x 32000 fp32 24.2 (0.81), with 5
// alternatives 30 (0.65), 2048 x 50257 bf16 40 (0.79), with 20 alternatives 61 (0.51),
// 8192 x 1000 7.7 (0.33: a warp's row is four vectors a lane, and its loads, its join and
// its results follow one another), 8192 x 4000 18.7 (0.54), 5 x 50257 4.3 us, with 20
// alternatives 9.2; gradient 4096 x 50257 bf16 138 us (0.91), in a loop 143, 2048 x 50304
// fp32 132 (0.96), 8192 x 1000 bf16 8.7 (0.58).
//
// Top alternatives: a thread remembers in which vector it saw its maximum.  The
// k-th largest of 64 groups' maxima (as 64-bit keys: value, then lowest index)
// bounds the k-th largest element from below, so only threads whose maximum
// reaches it hold candidates, a few more than k of them as a rule; their
// elements are read again (from L2), and a candidate's place is the number of
// candidates above it.  Keys are distinct: ties fall to the lowest index, and
// the order in which candidates are found does not matter.  (Sorting the threads'
// maxima and merging lists by warps: 82 us instead of 63 at 2048 x 50257.)
//
// Included by libgptlayer.cu after gptlayer.cu, in the same translation unit.
#pragma once

#include <cooperative_groups.h>

#include <type_traits>

#include "gptlayer_parts.h"

namespace gptl {

namespace cg = cooperative_groups;

constexpr int kLpMaxWarps = 8;
constexpr int kLpMaxCluster = 8;
constexpr int kLpNarrow = 5;            // blocks an SM from which on they are narrow
constexpr int kLpWarpVecs = 64, kLpWarpVecsMany = 2048, kLpManyRows = 8;   // rows of a warp
constexpr int kLpBwdVecs = 32, kLpBwdWarps = 64;   // gradient: a lane's vectors, warps of an SM
constexpr int kLpBatch = 4;             // 16-byte loads of a thread in a batch
constexpr int kLpShortBatch = 2;        // the same where a warp takes a short row
constexpr float kLog2e = 1.44269504f, kLn2 = 0.69314718f;

struct LpParams {
  const void *logits;
  const int *target;
  float *logp, *entropy, *stats, *top_logp;
  int *top_id;
  long long ld;
  int rows, vocab, top_k;
  int cluster_log2;                     // blocks of a row
  // backward
  const float *in_stats, *in_entropy, *dlogp, *dentropy;
  void *dlogits;
  int per;                              // vectors of a part
};

// ------------------------------------------------------- 16-byte vectors
template <typename T> struct LpVec {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4 &u, float (&f)[8]) { unpack8<T>(u, f); }
  static __device__ __forceinline__ float to_f(T v) { return Cvt<T>::to_f(v); }
};
template <> struct LpVec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4 &u, float (&f)[4]) {
    f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ float to_f(float v) { return v; }
};
template <typename T> __device__ __forceinline__ uint32_t minus_inf_bits();
template <> __device__ __forceinline__ uint32_t minus_inf_bits<__half>() { return 0xFC00FC00u; }
template <> __device__ __forceinline__ uint32_t minus_inf_bits<__nv_bfloat16>() { return 0xFF80FF80u; }
template <> __device__ __forceinline__ uint32_t minus_inf_bits<float>() { return 0xFF800000u; }

// Largest of a vector's elements (a NaN is passed over; the sum finds it).
template <typename T>
__device__ __forceinline__ float vec_max(const uint4 &u) {
  if constexpr (sizeof(T) == 4) {
    return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)),
                 fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
  } else if constexpr (std::is_same_v<T, __half>) {
    const __half2 *h = reinterpret_cast<const __half2 *>(&u);
    const float2 f = __half22float2(__hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3])));
    return fmaxf(f.x, f.y);
  } else {
    const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&u);
    const float2 f = __bfloat1622float2(__hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3])));
    return fmaxf(f.x, f.y);
  }
}

// A row's 16-byte vectors: `head` elements before the first aligned one,
// `nvec` vectors from `body`, `tail` elements after the last.
template <typename T> struct LpRow {
  const T *row, *body;
  int head, nvec, tail;
  __device__ LpRow(const T *r, int vocab) : row(r) {
    constexpr int N = LpVec<T>::N;
    const int off = (int)((reinterpret_cast<uintptr_t>(r) & 15u) / sizeof(T));
    head = off ? min(N - off, vocab) : 0;
    body = r + head;
    nvec = (vocab - head) / N;
    tail = vocab - head - nvec * N;
  }
  __device__ int tail_index() const { return head + nvec * LpVec<T>::N; }
};

// ------------------------------------------- running maximum and sums
struct LpSum {
  float m, z, s;                        // max, sum 2^t, sum 2^t t (0 terms: -inf, 0, 0)
};

// Brings (z, s) from maximum m to the larger one: t falls by (to - m) log2 e.
// A part without a finite term has z = 0, or NaN, which has to stay.
__device__ __forceinline__ void lp_rescale(LpSum &a, float to) {
  if (a.m == -INFINITY) {
    a.m = to;
    return;
  }
  const float dt = (a.m - to) * kLog2e;
  const float c = ex2_approx(dt);
  a.s = c * fmaf(fmaxf(dt, -200.f), a.z, a.s);
  a.z *= c;
  a.m = to;
}
__device__ __forceinline__ LpSum lp_join(LpSum a, LpSum b) {
  const float m = fmaxf(a.m, b.m);
  lp_rescale(a, m);
  lp_rescale(b, m);
  return LpSum{m, a.z + b.z, a.s + b.s};
}

// Adds one element's term at maximum mr (finite, or +inf).
template <bool ENT>
__device__ __forceinline__ void lp_term(float x, float mr, float &z, float &s) {
  float t = (x - mr) * kLog2e;
  const float e = ex2_approx(t);
  z += e;
  if constexpr (ENT) s = fmaf(e, fmaxf(t, -200.f), s);       // 2^t is 0 there; 0 * -inf is not
}

// The same for two elements at once.
template <bool ENT>
__device__ __forceinline__ void lp_terms(float2 x, float mr, float2 &z, float2 &s) {
  float2 t = mul2(add2(x, make_float2(-mr, -mr)), make_float2(kLog2e, kLog2e));
  const float2 e = make_float2(ex2_approx(t.x), ex2_approx(t.y));
  z = add2(z, e);
  if constexpr (ENT) {
    t.x = fmaxf(t.x, -200.f);
    t.y = fmaxf(t.y, -200.f);
    s = fma2(e, t, s);
  }
}

// ----------------------------------------------------------- sort keys
// Order of (value, lowest index) as one 64-bit number; 0 is below all.
__device__ __forceinline__ unsigned long long lp_key(float x, int index) {
  const int b = __float_as_int(x + 0.0f);                    // -0 counts as 0
  const uint32_t o = (uint32_t)b ^ (uint32_t)((b >> 31) | 0x80000000);
  return ((unsigned long long)o << 32) | (uint32_t)~index;
}
__device__ __forceinline__ float lp_key_value(unsigned long long k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ int lp_key_index(unsigned long long k) { return (int)~(uint32_t)k; }

constexpr int kLpGroups = 64;           // groups of threads whose maxima bound the k-th element
constexpr int kLpHits = 256;            // vectors that may hold candidates
constexpr int kLpCandidates = 1024;     // more than a slice that leaves groups empty has

constexpr int kLpPasses = 8192;
constexpr int kLpMaxTopVocab = 1 << 20;

struct LpTop {
  uint4 hit[kLpHits];
  unsigned long long group[kLpGroups], least;
  unsigned long long candidate[kLpCandidates], best[32];
  int hit_at[kLpHits], hits, found;
};

// Largest of a key over `width` neighbouring lanes (a power of two).
__device__ __forceinline__ unsigned long long key_max(unsigned long long k, int width) {
  for (int o = width / 2; o > 0; o >>= 1) {
    const unsigned long long other = __shfl_xor_sync(0xffffffffu, k, o);
    k = other > k ? other : k;
  }
  return k;
}

// How many of the n keys are above k, counted by `width` neighbouring lanes (a power
// of two) that all call it with the same k; each gets the sum.
__device__ __forceinline__ int key_rank(unsigned long long k, const unsigned long long *keys, int n,
                                        int width, int lane) {
  int above = 0;
  for (int j = lane & (width - 1); j < n; j += width) above += keys[j] > k;
  for (int o = width / 2; o > 0; o >>= 1) above += __shfl_xor_sync(0xffffffffu, above, o);
  return above;
}

// How many of a falling list's first n <= 32 keys are above k.
__device__ __forceinline__ int key_rank_sorted(unsigned long long k, const unsigned long long *list, int n) {
  int above = 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (above + o <= n && list[above + o - 1] > k) above += o;
  return above + (above < n && list[above] > k);
}

// ------------------------------------------------------------- forward
constexpr int kLpNone = -1;             // no vector yet

// WARP: a warp takes a row, for short rows; else a block or a cluster does.
template <typename T, bool ENT, bool TOP, bool WARP>
__global__ void __launch_bounds__(256, WARP ? 5 : 4) logprob_fwd_kernel(const LpParams p) {
  static_assert(!(TOP && WARP), "the alternatives take a block");
  constexpr int N = LpVec<T>::N;
  __shared__ LpSum warp_sum[kLpMaxWarps], rank_sum[kLpMaxCluster];
  __shared__ float final_stats[3];                           // m, ln Z, 1 for NaN, 2 for -inf alone
  __shared__ std::conditional_t<TOP, LpTop, int> top[1];
  __shared__ unsigned long long rank_top[TOP ? kLpMaxCluster * 32 : 1];
  cg::cluster_group cluster = cg::this_cluster();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x / 32;
  const int nt = WARP ? 32 : blockDim.x, tid = WARP ? lane : threadIdx.x;
  const int cs = WARP ? 1 : 1 << p.cluster_log2, rank = blockIdx.x & (cs - 1);
  const long long row = WARP ? (long long)blockIdx.x * nw + warp : blockIdx.x >> p.cluster_log2;
  if (WARP && row >= p.rows) return;
  if (cs > 1) cluster.barrier_arrive();
  const LpRow<T> R(static_cast<const T *>(p.logits) + row * p.ld, p.vocab);
  const uint4 *body = reinterpret_cast<const uint4 *>(R.body);
  const int per = (R.nvec + cs - 1) >> p.cluster_log2;
  const int v_lo = min(per * rank, R.nvec), v_hi = min(v_lo + per, R.nvec);
  const bool has_head = rank == 0 && tid < R.head, has_tail = rank == cs - 1 && tid < R.tail;
  float x_target = 0.f;
  int target = -1;
  if (rank == 0 && tid == 0 && p.target) {
    target = p.target[row];
    if (target >= 0 && target < p.vocab) x_target = LpVec<T>::to_f(R.row[target]);
  }

  // one pass: running maximum, sums, and the first vector that holds the maximum
  // (counted through the thread's vectors)
  LpSum a{-INFINITY, 0.f, 0.f};
  int seen = kLpNone;
  const float x_head = has_head ? LpVec<T>::to_f(R.row[tid]) : 0.f;
  const float x_tail = has_tail ? LpVec<T>::to_f(R.row[R.tail_index() + tid]) : 0.f;
  // full batches of B vectors, each loaded while the one before it is
  // added, then the rest one by one
  constexpr int B = WARP ? kLpShortBatch : kLpBatch;
  int v = v_lo + tid;
  auto add = [&](const auto &u) {
    constexpr int M = sizeof(u) / sizeof(uint4);
    float vm[B], bm = -INFINITY;
#pragma unroll
    for (int i = 0; i < M; ++i) bm = fmaxf(bm, vm[i] = vec_max<T>(u[i]));
    if (bm > a.m || (TOP && a.m == -INFINITY && seen == kLpNone)) {
      if (bm > a.m) lp_rescale(a, bm);
#pragma unroll
      for (int i = M - 1; i >= 0; --i)
        if (vm[i] == bm) seen = v + i * nt;
    }
    const float mr = a.m == -INFINITY ? 0.f : a.m;
    float2 z = make_float2(a.z, 0.f), s = make_float2(a.s, 0.f);
#pragma unroll
    for (int i = 0; i < M; ++i) {
      float f[N];
      LpVec<T>::unpack(u[i], f);
#pragma unroll
      for (int e = 0; e < N; e += 2) lp_terms<ENT>(make_float2(f[e], f[e + 1]), mr, z, s);
    }
    a.z = z.x + z.y;
    a.s = s.x + s.y;
  };
  const int last = v_hi - (B - 1) * nt;               // a batch may start before it
  uint4 next[B];
#pragma unroll
  for (int i = 0; i < B; ++i)
    if (v < last) next[i] = __ldg(body + v + i * nt);
  for (; v < last; v += nt * B) {
    uint4 u[B];
#pragma unroll
    for (int i = 0; i < B; ++i) {
      u[i] = next[i];
      if (v + nt * B < last) next[i] = __ldg(body + v + (B + i) * nt);
    }
    add(u);
  }
  for (; v < v_hi; v += nt) {
    const uint4 u[1] = {__ldg(body + v)};
    add(u);
  }
  const float vector_max = a.m;
  auto one = [&](float x) {
    if (x > a.m) lp_rescale(a, x);
    lp_term<ENT>(x, a.m == -INFINITY ? 0.f : a.m, a.z, a.s);
  };
  if (has_head) one(x_head);
  if (has_tail) one(x_tail);

  // join the block's parts, then the cluster's in its first block
  LpSum t = a;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    t = lp_join(t, LpSum{__shfl_xor_sync(0xffffffffu, t.m, o), __shfl_xor_sync(0xffffffffu, t.z, o),
                         __shfl_xor_sync(0xffffffffu, t.s, o)});
  // the row's results from its sums, by one thread
  auto finish = [&](const LpSum &w) {
    const float nan = __int_as_float(0x7FC00000);
    const bool bad = !(w.z < INFINITY);                    // NaN or +inf among the logits
    const bool empty = w.z == 0.f;                         // -inf alone
    const float lz = bad ? nan : empty ? -INFINITY : logf(w.z);
    if (p.logp) {
      float lp = 0.f;
      if (target >= p.vocab) {
        set_device_error(kErrIndex);
        lp = nan;
      } else if (target >= 0) {
        lp = bad ? nan : empty ? -INFINITY : (x_target - w.m) - lz;
      }
      p.logp[row] = lp;
    }
    if (p.entropy) p.entropy[row] = bad ? nan : empty ? 0.f : lz - kLn2 * (w.s / w.z);
    if (p.stats) {
      p.stats[2 * row] = w.m;
      p.stats[2 * row + 1] = lz;
    }
    if constexpr (TOP) {
      final_stats[0] = w.m;
      final_stats[1] = lz;
      final_stats[2] = bad ? 1.f : empty ? 2.f : 0.f;
    }
  };
  if constexpr (WARP) {
    if (lane == 0) finish(t);
    return;
  }
  if (lane == 0) warp_sum[warp] = t;

  if constexpr (TOP) {
    // `low` is at most the thread's largest key: it takes the last index of the
    // vector that holds the maximum; `high`, with its first index, is at least the
    // largest key of the thread's vectors
    LpTop &S = top[0];
    const unsigned long long kh = has_head ? lp_key(x_head, tid) : 0ull;
    const unsigned long long kt = has_tail ? lp_key(x_tail, R.tail_index() + tid) : 0ull;
    unsigned long long low = kh > kt ? kh : kt, high = 0;
    if (seen != kLpNone) {
      high = lp_key(vector_max, R.head + seen * N);
      const unsigned long long l = lp_key(vector_max, R.head + seen * N + N - 1);
      low = l > low ? l : low;
    }
    // (32 groups for 20 alternatives: fewer ranks to count, more candidates, 67 us
    // instead of 63 at 2048 x 50257)
    const int width = nt / kLpGroups;
    const unsigned long long g = key_max(low, width);
    if (tid % width == 0) S.group[tid / width] = g;
    if (tid == 0) S.found = S.hits = 0;
    if (tid < 32) S.best[tid] = 0;
    // A NaN or +inf in the block's part makes its sum NaN and leaves the row no
    // alternatives; the search would not end well, as a NaN may raise a bound that no
    // number reaches.
    const bool bad_part = __syncthreads_or(!(a.z < INFINITY));
    if (!bad_part) {
      // (empty groups are all 0: the first of equals takes the place)
      const int mine = tid / width;
      const unsigned long long k = S.group[mine];
      int rank = 0;
      for (int j = tid % width; j < kLpGroups; j += width) rank += S.group[j] > k || (S.group[j] == k && j < mine);
      for (int o = width / 2; o > 0; o >>= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
      if (rank == p.top_k - 1) S.least = k;
    }
    __syncthreads();
    for (int pass = 1; !bad_part; ++pass) {
      const unsigned long long least = S.least;
      const float least_value = least ? lp_key_value(least) : -INFINITY;
      auto offer = [&](unsigned long long k) {
        if (k < least || k == 0) return;
        const int at = atomicAdd(&S.found, 1);
        if (at < kLpCandidates) S.candidate[at] = k;
      };
      offer(kh);
      offer(kt);
      // a warp reads the vectors of its threads that may hold candidates, four
      // threads at a time
      for (unsigned todo = __ballot_sync(0xffffffffu, high != 0 && high >= least); todo;) {
        int of[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          of[i] = todo ? __ffs(todo) - 1 : v_hi;
          todo &= todo - 1;
        }
        for (int base = v_lo + warp * 32 + lane * nt; base < v_hi; base += 32 * nt) {
          uint4 u[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (base + of[i] < v_hi) u[i] = __ldg(body + base + of[i]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int at = base + of[i];
            if (at >= v_hi) continue;
            const float vm = vec_max<T>(u[i]);
            if (vm < least_value || lp_key(vm, R.head + at * N) < least) continue;
            const int n = atomicAdd(&S.hits, 1);
            if (n < kLpHits) {
              S.hit[n] = u[i];
              S.hit_at[n] = at;
            }
          }
        }
      }
      __syncthreads();
      // their elements, one a thread
      const int hits = S.hits;
      for (int i = tid; i < min(hits, kLpHits) * N; i += nt) {
        const T x = reinterpret_cast<const T *>(&S.hit[i / N])[i % N];
        offer(lp_key(LpVec<T>::to_f(x), R.head + S.hit_at[i / N] * N + i % N));
      }
      __syncthreads();
      const int found = S.found, kept = min(found, kLpCandidates);
      const bool whole = found <= kLpCandidates && hits <= kLpHits;
      unsigned long long mine = 0;
      const int share = nt / 32;                             // lanes for each candidate
      for (int base = 0; base < kept; base += 32) {
        const int i = base + tid / share;
        const unsigned long long k = i < kept ? S.candidate[i] : ~0ull;
        const int rank = key_rank(k, S.candidate, kept, share, lane);
        if (i >= kept || tid % share) continue;
        if (whole) {
          if (rank < p.top_k) S.best[rank] = k;
        } else if (rank == p.top_k - 1) {
          mine = k;
        }
      }
      __syncthreads();
      if (whole) break;
      // More than were kept: the k-th of those kept is a sharper bound (of kLpHits
      // vectors all but one hold a candidate, so there is a k-th).  It leaves over 200
      // fewer each time, so 2^20 elements end long before the limit.
      if (pass == kLpPasses) {
        if (tid == 0) set_device_error(kErrIndex);
        break;
      }
      if (mine) S.least = mine;
      if (tid == 0) S.found = S.hits = 0;
      __syncthreads();
    }
  } else {
    __syncthreads();
  }

  if (cs > 1) {
    cluster.barrier_wait();                                  // every block has started
    if (warp == 0) {
      LpSum w = lane < nw ? warp_sum[lane] : LpSum{-INFINITY, 0.f, 0.f};
#pragma unroll
      for (int o = 8; o > 0; o >>= 1)
        w = lp_join(w, LpSum{__shfl_xor_sync(0xffffffffu, w.m, o), __shfl_xor_sync(0xffffffffu, w.z, o),
                             __shfl_xor_sync(0xffffffffu, w.s, o)});
      if (lane == 0) *cluster.map_shared_rank(&rank_sum[rank], 0) = w;
      if constexpr (TOP)
        if (lane < p.top_k)
          *cluster.map_shared_rank(&rank_top[rank * p.top_k + lane], 0) = top[0].best[lane];
    }
    cluster.sync();
    if (rank != 0) return;
  }
  if (warp == 0) {
    const int parts = cs > 1 ? cs : nw;
    LpSum w{-INFINITY, 0.f, 0.f};
    if (lane < parts) w = cs > 1 ? rank_sum[lane] : warp_sum[lane];
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
      w = lp_join(w, LpSum{__shfl_xor_sync(0xffffffffu, w.m, o), __shfl_xor_sync(0xffffffffu, w.z, o),
                           __shfl_xor_sync(0xffffffffu, w.s, o)});
    if (lane == 0) finish(w);
  }
  if constexpr (TOP) {
    __syncthreads();
    const float kind = final_stats[2];
    auto put = [&](int place, float lp, int id) {
      p.top_logp[row * p.top_k + place] = lp;
      p.top_id[row * p.top_k + place] = id;
    };
    if (kind == 1.f) {                                       // a bad part left no keys to rank
      if (tid < p.top_k) put(tid, __int_as_float(0x7FC00000), -1);
      return;
    }
    auto put_key = [&](int place, unsigned long long k) {
      put(place, kind == 2.f ? -INFINITY : (lp_key_value(k) - final_stats[0]) - final_stats[1], lp_key_index(k));
    };
    if (cs == 1) {
      if (tid < p.top_k) put_key(tid, top[0].best[tid]);
    } else {
      for (int i = tid; i < cs * p.top_k; i += nt) {
        const unsigned long long k = rank_top[i];
        int place = 0;
#pragma unroll
        for (int r = 0; r < kLpMaxCluster; ++r)
          if (r < cs) place += key_rank_sorted(k, rank_top + r * p.top_k, p.top_k);
        if (place < p.top_k) put_key(place, k);
      }
    }
  }
}

// ------------------------------------------------------------ backward
template <typename T>
__device__ __forceinline__ uint4 lp_pack(const float (&f)[LpVec<T>::N]) {
  if constexpr (sizeof(T) == 4)
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  else
    return pack8<T>(f);
}

// A warp takes a part of a row, in batches of B vectors a lane.
template <typename T, int B>
__global__ void __launch_bounds__(256) logprob_bwd_kernel(const LpParams p) {
  constexpr int N = LpVec<T>::N;
  const int nt = 32, tid = threadIdx.x & 31, part = blockIdx.y;
  const long long row = (long long)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
  if (row >= p.rows) return;
  const LpRow<T> R(static_cast<const T *>(p.logits) + row * p.ld, p.vocab);
  T *out = static_cast<T *>(p.dlogits) + row * p.ld;         // the same offset from 16 bytes
  const uint4 *src = reinterpret_cast<const uint4 *>(R.body);
  uint4 *dst = reinterpret_cast<uint4 *>(out + R.head);
  const int v_lo = min(part * p.per, R.nvec), v_hi = min(v_lo + p.per, R.nvec);

  // the first vectors go out before the row's gradients are known, and each
  // batch before the one ahead of it is computed
  uint4 next[B];
  auto fetch = [&](int v) {
#pragma unroll
    for (int i = 0; i < B; ++i)
      if (v + i * nt < v_hi) next[i] = src[v + i * nt];
  };
  fetch(v_lo + tid);
  int target = p.target ? __ldg(p.target + row) : -1;
  if (target >= p.vocab) {
    if (part == 0 && tid == 0) set_device_error(kErrIndex);
    target = -1;
  }
  float up = p.dlogp && target >= 0 ? __ldg(p.dlogp + row) : 0.f;
  const float de = p.dentropy ? __ldg(p.dentropy + row) : 0.f;
  const float m = __ldg(p.in_stats + 2 * row), lz = __ldg(p.in_stats + 2 * row + 1);
  const bool empty = lz == -INFINITY;                        // -inf alone: no gradient
  const bool head = part == 0 && tid < R.head, tail = part == (int)gridDim.y - 1 && tid < R.tail;
  if ((up == 0.f && de == 0.f) || empty) {
    if (head) out[tid] = T(0.f);
    for (int v = v_lo + tid; v < v_hi; v += nt) dst[v] = make_uint4(0, 0, 0, 0);
    if (tail) out[R.tail_index() + tid] = T(0.f);
    return;
  }
  // dx = -p (c1 + de l), c1 = up + de entropy; l is held above -1e4, where p is
  // 0 all the same, so that -inf does not meet 0.  Rows with NaN have a NaN lz.
  float c1 = p.dentropy ? fmaf(de, __ldg(p.in_entropy + row), up) : up;
  if (lz != lz) c1 = lz;
  auto grad = [&](float2 x) {
    float2 l = add2(add2(x, make_float2(-m, -m)), make_float2(-lz, -lz));
    l.x = fmaxf(l.x, -1e4f);
    l.y = fmaxf(l.y, -1e4f);
    const float2 t = mul2(l, make_float2(kLog2e, kLog2e));
    return mul2(make_float2(ex2_approx(t.x), ex2_approx(t.y)),
                fma2(make_float2(-de, -de), l, make_float2(-c1, -c1)));
  };
  auto scalar = [&](int i) {
    const float x = LpVec<T>::to_f(R.row[i]);
    const float g = grad(make_float2(x, x)).x + (i == target ? up : 0.f);
    if constexpr (sizeof(T) == 4) out[i] = g;
    else out[i] = Cvt<T>::from_f(g);
  };
  if (head) scalar(tid);
  const int tv = target >= R.head ? (target - R.head) / N : -1;     // the target's vector
  for (int v = v_lo + tid; v < v_hi; v += nt * B) {
    uint4 u[B];
#pragma unroll
    for (int i = 0; i < B; ++i) u[i] = next[i];
    fetch(v + nt * B);
#pragma unroll
    for (int i = 0; i < B; ++i) {
      if (v + i * nt >= v_hi) break;
      float f[N];
      LpVec<T>::unpack(u[i], f);
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        const float2 g = grad(make_float2(f[e], f[e + 1]));
        f[e] = g.x;
        f[e + 1] = g.y;
      }
      if (v + i * nt == tv) {
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (R.head + tv * N + e == target) f[e] += up;
      }
      dst[v + i * nt] = lp_pack<T>(f);
    }
  }
  if (tail) scalar(R.tail_index() + tid);
}

}  // namespace gptl

namespace {

int check_lp(int rows, int vocab, long long ld, gptl_dtype dt, int f32, const void *logits,
             const int *target, LpParams *p) {
  if (dt != GPTL_FP16 && dt != GPTL_BF16) return GPTL_E_DTYPE;
  if (f32 != 0 && f32 != 1) return GPTL_E_ARG;
  if (rows < 1 || vocab < 1 || vocab >= (1 << 30) || ld < vocab || ld >= (1ll << 40) ||
      !far_rows(rows, ld))
    return GPTL_E_SHAPE;
  if (!aligned16(logits) || (reinterpret_cast<uintptr_t>(target) & 3u)) return GPTL_E_ALIGN;
  p->logits = logits;
  p->target = target;
  p->ld = ld;
  p->rows = rows;
  p->vocab = vocab;
  return GPTL_OK;
}

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

template <typename T>
int launch_lp_fwd(const LpParams &p, bool warp_rows, unsigned grid, int threads, cudaStream_t st) {
  auto kern = p.top_k ? (p.entropy ? logprob_fwd_kernel<T, true, true, false>
                                   : logprob_fwd_kernel<T, false, true, false>)
              : warp_rows ? (p.entropy ? logprob_fwd_kernel<T, true, false, true>
                                       : logprob_fwd_kernel<T, false, false, true>)
                          : (p.entropy ? logprob_fwd_kernel<T, true, false, false>
                                       : logprob_fwd_kernel<T, false, false, false>);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 1u << p.cluster_log2;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = p.cluster_log2 > 0 ? 1 : 0;
  GPTL_CK(cudaLaunchKernelEx(&cfg, kern, p));
  return GPTL_OK;
}

}  // namespace

extern "C" {

int gptl_token_logprob_fwd(int rows, int vocab, long long ld, gptl_dtype dtype, int logits_f32,
                           const void *logits, const int *target, float *logp, float *entropy,
                           float *stats, int top_k, float *top_logp, int *top_id,
                           gptl_stream_t stream) {
  if (!logits || (target == nullptr) != (logp == nullptr)) return GPTL_E_NULL;
  if (!logp && !entropy && !stats && top_k == 0) return GPTL_E_NULL;
  LpParams p{};
  GPTL_TRY(check_lp(rows, vocab, ld, dtype, logits_f32, logits, target, &p));
  if (top_k < 0 || top_k > 32 || top_k > vocab) return GPTL_E_ARG;
  if (top_k && vocab > kLpMaxTopVocab) return GPTL_E_SHAPE;
  if (top_k && (!top_logp || !top_id)) return GPTL_E_NULL;
  if (!aligned4(logp) || !aligned4(entropy) || !aligned4(stats) || !aligned4(top_logp) ||
      !aligned4(top_id))
    return GPTL_E_ALIGN;
  int sms = 0;
  GPTL_TRY(device_check(&sms));
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  p.logp = logp;
  p.entropy = entropy;
  p.stats = stats;
  p.top_k = top_k;
  p.top_logp = top_logp;
  p.top_id = top_id;
  // Short rows go to a warp each: up to 64 vectors always (100 x 500 bf16: 2.4 us
  // against a block's 2.7; 100 x 2000: 3.1 against 2.8), up to 2048 once there are
  // warps enough for every SM (8192 x 4000: 19 against 33; 8192 x 16000: 55 against
  // 58; 600 x 2000: 3.7 against 3.4).  The alternatives need a block's shared memory.
  const int vecs = vocab / (logits_f32 ? 4 : 8);
  const bool warp_rows =
      top_k == 0 && (vecs <= kLpWarpVecs || (vecs <= kLpWarpVecsMany && rows >= kLpManyRows * sms));
  // Else a row's blocks: 1 once the rows fill the SMs, up to 8 of at least 2048
  // elements each before (64 x 128000: 4 blocks 6.9 us, 8 blocks 7.7; going on to
  // 8 blocks an SM, 1000 x 32000 fp32 takes 29 us instead of 26).
  int cs = 1;
  while (!warp_rows && cs < kLpMaxCluster && (long long)rows * cs < sms && vocab / (2 * cs) >= 2048) {
    cs *= 2;
    ++p.cluster_log2;
  }
  // 256 threads a block while blocks are few (300 x 128000: 25 us, with 128 35), 128
  // once they fill the SMs, which wait less at the end of a row (8192 x 50257: 156
  // and 147 us before the loads were overlapped, 1000 x 32000 fp32 with 5
  // alternatives 33 and 30).
  const long long blocks = (long long)rows * cs;
  const int threads = !warp_rows && vecs / cs >= 256 && blocks < kLpNarrow * sms ? 256 : 128;
  if (blocks >= (1ll << 31)) return GPTL_E_SHAPE;
  const unsigned grid = warp_rows ? (unsigned)((rows + 3ll) / 4) : (unsigned)blocks;
  prof_start(st);
  if (logits_f32) GPTL_TRY(launch_lp_fwd<float>(p, warp_rows, grid, threads, st));
  else if (dtype == GPTL_FP16) GPTL_TRY(launch_lp_fwd<__half>(p, warp_rows, grid, threads, st));
  else GPTL_TRY(launch_lp_fwd<__nv_bfloat16>(p, warp_rows, grid, threads, st));
  prof_launched(st, GPTL_KIND_LOGPROB_FWD);
  return GPTL_OK;
}

int gptl_token_logprob_bwd(int rows, int vocab, long long ld, gptl_dtype dtype, int logits_f32,
                           const void *logits, const int *target, const float *stats,
                           const float *entropy, const float *dlogp, const float *dentropy,
                           void *dlogits, gptl_stream_t stream) {
  if (!logits || !stats || !dlogits || (!dlogp && !dentropy) || (dlogp && !target) ||
      (dentropy && !entropy))
    return GPTL_E_NULL;
  LpParams p{};
  GPTL_TRY(check_lp(rows, vocab, ld, dtype, logits_f32, logits, target, &p));
  if (!aligned16(dlogits) || !aligned4(stats) || !aligned4(entropy) || !aligned4(dlogp) ||
      !aligned4(dentropy))
    return GPTL_E_ALIGN;
  const long long es = logits_f32 ? 4 : 2;
  if (dlogits != logits && rows_overlap(logits, dlogits, RowsShape{1, 0, rows, es * ld, es * vocab}))
    return GPTL_E_ARG;
  int sms = 0;
  GPTL_TRY(device_check(&sms));
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  p.in_stats = stats;
  p.in_entropy = entropy;
  p.dlogp = dlogp;
  p.dentropy = dentropy;
  p.dlogits = dlogits;
  // A warp's part of a row: as long as leaves kLpBwdWarps warps an SM, so that the
  // row's scalars and the first loads are small beside it (4096 x 50257 with one
  // batch a thread 168 us, with 32 vectors 137), but at most kLpBwdVecs vectors a
  // lane, and one batch at least.
  const int vecs = vocab / (logits_f32 ? 4 : 8) + 1;
  long long lane_vecs = (long long)rows * vecs / (32ll * kLpBwdWarps * sms);
  if (lane_vecs > kLpBwdVecs) lane_vecs = kLpBwdVecs;
  if (lane_vecs < kLpBatch) lane_vecs = kLpBatch;
  int parts = (int)((vecs + 32 * lane_vecs - 1) / (32 * lane_vecs));
  if (parts > 65535) parts = 65535;
  p.per = (vecs + parts - 1) / parts;
  const dim3 grid((unsigned)((rows + 7ll) / 8), parts);
  prof_start(st);
  auto go = [&]<typename T>() {
    if (p.per <= 32 * 2 * kLpBatch) logprob_bwd_kernel<T, kLpShortBatch><<<grid, 256, 0, st>>>(p);
    else logprob_bwd_kernel<T, kLpBatch><<<grid, 256, 0, st>>>(p);
  };
  if (logits_f32) go.template operator()<float>();
  else if (dtype == GPTL_FP16) go.template operator()<__half>();
  else go.template operator()<__nv_bfloat16>();
  GPTL_CK(cudaGetLastError());
  prof_launched(st, GPTL_KIND_LOGPROB_BWD);
  return GPTL_OK;
}

}  // extern "C"
