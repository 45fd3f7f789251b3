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
// large logits lose the difference.  Sums are fp32, each of at most a few
// hundred terms before they are joined in a tree.
//
// Bound by HBM (2 or 4 bytes an element forward, twice that backward), with
// one exponential an element close behind (16 a clock and SM).  A block takes
// a row; with few rows a cluster of up to 8 blocks shares it and joins its
// parts through distributed shared memory, in one launch without scratch.
//
// Top alternatives: a thread remembers where it saw its maximum.  The k-th
// largest of the threads' maxima (as 64-bit keys: value, then lowest index)
// bounds the k-th largest element from below, so only threads whose maximum
// reaches it hold candidates; a warp reads those threads' elements again (from
// L2) and keeps its best 32 sorted in its lanes.  No list can overflow, and ties
// fall to the lowest index by the key's order.
//
// Included by libgptlayer.cu after gptlayer.cu, in the same translation unit.
#pragma once

#include <cooperative_groups.h>

#include "gptlayer_parts.h"

namespace gptl {

namespace cg = cooperative_groups;

constexpr int kLpMaxWarps = 16;
constexpr int kLpMaxCluster = 8;
constexpr int kLpBatch = 4;             // 16-byte loads of a thread in flight
constexpr float kLog2e = 1.44269504f, kLn2 = 0.69314718f;

struct LpParams {
  const void *logits;
  const int *target;
  float *logp, *entropy, *stats, *top_logp;
  int *top_id;
  long long ld;
  int rows, vocab, top_k, cluster;
  // backward
  const float *in_stats, *in_entropy, *dlogp, *dentropy;
  void *dlogits;
  int parts;                            // blocks of a row
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

__device__ __forceinline__ unsigned long long key_step(unsigned long long k, int lane, int o, bool up) {
  const unsigned long long other = __shfl_xor_sync(0xffffffffu, k, o);
  const bool keep_max = ((lane & o) == 0) != up;
  return keep_max == (k > other) ? k : other;
}
// Sorts one key a lane, falling.
__device__ __forceinline__ unsigned long long warp_sort(unsigned long long k, int lane) {
#pragma unroll
  for (int n = 2; n <= 32; n *= 2)
#pragma unroll
    for (int o = n / 2; o > 0; o /= 2) k = key_step(k, lane, o, (lane & n) != 0 && n < 32);
  return k;
}
// The 32 largest of two falling lists, falling; `b` comes reversed.
__device__ __forceinline__ unsigned long long warp_merge(unsigned long long a,
                                                         unsigned long long b_reversed, int lane) {
  unsigned long long k = a > b_reversed ? a : b_reversed;
#pragma unroll
  for (int o = 16; o > 0; o /= 2) k = key_step(k, lane, o, false);
  return k;
}
// lists[0] becomes the 32 largest of n falling lists (n a power of two, at most
// twice the block's warps).  Every thread of the block calls it.
__device__ __forceinline__ void block_merge(unsigned long long (*lists)[32], int n, int warp,
                                            int lane) {
  for (int s = n / 2; s > 0; s /= 2) {
    __syncthreads();
    if (warp < s) {
      const unsigned long long k = warp_merge(lists[warp][lane], lists[warp + s][31 - lane], lane);
      lists[warp][lane] = k;
    }
  }
  __syncthreads();
}

// The running best 32 of a warp: `best` falls over the lanes, `buf` holds up to
// 63 keys that have not been sorted in yet.
struct WarpTop {
  unsigned long long best, *buf;
  int n;
  __device__ void flush(int lane) {
    __syncwarp();
    unsigned long long k = lane < n ? buf[lane] : 0ull;
    unsigned long long rest = 32 + lane < n ? buf[32 + lane] : 0ull;
    __syncwarp();
    k = warp_sort(k, lane);
    best = warp_merge(best, __shfl_sync(0xffffffffu, k, 31 - lane), lane);
    n = n > 32 ? n - 32 : 0;
    if (lane < n) buf[lane] = rest;
    __syncwarp();
  }
  __device__ void add(unsigned long long k, bool take, int lane) {
    const unsigned mask = __ballot_sync(0xffffffffu, take);
    if (!mask) return;
    if (take) buf[n + __popc(mask & ((1u << lane) - 1))] = k;
    n += __popc(mask);
    if (n >= 32) flush(lane);
  }
};

// ------------------------------------------------------------- forward
enum : int { kLpNone = -3, kLpHead = -2, kLpTail = -1 };

template <typename T, bool ENT, bool TOP>
__global__ void __launch_bounds__(512) logprob_fwd_kernel(const LpParams p) {
  constexpr int N = LpVec<T>::N;
  __shared__ LpSum warp_sum[kLpMaxWarps], rank_sum[kLpMaxCluster];
  __shared__ float final_stats[3];                           // m, ln Z, 1 if the row is bad
  __shared__ unsigned long long lists[TOP ? kLpMaxWarps : 1][32];
  __shared__ unsigned long long rank_top[TOP ? kLpMaxCluster : 1][32];
  __shared__ unsigned long long bufs[TOP ? kLpMaxWarps : 1][64];
  cg::cluster_group cluster = cg::this_cluster();
  const int nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = nt / 32;
  const int cs = p.cluster, rank = cs > 1 ? blockIdx.x % cs : 0;
  const long long row = blockIdx.x / cs;
  if (cs > 1) cluster.barrier_arrive();
  const LpRow<T> R(static_cast<const T *>(p.logits) + row * p.ld, p.vocab);
  const uint4 *body = reinterpret_cast<const uint4 *>(R.body);
  const int v_lo = (int)((long long)R.nvec * rank / cs);
  const int v_hi = (int)((long long)R.nvec * (rank + 1) / cs);
  const bool has_head = rank == 0 && tid < R.head, has_tail = rank == cs - 1 && tid < R.tail;
  float x_target = 0.f;
  int target = -1;
  if (rank == 0 && tid == 0 && p.target) {
    target = p.target[row];
    if (target >= 0 && target < p.vocab) x_target = LpVec<T>::to_f(R.row[target]);
  }

  // one pass: running maximum, sums, and where the maximum was first seen
  LpSum a{-INFINITY, 0.f, 0.f};
  int seen = kLpNone;
  auto one = [&](float x, int where) {
    if (seen == kLpNone) seen = where;
    if (x > a.m) {
      lp_rescale(a, x);
      seen = where;
    }
    lp_term<ENT>(x, a.m == -INFINITY ? 0.f : a.m, a.z, a.s);
  };
  if (has_head) one(LpVec<T>::to_f(R.row[tid]), kLpHead);
  if (TOP && seen == kLpNone && v_lo + tid < v_hi) seen = 0;
  int batch = 0;
  for (int v = v_lo + tid; v < v_hi; v += nt * kLpBatch, ++batch) {
    uint4 u[kLpBatch];
    const uint32_t fill = minus_inf_bits<T>();
#pragma unroll
    for (int i = 0; i < kLpBatch; ++i) {
      u[i] = make_uint4(fill, fill, fill, fill);
      if (v + i * nt < v_hi) u[i] = __ldg(body + v + i * nt);
    }
    float bm = vec_max<T>(u[0]);
#pragma unroll
    for (int i = 1; i < kLpBatch; ++i) bm = fmaxf(bm, vec_max<T>(u[i]));
    if (bm > a.m) {
      lp_rescale(a, bm);
      seen = batch;
    }
    const float mr = a.m == -INFINITY ? 0.f : a.m;
#pragma unroll
    for (int i = 0; i < kLpBatch; ++i) {
      float f[N];
      LpVec<T>::unpack(u[i], f);
#pragma unroll
      for (int e = 0; e < N; ++e) lp_term<ENT>(f[e], mr, a.z, a.s);
    }
  }
  if (has_tail) one(LpVec<T>::to_f(R.row[R.tail_index() + tid]), kLpTail);

  // join the block's parts, then the cluster's in its first block
  LpSum t = a;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    t = lp_join(t, LpSum{__shfl_xor_sync(0xffffffffu, t.m, o), __shfl_xor_sync(0xffffffffu, t.z, o),
                         __shfl_xor_sync(0xffffffffu, t.s, o)});
  if (lane == 0) warp_sum[warp] = t;

  if constexpr (TOP) {
    // this thread's largest element, found again where it was seen
    unsigned long long mine = 0;
    if (seen == kLpHead) {
      mine = lp_key(LpVec<T>::to_f(R.row[tid]), tid);
    } else if (seen == kLpTail) {
      mine = lp_key(LpVec<T>::to_f(R.row[R.tail_index() + tid]), R.tail_index() + tid);
    } else if (seen >= 0) {
      const int v0 = v_lo + tid + seen * nt * kLpBatch;
#pragma unroll
      for (int i = 0; i < kLpBatch; ++i) {
        const int v = v0 + i * nt;
        if (v >= v_hi) break;
        float f[N];
        LpVec<T>::unpack(__ldg(body + v), f);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const unsigned long long k = lp_key(f[e], R.head + v * N + e);
          mine = k > mine ? k : mine;
        }
      }
    }
    lists[warp][lane] = warp_sort(mine, lane);
    block_merge(lists, nw, warp, lane);
    const unsigned long long least = lists[0][p.top_k - 1];
    __syncthreads();
    WarpTop top{0ull, bufs[warp], 0};
    {
      unsigned long long k = has_head ? lp_key(LpVec<T>::to_f(R.row[tid]), tid) : 0ull;
      top.add(k, k != 0 && k >= least, lane);
      k = has_tail ? lp_key(LpVec<T>::to_f(R.row[R.tail_index() + tid]), R.tail_index() + tid) : 0ull;
      top.add(k, k != 0 && k >= least, lane);
    }
    for (unsigned todo = __ballot_sync(0xffffffffu, mine != 0 && mine >= least); todo;
         todo &= todo - 1) {
      const int v0 = v_lo + warp * 32 + __ffs(todo) - 1;     // the first vector of that thread
      for (int base = v0; base < v_hi; base += 32 * nt) {
        const int v = base + lane * nt;
        float f[N];
        if (v < v_hi) LpVec<T>::unpack(__ldg(body + v), f);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const unsigned long long k = v < v_hi ? lp_key(f[e], R.head + v * N + e) : 0ull;
          top.add(k, k != 0 && k >= least, lane);
        }
      }
    }
    if (top.n) top.flush(lane);
    lists[warp][lane] = top.best;
    block_merge(lists, nw, warp, lane);
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
      if constexpr (TOP) *cluster.map_shared_rank(&rank_top[rank][lane], 0) = lists[0][lane];
    }
    cluster.sync();
    if (rank != 0) return;
    if constexpr (TOP) block_merge(rank_top, cs, warp, lane);
  }
  if (warp != 0) return;
  const int parts = cs > 1 ? cs : nw;
  LpSum w{-INFINITY, 0.f, 0.f};
  if (lane < parts) w = cs > 1 ? rank_sum[lane] : warp_sum[lane];
#pragma unroll
  for (int o = 8; o > 0; o >>= 1)
    w = lp_join(w, LpSum{__shfl_xor_sync(0xffffffffu, w.m, o), __shfl_xor_sync(0xffffffffu, w.z, o),
                         __shfl_xor_sync(0xffffffffu, w.s, o)});
  if (lane == 0) {
    const float nan = __int_as_float(0x7FC00000);
    const bool bad = !(w.z < INFINITY);                      // NaN or +inf among the logits
    const bool empty = w.z == 0.f;                           // -inf alone
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
    final_stats[0] = w.m;
    final_stats[1] = lz;
    final_stats[2] = bad ? 1.f : empty ? 2.f : 0.f;
  }
  if constexpr (TOP) {
    __syncwarp();
    if (lane < p.top_k) {
      const unsigned long long k = cs > 1 ? rank_top[0][lane] : lists[0][lane];
      const float kind = final_stats[2];
      const float lp = kind == 1.f   ? __int_as_float(0x7FC00000)
                       : kind == 2.f ? -INFINITY
                                     : (lp_key_value(k) - final_stats[0]) - final_stats[1];
      p.top_logp[row * p.top_k + lane] = lp;
      p.top_id[row * p.top_k + lane] = kind == 1.f ? -1 : lp_key_index(k);
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

template <typename T>
__global__ void __launch_bounds__(256) logprob_bwd_kernel(const LpParams p) {
  constexpr int N = LpVec<T>::N;
  const long long row = blockIdx.x / p.parts;
  const int part = (int)(blockIdx.x % p.parts), tid = threadIdx.x, nt = blockDim.x;
  const LpRow<T> R(static_cast<const T *>(p.logits) + row * p.ld, p.vocab);
  T *out = static_cast<T *>(p.dlogits) + row * p.ld;         // the same offset from 16 bytes
  const uint4 *src = reinterpret_cast<const uint4 *>(R.body);
  uint4 *dst = reinterpret_cast<uint4 *>(out + R.head);
  const int v_lo = (int)((long long)R.nvec * part / p.parts);
  const int v_hi = (int)((long long)R.nvec * (part + 1) / p.parts);

  int target = p.target ? __ldg(p.target + row) : -1;
  if (target >= p.vocab) {
    if (part == 0 && tid == 0) set_device_error(kErrIndex);
    target = -1;
  }
  float up = p.dlogp && target >= 0 ? __ldg(p.dlogp + row) : 0.f;
  const float de = p.dentropy ? __ldg(p.dentropy + row) : 0.f;
  const float m = __ldg(p.in_stats + 2 * row), lz = __ldg(p.in_stats + 2 * row + 1);
  const bool empty = lz == -INFINITY;                        // -inf alone: no gradient
  const bool head = part == 0 && tid < R.head, tail = part == p.parts - 1 && tid < R.tail;
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
  auto grad = [&](float x) {
    const float l = fmaxf((x - m) - lz, -1e4f);
    return -ex2_approx(l * kLog2e) * fmaf(de, l, c1);
  };
  auto scalar = [&](int i) {
    const float g = grad(LpVec<T>::to_f(R.row[i])) + (i == target ? up : 0.f);
    if constexpr (sizeof(T) == 4) out[i] = g;
    else out[i] = Cvt<T>::from_f(g);
  };
  if (head) scalar(tid);
  const int tv = target >= R.head ? (target - R.head) / N : -1;     // the target's vector
  for (int v = v_lo + tid; v < v_hi; v += nt * kLpBatch) {
    uint4 u[kLpBatch];
#pragma unroll
    for (int i = 0; i < kLpBatch; ++i)
      if (v + i * nt < v_hi) u[i] = src[v + i * nt];
#pragma unroll
    for (int i = 0; i < kLpBatch; ++i) {
      if (v + i * nt >= v_hi) break;
      float f[N];
      LpVec<T>::unpack(u[i], f);
#pragma unroll
      for (int e = 0; e < N; ++e) f[e] = grad(f[e]);
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
  if (rows < 1 || vocab < 1 || vocab >= (1 << 30) || ld < vocab || ld >= (1ll << 40))
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
int launch_lp_fwd(const LpParams &p, unsigned grid, int threads, cudaStream_t st) {
  auto kern = p.top_k ? (p.entropy ? logprob_fwd_kernel<T, true, true>
                                   : logprob_fwd_kernel<T, false, true>)
                      : (p.entropy ? logprob_fwd_kernel<T, true, false>
                                   : logprob_fwd_kernel<T, false, false>);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)p.cluster;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = p.cluster > 1 ? 1 : 0;
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
  // A row's blocks: 1 once the rows fill the SMs, else up to 8 of at least
  // 2048 elements each.
  int cs = 1;
  while (cs < kLpMaxCluster && (long long)rows * cs * 2 <= 2ll * sms && vocab / (2 * cs) >= 2048)
    cs *= 2;
  p.cluster = cs;
  const int per_vec = logits_f32 ? 4 : 8;
  const int vecs = vocab / per_vec / cs;
  const int threads = vecs >= 1024 ? 512 : vecs >= 256 ? 256 : 128;
  if ((long long)rows * cs >= (1ll << 31)) return GPTL_E_SHAPE;
  const unsigned grid = (unsigned)rows * (unsigned)cs;
  prof_start(st);
  if (logits_f32) GPTL_TRY(launch_lp_fwd<float>(p, grid, threads, st));
  else if (dtype == GPTL_FP16) GPTL_TRY(launch_lp_fwd<__half>(p, grid, threads, st));
  else GPTL_TRY(launch_lp_fwd<__nv_bfloat16>(p, grid, threads, st));
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
  const long long bytes = ((rows - 1) * ld + vocab) * (logits_f32 ? 4 : 2);
  if (dlogits != logits && ranges_overlap(logits, bytes, dlogits, bytes)) return GPTL_E_ARG;
  GPTL_TRY(device_check());
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  p.in_stats = stats;
  p.in_entropy = entropy;
  p.dlogp = dlogp;
  p.dentropy = dentropy;
  p.dlogits = dlogits;
  const int vecs = vocab / (logits_f32 ? 4 : 8);
  p.parts = (vecs + 256 * kLpBatch - 1) / (256 * kLpBatch);
  if (p.parts < 1) p.parts = 1;
  if ((long long)rows * p.parts >= (1ll << 31)) return GPTL_E_SHAPE;
  const unsigned grid = (unsigned)((long long)rows * p.parts);
  prof_start(st);
  if (logits_f32) logprob_bwd_kernel<float><<<grid, 256, 0, st>>>(p);
  else if (dtype == GPTL_FP16) logprob_bwd_kernel<__half><<<grid, 256, 0, st>>>(p);
  else logprob_bwd_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(p);
  GPTL_CK(cudaGetLastError());
  prof_launched(st, GPTL_KIND_LOGPROB_BWD);
  return GPTL_OK;
}

}  // extern "C"
