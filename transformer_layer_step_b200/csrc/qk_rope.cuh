// Norm and rotation of queries and keys, forward and backward, on the packed
// [Q | K | V] rows between the QKV product and attention.
//
// With x one head of one token, g its gain and r = 1 / sqrt(mean(x^2) + eps):
//   forward   n = x r g, then each pair (a, b) of n turns by phi;
//   backward  dn = dy turned back by phi, d = dn g,
//             dx = r d - x r^3 mean(d x),   dg = sum dn x r,
// where mean(x^2) and mean(d x) are summed together, so a head needs one
// reduction.  phi in turns is pos * turns_j modulo 1, taken in 64-bit integers, since
// fp32 has lost the fraction of far positions; its sine and cosine are fp32.
//
// Bytes: 4 an element forward, 6 backward (value heads 4), against about 6 and 9
// instructions an element, so that HBM and issue are close.  A warp takes a run of a
// token's heads: its lanes compute the token's rot_dim/2 sines and cosines once, into
// shared memory, and use them for every head.  A lane owns 16 elements of a head, two
// 16-byte vectors chosen so that it holds both elements of each of its 8 pairs:
// rotation needs no exchange, and the norm log2(lanes) shuffles.  Gains and angles
// stay in shared memory, in the lanes' order; the next heads' vectors are loaded while
// these are worked on.
//
// B200, GPU time (share of the bytes at 6535 GB/s): forward 8192 tokens x 4 groups x
// (4 + 4 + 4) heads of 64 fp16 21.2 us (0.73; in place 17.1), 2048 x 4 x (20 + 20) of 128
// bf16 32.0 (0.80); backward with gains 2048 x 4 x (20 + 20) of 128 49.3 (0.78), 5003 x
// (32 + 8 + 8) of 80 33.0 (0.50), of 64 21.9 (0.54); 16 tokens x (32 + 8) of 128 3.5 us, a
// launch's time.  Rotation alone: the same forwards 19.9 (0.77; in place 15.3) and 31.5
// (0.82), backward 31.7 (0.81) and 5003 tokens of 80 19.3 (0.61).
// What bounds it is latency.  The next slot is fetched ahead only within a token: a
// token's first loads, its positions and its angles follow one another, every 20 slots
// at (20 + 20) heads of 128, but every 2 at 8192 x 4 x 4 and every 6 (queries) and 2 (keys)
// at 32 + 8 of 80, where the eight key heads also fill only 8 of 12 places.  The
// backward with gains has 128 registers, which allow 16 warps an SM to hide that; issue
// is half used.  Tried and slower there: rings of asynchronous copies (58 us at
// 10240), bulk copies of tiles into shared memory (63), three blocks an SM (92, spills),
// forming dn x twice to save registers (51).  What is kept spills little: 4 to 8 bytes
// with gains at 5, 6, 9 and 10 lanes backward, 4 bytes forward at a power of two.
//
// Included by libgptlayer.cu after gptlayer.cu, in the same translation unit.
#pragma once

#include <utility>

#include "gptlayer_parts.h"

namespace gptl {

constexpr int kQkWarps = 8;             // warps of a block
constexpr int kQkMaxBlocks = 592;       // partial rows of the gains' gradients
// Blocks resident on an SM, by registers: the forward takes 64, the backward 80, or
// 128 with the gains' gradients (at 80 that one spills far more: 49 -> 92 us).
constexpr int qk_blocks(bool bwd, bool norm) { return !bwd ? 4 : norm ? 2 : 3; }
constexpr double kQkAngles = 1.0;       // cost of a token's angles, in slots

// The heads of one kind.  A slot is a warp's step: 32/lanes heads of a token, counted
// through all groups.
struct QkKind {
  int heads, first;                     // heads of a group, the first one's place in the row
  int slots;                            // of a token
  int warps;                            // they share the tokens' slots evenly
};

struct QkParams {
  const void *x, *dy;
  void *out;
  const void *gain[2];
  const int *pos;
  const gptl_rope_pair *table;
  float *part;                          // partial sums: queries' blocks, then keys', [hd] each
  long long x_ld, x_gs, y_ld, y_gs;
  QkKind kind[2];                       // queries, keys
  int blocks_q, blocks_qk;              // blocks [0, blocks_q), [blocks_q, blocks_qk), then values
  int v_vecs, v_first, v_blocks;        // 16-byte vectors of a row's values, the first's place
  int tokens, groups, hd, rot, axes, seq;
  int lanes, heads_per_warp;            // lanes of a head (see qk_lanes)
  float eps, inv_hd;
};

// The rotated pairs' turns, as 64-bit fractions of a turn, and axes, in shared
// memory.  Position times fraction, modulo 2^64, is the fraction of a turn that is
// left, with no rounding: far positions keep all their bits, and the loop over
// tokens needs no fp64.
struct QkTurns {
  unsigned long long turn[128];
  int axis[128];
};

__device__ __forceinline__ void qk_load_turns(const QkParams &p, QkTurns &t) {
  for (int j = threadIdx.x; j < p.rot / 2; j += blockDim.x) {
    const gptl_rope_pair e = p.table[j];
    t.turn[j] = __double2ull_rn((e.turns - floor(e.turns)) * 18446744073709551616.0);
    t.axis[j] = e.axis;
    if ((unsigned)e.axis >= (unsigned)p.axes) {
      set_device_error(kErrIndex);
      t.axis[j] = 0;
    }
  }
}

// Sines and cosines of one token's pairs, by the whole warp.  Lane c of a head
// holds pairs 8c .. 8c + 7; cs[i * lanes + c] = cosines of its pairs 2i and 2i + 1,
// then their sines, so that the lanes of a head read 16 neighbouring bytes each.
// The fast sine and cosine are documented as good to 2^-21.41 and 2^-21.19 absolute
// in [-pi, pi], and phi's three fp32 roundings are up to 2^-20.8: together a pair turns
// to within 2^-19 of its larger element, 2^-8 of a half step of fp16 and 2^-11 of bf16.
// (Of the pair: where a cos - b sin cancels, the result's own step may be smaller.)
__device__ __forceinline__ void qk_angles(const QkParams &p, const QkTurns &t, int token, float4 *cs,
                                          int lane) {
  __syncwarp();
  float *to = reinterpret_cast<float *>(cs + (lane % 8 / 2) * p.lanes + lane / 8) + lane % 2;
  const int by_row = p.pos ? 0 : token % p.seq;
  for (int j = lane; j < p.rot / 2; j += 32, to += 16) {
    const int at = p.pos ? __ldg(p.pos + (long long)t.axis[j] * p.tokens + token) : by_row;
    const long long left = (long long)((unsigned long long)(long long)at * t.turn[j]);
    const float phi = (float)(int)(left >> 32) * 1.4629180792671596e-9f;      // 2 pi / 2^32
    to[0] = __cosf(phi);
    to[2] = __sinf(phi);
  }
  __syncwarp();
}

// A lane's 8 pairs (a, b), two to a register pair: v0 and v1 hold them as
// neighbours (INTER) or as the vectors of first and of second elements.
template <typename T, bool INTER>
__device__ __forceinline__ void qk_unpack(const uint4 &v0, const uint4 &v1, float2 (&a)[4],
                                          float2 (&b)[4]) {
  const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (INTER) {
      const float2 p = Cvt<T>::unpack2(w[2 * i]), q = Cvt<T>::unpack2(w[2 * i + 1]);
      a[i] = make_float2(p.x, q.x);
      b[i] = make_float2(p.y, q.y);
    } else {
      a[i] = Cvt<T>::unpack2(w[i]);
      b[i] = Cvt<T>::unpack2(w[4 + i]);
    }
  }
}
template <typename T, bool INTER>
__device__ __forceinline__ void qk_pack(const float2 (&a)[4], const float2 (&b)[4], uint4 &v0,
                                        uint4 &v1) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (INTER) {
      w[2 * i] = Cvt<T>::pack2(a[i].x, b[i].x);
      w[2 * i + 1] = Cvt<T>::pack2(a[i].y, b[i].y);
    } else {
      w[i] = Cvt<T>::pack2(a[i].x, a[i].y);
      w[4 + i] = Cvt<T>::pack2(b[i].x, b[i].y);
    }
  }
  v0 = make_uint4(w[0], w[1], w[2], w[3]);
  v1 = make_uint4(w[4], w[5], w[6], w[7]);
}

// Turns the pairs (a, b) by the lane's table entries, or (BACK) the other way.
template <bool BACK>
__device__ __forceinline__ void qk_turn(float2 (&a)[4], float2 (&b)[4], const float4 *cs, int lanes) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 q = cs[i * lanes];
    const float2 c = make_float2(q.x, q.y), s = make_float2(q.z, q.w), n = make_float2(-q.z, -q.w);
    const float2 x = a[i];
    a[i] = fma2(x, c, mul2(b[i], BACK ? s : n));
    b[i] = fma2(b[i], c, mul2(x, BACK ? n : s));
  }
}

// Sums of v and w over a head's lanes, the same bits in each.  LANES = 0: a power
// of two of lanes (p.lanes), in a butterfly; else that number, added in lane order,
// in two steps where it has two factors.
template <int LANES, bool TWO>
__device__ __forceinline__ void qk_head_sum(const QkParams &p, int lane, int c, float &v, float &w) {
  if constexpr (LANES == 0) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
      if (o < p.lanes) {
        v += __shfl_xor_sync(0xffffffffu, v, o);
        if constexpr (TWO) w += __shfl_xor_sync(0xffffffffu, w, o);
      }
  } else {
    constexpr int R0 = LANES == 9 ? 3 : LANES % 2 == 0 ? 2 : LANES, R1 = LANES / R0;
    auto add = [&](int from, int n, int stride) {
      float a = __shfl_sync(0xffffffffu, v, from), b = 0.f;
      if constexpr (TWO) b = __shfl_sync(0xffffffffu, w, from);
#pragma unroll
      for (int k = 1; k < n; ++k) {
        a += __shfl_sync(0xffffffffu, v, from + k * stride);
        if constexpr (TWO) b += __shfl_sync(0xffffffffu, w, from + k * stride);
      }
      v = a;
      w = b;
    };
    add(lane - c % R0, R0, 1);
    if constexpr (R1 > 1) add(lane - c + c % R0, R1, R0);
  }
}

// The value heads of the last blocks: a warp copies every v_warps-th row, four at
// a time.
template <typename T>
__device__ void qk_copy_values(const QkParams &p, const T *from, long long f_ld, long long f_gs, T *to) {
  const int lane = threadIdx.x & 31;
  const unsigned warps = p.v_blocks * kQkWarps, rows = (unsigned)p.tokens * p.groups;
  for (unsigned r0 = (blockIdx.x - p.blocks_qk) * kQkWarps + threadIdx.x / 32; r0 < rows; r0 += 4 * warps) {
    const uint4 *src[4];
    uint4 *dst[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const unsigned r = r0 + k * warps < rows ? r0 + k * warps : r0;       // r0 again: the same bits
      const unsigned g = r / p.tokens, t = r - g * p.tokens;
      src[k] = reinterpret_cast<const uint4 *>(from + g * f_gs + t * f_ld) + p.v_first;
      dst[k] = reinterpret_cast<uint4 *>(to + g * p.y_gs + t * p.y_ld) + p.v_first;
    }
    for (int i = lane; i < p.v_vecs; i += 32) {
      uint4 u[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) u[k] = src[k][i];
#pragma unroll
      for (int k = 0; k < 4; ++k) dst[k][i] = u[k];
    }
  }
}

// BWD: out = dx from x and dy; else out = y from x.  NORM: with gains.
template <typename T, int LANES, bool INTER, bool NORM, bool BWD>
__global__ void __launch_bounds__(kQkWarps * 32, qk_blocks(BWD, NORM))
    qk_rope_kernel(const QkParams p) {
  constexpr bool kX = NORM || !BWD;                        // x is read
  __shared__ __align__(16) float4 cs_all[kQkWarps][4 * 16];
  __shared__ __align__(16) float4 gain_all[NORM ? 4 * 16 : 1];   // as cs_all: (a, a, b, b)
  __shared__ QkTurns turns_all;
  __shared__ float sums[BWD && NORM ? kQkWarps : 1][256];
  if constexpr (BWD && NORM) grid_dependents_launch();
  const T *in_x = static_cast<const T *>(p.x), *in_dy = static_cast<const T *>(p.dy);
  T *out = static_cast<T *>(p.out);
  if ((int)blockIdx.x >= p.blocks_qk) {
    if constexpr (BWD) qk_copy_values<T>(p, in_dy, p.y_ld, p.y_gs, out);
    else qk_copy_values<T>(p, in_x, p.x_ld, p.x_gs, out);
    return;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool key = (int)blockIdx.x >= p.blocks_q;
  const QkKind &K = p.kind[key];
  const int w = ((int)blockIdx.x - (key ? p.blocks_q : 0)) * kQkWarps + warp;

  // the lane's 16 elements of a head: two vectors of 8 at v0 and v1
  const int LPH = LANES ? LANES : p.lanes, HPW = LANES ? 32 / LANES : p.heads_per_warp;
  const int sub = lane / LPH, c = lane - sub * LPH;
  const bool on = c < p.hd / 16 && sub < HPW, turns = on && c < p.rot / 16;
  const bool split = turns && !INTER;                      // partners rot/2 apart
  const int v0 = !on ? 0 : split ? 8 * c : 16 * c, v1 = split ? v0 + p.rot / 2 : v0 + 8;

  qk_load_turns(p, turns_all);
  if constexpr (NORM) {
    if (warp == 0 && lane < LPH) {
      const T *g = static_cast<const T *>(p.gain[key]);
      float2 ga[4] = {}, gb[4] = {};                       // 0 beyond the head's elements
      if (on)
        qk_unpack<T, INTER>(*reinterpret_cast<const uint4 *>(g + v0),
                            *reinterpret_cast<const uint4 *>(g + v1), ga, gb);
#pragma unroll
      for (int i = 0; i < 4; ++i) gain_all[i * LPH + c] = make_float4(ga[i].x, ga[i].y, gb[i].x, gb[i].y);
    }
  }
  __syncthreads();
  const float4 *gain = gain_all + c, *cs = cs_all[warp] + c;
  float2 acc_a[4] = {}, acc_b[4] = {};                     // the gain's gradient

  // the warp's share of all tokens' slots, and its steps from slot to slot
  const int all = p.groups * K.heads;
  const int dg = HPW / K.heads, dh = HPW - dg * K.heads, dv = v1 - v0;
  const int g_sub = sub / K.heads, h_sub = sub - g_sub * K.heads;
  const long long x_step = dg * p.x_gs + dh * p.hd, x_wrap = p.x_gs - (long long)K.heads * p.hd;
  const long long y_step = dg * p.y_gs + dh * p.hd, y_wrap = p.y_gs - (long long)K.heads * p.hd;
  const long long total = (long long)p.tokens * K.slots;
  const long long lo = total * w / K.warps;
  int left = (int)(total * (w + 1) / K.warps - lo);
  int token = (int)(lo / K.slots), s0 = (int)(lo - (long long)token * K.slots);
  for (int n_slots; left > 0; left -= n_slots, ++token, s0 = 0) {
    n_slots = min(K.slots - s0, left);
    const int first = s0 * HPW + sub;                      // the lane's head among all
    int g0 = g_sub, h0 = h_sub;
    if (s0) {
      g0 = first / K.heads;
      h0 = first - g0 * K.heads;
    }
    const int col = (K.first + h0) * p.hd + v0;
    // the next slot to fetch: the lane's head, its number in all, its places
    int h = h0, n = first;
    const T *px = in_x + g0 * p.x_gs + token * p.x_ld + col;
    const T *pd = in_dy + g0 * p.y_gs + token * p.y_ld + col;
    T *po = out + g0 * p.y_gs + token * p.y_ld + col, *o = po;
    uint4 nx0, nx1, nd0, nd1;
    bool live;
    auto fetch = [&]() {
      live = on && n < all;
      o = po;
      if (live) {
        if constexpr (kX) {
          nx0 = *reinterpret_cast<const uint4 *>(px);
          nx1 = *reinterpret_cast<const uint4 *>(px + dv);
        }
        if constexpr (BWD) {
          nd0 = *reinterpret_cast<const uint4 *>(pd);
          nd1 = *reinterpret_cast<const uint4 *>(pd + dv);
        }
      } else {
        nx0 = nx1 = nd0 = nd1 = uint4{};
      }
      n += HPW;
      h += dh;
      px += x_step;
      pd += y_step;
      po += y_step;
      if (h >= K.heads) {
        h -= K.heads;
        px += x_wrap;
        pd += y_wrap;
        po += y_wrap;
      }
    };
    fetch();
    if (p.rot) qk_angles(p, turns_all, token, cs_all[warp], lane);
    for (int u = 0; u < n_slots; ++u) {
      // the slot's values leave the registers that the next slot's are loaded into
      float2 a[4], b[4], xa[4], xb[4];
      if constexpr (kX) qk_unpack<T, INTER>(nx0, nx1, xa, xb);
      if constexpr (BWD) qk_unpack<T, INTER>(nd0, nd1, a, b);
      T *to = o;
      const bool here = live;
      if (u + 1 < n_slots) fetch();
      if constexpr (BWD)
        if (turns) qk_turn<true>(a, b, cs, LPH);
      if constexpr (NORM) {
        float2 s2 = make_float2(0.f, 0.f), d2 = s2;
#pragma unroll
        for (int i = 0; i < 4; ++i) s2 = fma2(xa[i], xa[i], fma2(xb[i], xb[i], s2));
        float ss = s2.x + s2.y, sd = 0.f;
        if constexpr (BWD) {
          // the gain's gradient takes dn x, then dn becomes d = dn g
          float2 ta[4], tb[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 g = gain[i * LPH];
            const float2 ga = make_float2(g.x, g.y), gb = make_float2(g.z, g.w);
            ta[i] = mul2(a[i], xa[i]);
            tb[i] = mul2(b[i], xb[i]);
            d2 = fma2(ta[i], ga, fma2(tb[i], gb, d2));
            a[i] = mul2(a[i], ga);
            b[i] = mul2(b[i], gb);
          }
          sd = d2.x + d2.y;
          qk_head_sum<LANES, true>(p, lane, c, ss, sd);
          const float r = rsqrtf(fmaf(ss, p.inv_hd, p.eps));
          const float m = -(sd * p.inv_hd * r) * r * r;    // r^3 alone may leave fp32
          const float2 r2 = make_float2(r, r), m2 = make_float2(m, m);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            acc_a[i] = fma2(ta[i], r2, acc_a[i]);
            acc_b[i] = fma2(tb[i], r2, acc_b[i]);
            a[i] = fma2(a[i], r2, mul2(xa[i], m2));
            b[i] = fma2(b[i], r2, mul2(xb[i], m2));
          }
        } else {
          qk_head_sum<LANES, false>(p, lane, c, ss, sd);
          const float r = rsqrtf(fmaf(ss, p.inv_hd, p.eps));
          const float2 r2 = make_float2(r, r);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 g = gain[i * LPH];
            a[i] = mul2(mul2(xa[i], r2), make_float2(g.x, g.y));
            b[i] = mul2(mul2(xb[i], r2), make_float2(g.z, g.w));
          }
        }
      } else if constexpr (!BWD) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = xa[i];
          b[i] = xb[i];
        }
      }
      if (!BWD && turns) qk_turn<false>(a, b, cs, LPH);
      if (here) {
        uint4 q0, q1;
        qk_pack<T, INTER>(a, b, q0, q1);
        *reinterpret_cast<uint4 *>(to) = q0;
        *reinterpret_cast<uint4 *>(to + dv) = q1;
      }
    }
  }
  if constexpr (BWD && NORM) {
    // the warp's head positions, then the block's warps, each in a fixed order
    float f[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {                          // in the order of v0 and v1
      f[INTER ? 4 * i : 2 * i] = acc_a[i].x;
      f[INTER ? 4 * i + 2 : 2 * i + 1] = acc_a[i].y;
      f[INTER ? 4 * i + 1 : 8 + 2 * i] = acc_b[i].x;
      f[INTER ? 4 * i + 3 : 9 + 2 * i] = acc_b[i].y;
    }
    if constexpr (LANES == 0) {
      for (int o = LPH; o < 32; o <<= 1)
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] += __shfl_xor_sync(0xffffffffu, f[i], o);
    }
    for (int k = 0; k < (LANES == 0 ? 1 : HPW); ++k) {
      if (sub == k && on)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          sums[warp][v0 + i] = f[i] + (k ? sums[warp][v0 + i] : 0.f);
          sums[warp][v1 + i] = f[8 + i] + (k ? sums[warp][v1 + i] : 0.f);
        }
      __syncwarp();
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.hd; e += blockDim.x) {
      float t = 0.f;
#pragma unroll
      for (int k = 0; k < kQkWarps; ++k) t += sums[k][e];
      p.part[(long long)blockIdx.x * p.hd + e] = t;
    }
  }
}

// Adds the partial rows of the queries' (blockIdx.y = 0) and the keys' blocks,
// in order: 32 columns and 16 runs of rows a block.
__global__ void __launch_bounds__(512) qk_gain_kernel(const float *__restrict__ part, int nq, int nqk,
                                                      int hd, float *__restrict__ dgq,
                                                      float *__restrict__ dgk) {
  __shared__ float sm[16][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  const int lo = blockIdx.y ? nq : 0, hi = blockIdx.y ? nqk : nq;
  float s = 0.f;
  grid_dependency_wait();
  if (c < hd) {
#pragma unroll 4
    for (int b = lo + threadIdx.y; b < hi; b += 16) s += part[(long long)b * hd + c];
  }
  sm[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && c < hd) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += sm[i][threadIdx.x];
    (blockIdx.y ? dgk : dgq)[c] = t;
  }
}

}  // namespace gptl

namespace {

// Launches a kernel that may be brought up while the one before it on the stream
// still runs; the kernel itself waits for that one's results.
template <typename... P, typename... A>
int launch_after(void (*kern)(P...), dim3 grid, dim3 block, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  GPTL_CK(cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...));
  return GPTL_OK;
}

// rows * ld, or 0 where that is 2^56 or more (rows >= 1, ld < 2^56).
long long far_rows(long long rows, long long ld) {
  return rows < (1ll << 56) / ld ? rows * ld : 0;
}

// Sizes and strides of a descriptor; dense strides filled in.
int check_qk(const gptl_qk_desc &d, gptl_dtype dt, gptl_qk_desc *out) {
  if (dt != GPTL_FP16 && dt != GPTL_BF16) return GPTL_E_DTYPE;
  *out = d;
  if (d.tokens <= 0 || d.groups <= 0 || d.q_heads <= 0 || d.k_heads <= 0 || d.v_heads < 0 ||
      d.head_dim <= 0 || d.head_dim > 256 || d.head_dim % 16 || d.rot_dim < 0 ||
      d.rot_dim > d.head_dim || d.rot_dim % 16 || d.axes < 1 || d.axes > 4)
    return GPTL_E_SHAPE;
  const long long heads = (long long)d.q_heads + d.k_heads + d.v_heads;
  const long long rows = (long long)d.tokens * d.groups;
  if (heads * d.groups > (1 << 20) || rows >= (1ll << 30)) return GPTL_E_SHAPE;
  const long long width = heads * d.head_dim;
  if (d.interleaved != 0 && d.interleaved != 1) return GPTL_E_ARG;
  long long *str[2][2] = {{&out->x_ld, &out->x_gstride}, {&out->y_ld, &out->y_gstride}};
  for (auto &s : str) {
    long long &ld = *s[0], &gs = *s[1];
    if (ld < 0 || gs < 0 || ld % 8 || gs % 8 || ld >= (1ll << 40) || gs >= (1ll << 40))
      return GPTL_E_SHAPE;
    if (ld == 0) ld = width;
    // offsets stay below 2^56 elements, more than there are addresses for
    const long long column = far_rows(d.tokens, ld);
    if (!column) return GPTL_E_SHAPE;
    if (gs == 0) gs = column;
    if (!far_rows(d.groups, gs)) return GPTL_E_SHAPE;
    if (d.tokens > 1 && ld < width) return GPTL_E_SHAPE;
    if (d.groups > 1 && gs < width) return GPTL_E_SHAPE;
    // groups outside tokens, or tokens outside groups: rows never overlap
    if (d.tokens > 1 && d.groups > 1 && gs < (long long)(d.tokens - 1) * ld + width &&
        ld < (long long)(d.groups - 1) * gs + width)
      return GPTL_E_SHAPE;
  }
  return GPTL_OK;
}

bool ranges_overlap(const void *a, long long na, const void *b, long long nb) {
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
  return pa < pb + (uintptr_t)nb && pb < pa + (uintptr_t)na;
}

// The same for two sets of rows with the same strides, `shape` = {groups, gstride,
// tokens, ld, width} in bytes: only the rows count, not what lies between them, so
// that column ranges of one buffer are apart.  (rows of a set never overlap; at most
// 2^15 steps, tokens * groups being below 2^30)
struct RowsShape {
  long long groups, gstride, tokens, ld, width;
  long long span() const { return (groups - 1) * gstride + (tokens - 1) * ld + width; }
};
bool rows_overlap(const void *a, const void *b, RowsShape s) {
  if (!ranges_overlap(a, s.span(), b, s.span())) return false;
  if (s.tokens < s.groups) {
    std::swap(s.tokens, s.groups);
    std::swap(s.ld, s.gstride);
  }
  const long long apart =
      (long long)(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a));
  for (long long g = 1 - s.groups; g < s.groups; ++g) {
    const long long rest = apart - g * s.gstride;
    long long t = s.tokens > 1 ? rest / s.ld - 1 : 0;          // ld >= width: three rows at most
    const long long last = s.tokens > 1 ? t + 2 : 0;
    for (; t <= last; ++t) {
      const long long off = s.tokens > 1 ? rest - t * s.ld : rest;
      if (t > -s.tokens && t < s.tokens && off < s.width && off > -s.width) return true;
    }
  }
  return false;
}

RowsShape qk_rows(const gptl_qk_desc &d, long long ld, long long gs) {
  const long long width = ((long long)d.q_heads + d.k_heads + d.v_heads) * d.head_dim;
  return RowsShape{d.groups, 2 * gs, d.tokens, 2 * ld, 2 * width};
}

// x (x strides) and a buffer with the y strides: row by row where the strides agree.
bool qk_overlap(const gptl_qk_desc &d, const void *x, const void *y) {
  const RowsShape sx = qk_rows(d, d.x_ld, d.x_gstride), sy = qk_rows(d, d.y_ld, d.y_gstride);
  if ((d.tokens == 1 || sx.ld == sy.ld) && (d.groups == 1 || sx.gstride == sy.gstride))
    return rows_overlap(x, y, sx);
  return ranges_overlap(x, sx.span(), y, sy.span());
}

// Lanes of a head: one for each 16 elements where that lets a warp hold more heads
// than the next power of two does (3, 5, 6, 9 and 10), else that power of two.
int qk_lanes(int hd) {
  const int n = hd / 16;
  int l = 1;
  while (l < n) l *= 2;
  return 32 / n > 32 / l ? n : l;
}

// Sizes, and the split of the work over `blocks` resident blocks.  Queries and
// keys get blocks of their own, in proportion to their slots (a token's angles
// cost about kQkAngles of them), so that a warp keeps one gain's gradient in
// registers; the warps of a kind take equal runs of its tokens' slots, to the
// slot, so that the last wave is as full as the others.  Value heads come in
// blocks behind these: with or without them, the sums have one order.
QkParams qk_params(const gptl_qk_desc &d, int v_heads, int blocks) {
  QkParams p{};
  const int lanes = qk_lanes(d.head_dim), hpw = 32 / lanes;
  p.lanes = lanes;
  p.heads_per_warp = hpw;
  const int heads[2] = {d.q_heads, d.k_heads};
  const double angles = d.rot_dim ? kQkAngles : 0.0;
  double weight[2];
  for (int i = 0; i < 2; ++i) {
    QkKind &k = p.kind[i];
    k.heads = heads[i];
    k.first = i ? d.q_heads : 0;
    k.slots = (int)(((long long)heads[i] * d.groups + hpw - 1) / hpw);
    weight[i] = angles + (double)k.slots;
  }
  for (int i = 0; i < 2; ++i) {
    QkKind &k = p.kind[i];
    long long nb = (long long)(blocks * weight[i] / (weight[0] + weight[1]) + 0.5);
    const int free_blocks = i ? blocks - p.blocks_q : blocks - 1;   // one at least for the keys
    if (nb > free_blocks) nb = free_blocks;
    const long long total = (long long)d.tokens * k.slots;
    const long long most = (total + kQkWarps - 1) / kQkWarps;
    if (nb > most) nb = most;
    if (nb < 1) nb = 1;
    k.warps = (int)(nb * kQkWarps);
    if (i == 0) p.blocks_q = (int)nb;
    else p.blocks_qk = p.blocks_q + (int)nb;
  }
  p.v_vecs = v_heads * d.head_dim / 8;
  p.v_first = (d.q_heads + d.k_heads) * d.head_dim / 8;
  if (v_heads) {
    const long long rows = (long long)d.tokens * d.groups, want = 4ll * blocks;
    const long long nb = (rows + 4 * kQkWarps - 1) / (4 * kQkWarps);
    p.v_blocks = (int)(nb < want ? nb : want);
  }
  p.x_ld = d.x_ld; p.x_gs = d.x_gstride; p.y_ld = d.y_ld; p.y_gs = d.y_gstride;
  p.tokens = d.tokens; p.groups = d.groups; p.hd = d.head_dim;
  p.rot = d.rot_dim; p.axes = d.axes; p.seq = d.seq;
  p.eps = d.eps; p.inv_hd = 1.0f / (float)d.head_dim;
  return p;
}

template <bool BWD>
int qk_launch(const QkParams &p, gptl_dtype dt, bool interleaved, cudaStream_t st) {
  const unsigned grid = (unsigned)(p.blocks_qk + p.v_blocks);
  const bool norm = p.gain[0] != nullptr;
  auto run = [&]<typename T, int LANES, bool INTER, bool NORM>() {
    qk_rope_kernel<T, LANES, INTER, NORM, BWD><<<grid, kQkWarps * 32, 0, st>>>(p);
  };
  auto go = [&]<typename T, bool INTER>() {
    if (!norm) return run.template operator()<T, 0, INTER, false>();      // no sums over lanes
    switch (p.lanes) {
      case 3: return run.template operator()<T, 3, INTER, true>();
      case 5: return run.template operator()<T, 5, INTER, true>();
      case 6: return run.template operator()<T, 6, INTER, true>();
      case 9: return run.template operator()<T, 9, INTER, true>();
      case 10: return run.template operator()<T, 10, INTER, true>();
      default: return run.template operator()<T, 0, INTER, true>();
    }
  };
  auto by_pairs = [&]<typename T>() {
    if (interleaved) go.template operator()<T, true>();
    else go.template operator()<T, false>();
  };
  if (dt == GPTL_FP16) by_pairs.template operator()<__half>();
  else by_pairs.template operator()<__nv_bfloat16>();
  GPTL_CK(cudaGetLastError());
  prof_launched(st, BWD ? GPTL_KIND_QK_ROPE_BWD : GPTL_KIND_QK_ROPE_FWD);
  return GPTL_OK;
}

int check_qk_common(const gptl_qk_desc &d, const void *gq, const void *gk, const int *pos,
                    const gptl_rope_pair *table) {
  if ((gq == nullptr) != (gk == nullptr) || (d.rot_dim && !table)) return GPTL_E_NULL;
  if (!aligned16(gq) || !aligned16(gk) || !aligned16(table) ||
      (reinterpret_cast<uintptr_t>(pos) & 3u))
    return GPTL_E_ALIGN;
  if (!pos && d.rot_dim && d.seq < 1) return GPTL_E_SHAPE;
  if (gq && !(d.eps > 0.f && d.eps <= 3.0e38f)) return GPTL_E_ARG;
  return GPTL_OK;
}

}  // namespace

extern "C" {

int gptl_rope_table(int rot_dim, int axes, const int *axis_pairs, int per_axis, double base,
                    gptl_rope_pair *table) {
  if (!table || (!axis_pairs && axes != 1)) return GPTL_E_NULL;
  if (rot_dim < 0 || rot_dim > 256 || rot_dim % 16 || axes < 1 || axes > 4) return GPTL_E_SHAPE;
  const int pairs = rot_dim / 2;
  long long sum = axis_pairs ? 0 : pairs;
  for (int a = 0; axis_pairs && a < axes; ++a) {
    if (axis_pairs[a] < 0) return GPTL_E_SHAPE;
    sum += axis_pairs[a];
  }
  if (sum != pairs) return GPTL_E_SHAPE;
  if (!(base > 0.0) || !(base <= 1.0e300) || (per_axis != 0 && per_axis != 1)) return GPTL_E_ARG;
  const double two_pi = 6.283185307179586476925286766559;
  int j = 0;
  for (int a = 0; a < axes; ++a) {
    const int n = axis_pairs ? axis_pairs[a] : pairs;
    for (int i = 0; i < n; ++i, ++j) {
      const double e = per_axis ? (double)i / n : (double)j / pairs;
      table[j] = gptl_rope_pair{pow(base, -e) / two_pi, a, 0};
    }
  }
  return GPTL_OK;
}

int gptl_qk_norm_rope_fwd(const gptl_qk_desc *desc, gptl_dtype dtype, const void *x, void *y,
                          const void *gq, const void *gk, const int *pos,
                          const gptl_rope_pair *table, gptl_stream_t stream) {
  if (!desc || !x || !y) return GPTL_E_NULL;
  gptl_qk_desc d;
  GPTL_TRY(check_qk(*desc, dtype, &d));
  if (!aligned16(x) || !aligned16(y)) return GPTL_E_ALIGN;
  GPTL_TRY(check_qk_common(d, gq, gk, pos, table));
  const bool in_place = x == y;
  if (in_place) {
    if (d.x_ld != d.y_ld || d.x_gstride != d.y_gstride) return GPTL_E_ARG;
  } else if (qk_overlap(d, x, y)) {
    return GPTL_E_ARG;
  }
  int sms = 0;
  GPTL_TRY(device_check(&sms));
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  QkParams p = qk_params(d, in_place ? 0 : d.v_heads, sms * qk_blocks(false, gq != nullptr));
  p.x = x;
  p.out = y;
  p.gain[0] = gq;
  p.gain[1] = gk;
  p.pos = pos;
  p.table = table;
  prof_start(st);
  return qk_launch<false>(p, dtype, d.interleaved, st);
}

size_t gptl_qk_norm_rope_scratch_bytes(const gptl_qk_desc *desc) {
  gptl_qk_desc d;
  if (!desc || check_qk(*desc, GPTL_BF16, &d) != GPTL_OK) return 0;
  return (size_t)kQkMaxBlocks * (size_t)d.head_dim * sizeof(float);
}

int gptl_qk_norm_rope_bwd(const gptl_qk_desc *desc, gptl_dtype dtype, const void *x, const void *dy,
                          void *dx, const void *gq, const void *gk, const int *pos,
                          const gptl_rope_pair *table, float *dgq, float *dgk, void *scratch,
                          gptl_stream_t stream) {
  if (!desc || !x || !dy || !dx) return GPTL_E_NULL;
  gptl_qk_desc d;
  GPTL_TRY(check_qk(*desc, dtype, &d));
  if (!aligned16(x) || !aligned16(dy) || !aligned16(dx)) return GPTL_E_ALIGN;
  GPTL_TRY(check_qk_common(d, gq, gk, pos, table));
  if (gq && (!dgq || !dgk || !scratch)) return GPTL_E_NULL;
  if (!gq && (dgq || dgk)) return GPTL_E_NULL;
  if (!aligned16(dgq) || !aligned16(dgk) || !aligned16(scratch)) return GPTL_E_ALIGN;
  if (qk_overlap(d, x, dx) || (dy != dx && rows_overlap(dy, dx, qk_rows(d, d.y_ld, d.y_gstride))))
    return GPTL_E_ARG;
  int sms = 0;
  GPTL_TRY(device_check(&sms));
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  int most = sms * qk_blocks(true, gq != nullptr);
  if (most > kQkMaxBlocks) most = kQkMaxBlocks;
  QkParams p = qk_params(d, dy == dx ? 0 : d.v_heads, most);
  p.x = x;
  p.dy = dy;
  p.out = dx;
  p.gain[0] = gq;
  p.gain[1] = gk;
  p.pos = pos;
  p.table = table;
  p.part = static_cast<float *>(scratch);
  prof_start(st);
  GPTL_TRY(qk_launch<true>(p, dtype, d.interleaved, st));
  if (!gq) return GPTL_OK;
  GPTL_TRY(launch_after(qk_gain_kernel, dim3((d.head_dim + 31) / 32, 2), dim3(32, 16), st,
                        (const float *)p.part, p.blocks_q, p.blocks_qk, d.head_dim, dgq, dgk));
  prof_launched(st, GPTL_KIND_REDUCE);
  return GPTL_OK;
}

}  // extern "C"
