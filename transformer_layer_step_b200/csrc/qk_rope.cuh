// Norm and rotation of queries and keys, forward and backward, on the packed
// [Q | K | V] rows between the QKV product and attention.
//
// With x one head of one token, g its gain and r = 1 / sqrt(mean(x^2) + eps):
//   forward   n = x r g, then each pair (a, b) of n turns by phi;
//   backward  dn = dy turned back by phi, d = dn g,
//             dx = r d - x r^3 mean(d x),   dg = sum dn x r,
// where mean(x^2) and mean(d x) are summed together, so a head needs one
// reduction.  phi in turns is pos * turns_j, taken and reduced to [-1/2, 1/2]
// in fp64, since fp32 has lost the fraction of far positions; its sine and
// cosine are fp32.
//
// Bound by HBM: 4 bytes an element forward, 6 backward.  A warp takes a token:
// its lanes compute the token's rot_dim/2 sines and cosines once, into shared
// memory, and use them for every head.  A lane owns 16 elements of a head, two
// 16-byte vectors chosen so that it holds both elements of each of its 8
// pairs: rotation needs no exchange, and the norm log2(lanes) shuffles.
//
// Included by libgptlayer.cu after gptlayer.cu, in the same translation unit.
#pragma once

#include "gptlayer_parts.h"

namespace gptl {

constexpr int kQkWarps = 8;             // warps of a block
constexpr int kQkMaxPairs = 128;        // head_dim <= 256
constexpr int kQkMaxBlocks = 592;       // partial rows of the gains' gradients

struct QkParams {
  const void *x, *dy;
  void *out;
  const void *gq, *gk;
  const int *pos;
  const gptl_rope_pair *table;
  float *part;                          // [2][gridDim.x][hd] (backward with gains)
  long long x_ld, x_gs, y_ld, y_gs;
  unsigned items, chunks, spc;          // (token, chunk of head slots) pairs; q, k slots per chunk
  int tokens, q, k, v, hd, rot, axes, seq, interleaved;
  int slots_q, slots_k, slots_v;        // groups of 32/LPH heads of each kind
  float eps, inv_hd;
};

// The 16 elements of a lane within its head: two vectors of 8 at v0 and v1.
struct QkLane {
  int sub, v0, v1;
  bool on, turns;
  __device__ QkLane(const QkParams &p, int lane, int lph) {
    const int c = lane % lph;
    sub = lane / lph;
    on = c < p.hd / 16;
    turns = c < p.rot / 16;
    const bool split = turns && !p.interleaved;       // partners rot/2 apart
    v0 = split ? 8 * c : 16 * c;
    v1 = split ? v0 + p.rot / 2 : v0 + 8;
  }
};

// Sines and cosines of one token's pairs, by the whole warp.
__device__ __forceinline__ void qk_angles(const QkParams &p, int token, float2 *cs, int lane) {
  __syncwarp();
  for (int j = lane; j < p.rot / 2; j += 32) {
    const gptl_rope_pair e = p.table[j];
    int axis = e.axis;
    if ((unsigned)axis >= (unsigned)p.axes) {
      set_device_error(kErrIndex);
      axis = 0;
    }
    const int at = p.pos ? __ldg(p.pos + (long long)axis * p.tokens + token) : token % p.seq;
    double t = (double)at * e.turns;
    t -= rint(t);
    float s, c;
    sincospif(2.0f * (float)t, &s, &c);
    cs[j] = make_float2(c, s);
  }
  __syncwarp();
}

// Turns the pairs held in a, b (vectors v0 and v1) by (cos, dir * sin).
__device__ __forceinline__ void qk_turn(float (&a)[8], float (&b)[8], const float2 (&cs)[8],
                                        bool interleaved, float dir) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float c0 = cs[i].x, s0 = dir * cs[i].y, c1 = cs[4 + i].x, s1 = dir * cs[4 + i].y;
      const float x0 = a[2 * i], y0 = a[2 * i + 1], x1 = b[2 * i], y1 = b[2 * i + 1];
      a[2 * i] = x0 * c0 - y0 * s0;
      a[2 * i + 1] = y0 * c0 + x0 * s0;
      b[2 * i] = x1 * c1 - y1 * s1;
      b[2 * i + 1] = y1 * c1 + x1 * s1;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float c = cs[i].x, s = dir * cs[i].y;
      const float x = a[i], y = b[i];
      a[i] = x * c - y * s;
      b[i] = y * c + x * s;
    }
  }
}

// Column of the first element of a lane's head in slot s (queries, then keys),
// or -1 for no head.  Heads of a kind fill their slots in order, 32/LPH to a slot.
__device__ __forceinline__ int qk_column(const QkParams &p, int s, int hpw, const QkLane &L) {
  const bool key = s >= p.slots_q;
  const int h = (key ? s - p.slots_q : s) * hpw + L.sub;
  return L.on && h < (key ? p.k : p.q) ? (key ? p.q + h : h) * p.hd : -1;
}

// Copies chunk `chunk`'s share of a row's value heads.
template <typename T>
__device__ __forceinline__ void qk_copy_values(const QkParams &p, unsigned chunk, int hpw,
                                               const QkLane &L, const T *from, T *to) {
  const int lo = (int)((long long)p.slots_v * chunk / p.chunks);
  const int hi = (int)((long long)p.slots_v * (chunk + 1) / p.chunks);
#pragma unroll 2
  for (int s = lo; s < hi; ++s) {
    const int h = s * hpw + L.sub;
    if (!L.on || h >= p.v) continue;
    const long long col = (long long)(p.q + p.k + h) * p.hd;
    const uint4 a = *reinterpret_cast<const uint4 *>(from + col + L.v0);
    const uint4 b = *reinterpret_cast<const uint4 *>(from + col + L.v1);
    *reinterpret_cast<uint4 *>(to + col + L.v0) = a;
    *reinterpret_cast<uint4 *>(to + col + L.v1) = b;
  }
}

// Gains of queries and keys in shared memory, fp32 (1 where there are none).
template <typename T>
__device__ __forceinline__ void qk_gains(const QkParams &p, float *gain) {
  for (int i = threadIdx.x; i < p.hd; i += blockDim.x) {
    gain[i] = p.gq ? Cvt<T>::to_f(static_cast<const T *>(p.gq)[i]) : 1.f;
    gain[p.hd + i] = p.gk ? Cvt<T>::to_f(static_cast<const T *>(p.gk)[i]) : 1.f;
  }
  __syncthreads();
}

__device__ __forceinline__ void qk_load_gain(const float *g, const QkLane &L, float (&a)[8],
                                             float (&b)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    const float4 u = *reinterpret_cast<const float4 *>(g + L.v0 + i);
    const float4 w = *reinterpret_cast<const float4 *>(g + L.v1 + i);
    a[i] = u.x; a[i + 1] = u.y; a[i + 2] = u.z; a[i + 3] = u.w;
    b[i] = w.x; b[i + 1] = w.y; b[i + 2] = w.z; b[i + 3] = w.w;
  }
}

template <typename T, int LPH>
__global__ void __launch_bounds__(kQkWarps * 32, 3) qk_rope_fwd_kernel(const QkParams p) {
  constexpr int HPW = 32 / LPH;
  __shared__ __align__(16) float2 cs_all[kQkWarps][kQkMaxPairs];
  __shared__ __align__(16) float gain[512];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const QkLane L(p, lane, LPH);
  const bool norm = p.gq != nullptr;
  if (norm) qk_gains<T>(p, gain);
  for (unsigned item = blockIdx.x * kQkWarps + warp; item < p.items; item += gridDim.x * kQkWarps) {
    const unsigned row = item / p.chunks, chunk = item - row * p.chunks;
    const unsigned g = row / p.tokens, token = row - g * p.tokens;
    const T *x = static_cast<const T *>(p.x) + g * p.x_gs + token * p.x_ld;
    T *y = static_cast<T *>(p.out) + g * p.y_gs + token * p.y_ld;
    const int s0 = chunk * p.spc, s1 = min(s0 + (int)p.spc, p.slots_q + p.slots_k);
    uint4 n0 = {}, n1 = {};
    int ncol = qk_column(p, s0, HPW, L);
    if (ncol >= 0) {
      n0 = *reinterpret_cast<const uint4 *>(x + ncol + L.v0);
      n1 = *reinterpret_cast<const uint4 *>(x + ncol + L.v1);
    }
    float2 cs[8];
    if (p.rot) {
      qk_angles(p, token, cs_all[warp], lane);
      if (L.turns) {
        const float4 *src = reinterpret_cast<const float4 *>(cs_all[warp] + 8 * (lane % LPH));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 u = src[i];
          cs[2 * i] = make_float2(u.x, u.y);
          cs[2 * i + 1] = make_float2(u.z, u.w);
        }
      }
    }
    for (int s = s0; s < s1; ++s) {
      const uint4 u0 = n0, u1 = n1;
      const int col = ncol;
      if (s + 1 < s1) {                          // the next slot's loads go out first
        ncol = qk_column(p, s + 1, HPW, L);
        n0 = n1 = uint4{};
        if (ncol >= 0) {
          n0 = *reinterpret_cast<const uint4 *>(x + ncol + L.v0);
          n1 = *reinterpret_cast<const uint4 *>(x + ncol + L.v1);
        }
      }
      float a[8], b[8];
      unpack8<T>(u0, a);
      unpack8<T>(u1, b);
      if (norm) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(a[i], a[i], fmaf(b[i], b[i], ss));
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float r = rsqrtf(fmaf(ss, p.inv_hd, p.eps));
        if (col >= 0) {
          float ga[8], gb[8];
          qk_load_gain(gain + (s < p.slots_q ? 0 : p.hd), L, ga, gb);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            a[i] = a[i] * r * ga[i];
            b[i] = b[i] * r * gb[i];
          }
        }
      }
      if (col < 0) continue;
      if (L.turns) qk_turn(a, b, cs, p.interleaved, 1.f);
      *reinterpret_cast<uint4 *>(y + col + L.v0) = pack8<T>(a);
      *reinterpret_cast<uint4 *>(y + col + L.v1) = pack8<T>(b);
    }
    if (p.slots_v) qk_copy_values<T>(p, chunk, HPW, L, x, y);
  }
}

template <typename T, int LPH>
__global__ void __launch_bounds__(kQkWarps * 32, 2) qk_rope_bwd_kernel(const QkParams p) {
  constexpr int HPW = 32 / LPH;
  __shared__ __align__(16) float2 cs_all[kQkWarps][kQkMaxPairs];
  __shared__ __align__(16) float gain[512];
  __shared__ float sums[kQkWarps][512];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const QkLane L(p, lane, LPH);
  const bool norm = p.gq != nullptr;
  if (norm) qk_gains<T>(p, gain);
  float dq0[8] = {}, dq1[8] = {}, dk0[8] = {}, dk1[8] = {};
  for (unsigned item = blockIdx.x * kQkWarps + warp; item < p.items; item += gridDim.x * kQkWarps) {
    const unsigned row = item / p.chunks, chunk = item - row * p.chunks;
    const unsigned g = row / p.tokens, token = row - g * p.tokens;
    const T *x = static_cast<const T *>(p.x) + g * p.x_gs + token * p.x_ld;
    const T *dy = static_cast<const T *>(p.dy) + g * p.y_gs + token * p.y_ld;
    T *dx = static_cast<T *>(p.out) + g * p.y_gs + token * p.y_ld;
    const int s0 = chunk * p.spc, s1 = min(s0 + (int)p.spc, p.slots_q + p.slots_k);
    float2 cs[8];
    if (p.rot) {
      qk_angles(p, token, cs_all[warp], lane);
      if (L.turns) {
        const float4 *src = reinterpret_cast<const float4 *>(cs_all[warp] + 8 * (lane % LPH));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 u = src[i];
          cs[2 * i] = make_float2(u.x, u.y);
          cs[2 * i + 1] = make_float2(u.z, u.w);
        }
      }
    }
    // the slots [lo, hi) of one kind of head, its gain's gradient in (acc0, acc1)
    auto heads = [&](int lo, int hi, const float *gp, float (&acc0)[8], float (&acc1)[8]) {
      uint4 nx0 = {}, nx1 = {}, nd0 = {}, nd1 = {};
      int ncol = -1;
      auto fetch = [&](int s) {
        ncol = qk_column(p, s, HPW, L);
        nx0 = nx1 = nd0 = nd1 = uint4{};
        if (ncol < 0) return;
        nd0 = *reinterpret_cast<const uint4 *>(dy + ncol + L.v0);
        nd1 = *reinterpret_cast<const uint4 *>(dy + ncol + L.v1);
        if (norm) {
          nx0 = *reinterpret_cast<const uint4 *>(x + ncol + L.v0);
          nx1 = *reinterpret_cast<const uint4 *>(x + ncol + L.v1);
        }
      };
      if (lo < hi) fetch(lo);
      for (int s = lo; s < hi; ++s) {
        const uint4 x0 = nx0, x1 = nx1, d0 = nd0, d1 = nd1;
        const int col = ncol;
        if (s + 1 < hi) fetch(s + 1);
        float a[8], b[8];
        unpack8<T>(d0, a);
        unpack8<T>(d1, b);
        if (L.turns) qk_turn(a, b, cs, p.interleaved, -1.f);
        if (norm) {
          float xa[8], xb[8], ga[8], gb[8], ss = 0.f, sd = 0.f;
          unpack8<T>(x0, xa);
          unpack8<T>(x1, xb);
          if (L.on) {
            qk_load_gain(gp, L, ga, gb);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) ga[i] = gb[i] = 0.f;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            ss = fmaf(xa[i], xa[i], fmaf(xb[i], xb[i], ss));
            sd = fmaf(a[i] * ga[i], xa[i], fmaf(b[i] * gb[i], xb[i], sd));
          }
#pragma unroll
          for (int o = LPH / 2; o > 0; o >>= 1) {
            ss += __shfl_xor_sync(0xffffffffu, ss, o);
            sd += __shfl_xor_sync(0xffffffffu, sd, o);
          }
          const float r = rsqrtf(fmaf(ss, p.inv_hd, p.eps));
          const float w = r * r * r * (sd * p.inv_hd);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            acc0[i] = fmaf(a[i], xa[i] * r, acc0[i]);
            acc1[i] = fmaf(b[i], xb[i] * r, acc1[i]);
            a[i] = r * (a[i] * ga[i]) - w * xa[i];
            b[i] = r * (b[i] * gb[i]) - w * xb[i];
          }
        }
        if (col < 0) continue;
        *reinterpret_cast<uint4 *>(dx + col + L.v0) = pack8<T>(a);
        *reinterpret_cast<uint4 *>(dx + col + L.v1) = pack8<T>(b);
      }
    };
    heads(s0, min(s1, p.slots_q), gain, dq0, dq1);
    heads(max(s0, p.slots_q), s1, gain + p.hd, dk0, dk1);
    if (p.slots_v) qk_copy_values<T>(p, chunk, HPW, L, dy, dx);
  }
  if (!norm) return;
  // the warp's head positions, then the block's warps, each in a fixed order
#pragma unroll
  for (int o = LPH; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      dq0[i] += __shfl_xor_sync(0xffffffffu, dq0[i], o);
      dq1[i] += __shfl_xor_sync(0xffffffffu, dq1[i], o);
      dk0[i] += __shfl_xor_sync(0xffffffffu, dk0[i], o);
      dk1[i] += __shfl_xor_sync(0xffffffffu, dk1[i], o);
    }
  if (lane < LPH && L.on)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      sums[warp][L.v0 + i] = dq0[i];
      sums[warp][L.v1 + i] = dq1[i];
      sums[warp][p.hd + L.v0 + i] = dk0[i];
      sums[warp][p.hd + L.v1 + i] = dk1[i];
    }
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * p.hd; c += blockDim.x) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kQkWarps; ++w) s += sums[w][c];
    const int kind = c >= p.hd;
    p.part[((long long)kind * gridDim.x + blockIdx.x) * p.hd + (c - kind * p.hd)] = s;
  }
}

}  // namespace gptl

namespace {

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
  if (heads > (1 << 20) || rows >= (1ll << 31)) return GPTL_E_SHAPE;
  const long long width = heads * d.head_dim;
  if (d.interleaved != 0 && d.interleaved != 1) return GPTL_E_ARG;
  long long *str[2][2] = {{&out->x_ld, &out->x_gstride}, {&out->y_ld, &out->y_gstride}};
  for (auto &s : str) {
    long long &ld = *s[0], &gs = *s[1];
    if (ld < 0 || gs < 0 || ld % 8 || gs % 8 || ld >= (1ll << 40) || gs >= (1ll << 40))
      return GPTL_E_SHAPE;
    if (ld == 0) ld = width;
    if (gs == 0) gs = (long long)d.tokens * ld;
    if (d.tokens > 1 && ld < width) return GPTL_E_SHAPE;
    if (d.groups > 1 && gs < width) return GPTL_E_SHAPE;
    // groups outside tokens, or tokens outside groups: rows never overlap
    if (d.tokens > 1 && d.groups > 1 && gs < (long long)(d.tokens - 1) * ld + width &&
        ld < (long long)(d.groups - 1) * gs + width)
      return GPTL_E_SHAPE;
  }
  return GPTL_OK;
}

long long qk_span_bytes(const gptl_qk_desc &d, long long ld, long long gs) {
  const long long width = ((long long)d.q_heads + d.k_heads + d.v_heads) * d.head_dim;
  return 2 * ((d.groups - 1) * gs + (long long)(d.tokens - 1) * ld + width);
}

bool ranges_overlap(const void *a, long long na, const void *b, long long nb) {
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
  return pa < pb + (uintptr_t)nb && pb < pa + (uintptr_t)na;
}

int qk_lanes(int hd) {                    // lanes per head: a power of two >= head_dim / 16
  int l = 1;
  while (l < hd / 16) l *= 2;
  return l;
}

// Fills the launch-independent fields and picks the split of a token's heads
// over warps: whole tokens once they give every resident warp several, else
// chunks of head slots, down to one slot a warp for a handful of tokens.  Value
// heads do not enter the split, so in place or not, the sums have one order.
QkParams qk_params(const gptl_qk_desc &d, int v_heads, int warps) {
  QkParams p{};
  const int hpw = 32 / qk_lanes(d.head_dim);
  p.slots_q = (d.q_heads + hpw - 1) / hpw;
  p.slots_k = (d.k_heads + hpw - 1) / hpw;
  p.slots_v = (v_heads + hpw - 1) / hpw;
  const int slots = p.slots_q + p.slots_k;
  const long long rows = (long long)d.tokens * d.groups;
  long long chunks = (4ll * warps + rows - 1) / rows;
  if (chunks > slots) chunks = slots;
  p.spc = (unsigned)((slots + chunks - 1) / chunks);
  p.chunks = (unsigned)((slots + p.spc - 1) / p.spc);
  p.items = (unsigned)(rows * p.chunks);
  p.x_ld = d.x_ld; p.x_gs = d.x_gstride; p.y_ld = d.y_ld; p.y_gs = d.y_gstride;
  p.tokens = d.tokens; p.q = d.q_heads; p.k = d.k_heads; p.v = v_heads; p.hd = d.head_dim;
  p.rot = d.rot_dim; p.axes = d.axes; p.seq = d.seq; p.interleaved = d.interleaved;
  p.eps = d.eps; p.inv_hd = 1.0f / (float)d.head_dim;
  return p;
}

template <bool BWD>
int qk_launch(const QkParams &p, gptl_dtype dt, unsigned grid, cudaStream_t st) {
  auto go = [&]<typename T, int LPH>() {
    if constexpr (BWD) qk_rope_bwd_kernel<T, LPH><<<grid, kQkWarps * 32, 0, st>>>(p);
    else qk_rope_fwd_kernel<T, LPH><<<grid, kQkWarps * 32, 0, st>>>(p);
  };
  auto by_lanes = [&]<typename T>() {
    switch (qk_lanes(p.hd)) {
      case 1: go.template operator()<T, 1>(); break;
      case 2: go.template operator()<T, 2>(); break;
      case 4: go.template operator()<T, 4>(); break;
      case 8: go.template operator()<T, 8>(); break;
      default: go.template operator()<T, 16>(); break;
    }
  };
  if (dt == GPTL_FP16) by_lanes.template operator()<__half>();
  else by_lanes.template operator()<__nv_bfloat16>();
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
  } else if (ranges_overlap(x, qk_span_bytes(d, d.x_ld, d.x_gstride), y,
                            qk_span_bytes(d, d.y_ld, d.y_gstride))) {
    return GPTL_E_ARG;
  }
  int sms = 0;
  GPTL_TRY(device_check(&sms));
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  QkParams p = qk_params(d, in_place ? 0 : d.v_heads, sms * 3 * kQkWarps);
  p.x = x;
  p.out = y;
  p.gq = gq;
  p.gk = gk;
  p.pos = pos;
  p.table = table;
  unsigned grid = (p.items + kQkWarps - 1) / kQkWarps;
  if (grid > 3u * sms) grid = 3u * sms;
  prof_start(st);
  return qk_launch<false>(p, dtype, grid, st);
}

size_t gptl_qk_norm_rope_scratch_bytes(const gptl_qk_desc *desc) {
  gptl_qk_desc d;
  if (!desc || check_qk(*desc, GPTL_BF16, &d) != GPTL_OK) return 0;
  return (size_t)2 * kQkMaxBlocks * (size_t)d.head_dim * sizeof(float);
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
  const long long xb = qk_span_bytes(d, d.x_ld, d.x_gstride);
  const long long yb = qk_span_bytes(d, d.y_ld, d.y_gstride);
  if (ranges_overlap(x, xb, dx, yb) || (dy != dx && ranges_overlap(dy, yb, dx, yb)))
    return GPTL_E_ARG;
  int sms = 0;
  GPTL_TRY(device_check(&sms));
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  unsigned most = 2u * sms;
  if (most > kQkMaxBlocks) most = kQkMaxBlocks;
  QkParams p = qk_params(d, dy == dx ? 0 : d.v_heads, (int)most * kQkWarps);
  p.x = x;
  p.dy = dy;
  p.out = dx;
  p.gq = gq;
  p.gk = gk;
  p.pos = pos;
  p.table = table;
  p.part = static_cast<float *>(scratch);
  unsigned grid = (p.items + kQkWarps - 1) / kQkWarps;
  if (grid > most) grid = most;
  prof_start(st);
  GPTL_TRY(qk_launch<true>(p, dtype, grid, st));
  if (!gq) return GPTL_OK;
  return launch_reduce_parts(p.part, (int)grid, d.head_dim, 2, dgq, dgk, nullptr, nullptr, st);
}

}  // extern "C"
