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
constexpr int kQkMaxBlocks = 592;       // partial rows of the gains' gradients
constexpr int kQkFwdBlocks = 4, kQkBwdBlocks = 2;              // resident on an SM
constexpr double kQkFwdAngles = 4.0, kQkBwdAngles = 2.0;       // a token's angles, in slots

// The heads of one kind.  A slot is a warp's step: 32/LPH neighbouring heads of
// one group.  A chunk is `spc` slots of the groups * slots of a token.
struct QkKind {
  int heads, first;                     // heads of a group, the first one's place in the row
  int slots, chunks, spc;
  int warps;                            // warps of one chunk: they share its tokens
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
  float eps, inv_hd;
};

// Sines and cosines of one token's pairs, by the whole warp.  Lane c of a head
// holds pairs 8c .. 8c + 7; cs[i * lanes + c] = cosines of its pairs 2i and 2i + 1,
// then their sines, so that the lanes of a head read 16 neighbouring bytes each.
__device__ __forceinline__ void qk_angles(const QkParams &p, int token, float4 *cs, int lanes, int lane) {
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
    float *to = reinterpret_cast<float *>(cs + (j % 8 / 2) * lanes + j / 8) + j % 2;
    to[0] = c;
    to[2] = s;
  }
  __syncwarp();
}

// A lane's 8 pairs (a, b): v0 and v1 hold them as neighbours (INTER) or as the
// vectors of first and of second elements.
template <typename T, bool INTER>
__device__ __forceinline__ void qk_unpack(const uint4 &v0, const uint4 &v1, float (&a)[8],
                                          float (&b)[8]) {
  if constexpr (INTER) {
    const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 q = Cvt<T>::unpack2(w[i]);
      a[i] = q.x;
      b[i] = q.y;
    }
  } else {
    unpack8<T>(v0, a);
    unpack8<T>(v1, b);
  }
}
template <typename T, bool INTER>
__device__ __forceinline__ void qk_pack(const float (&a)[8], const float (&b)[8], uint4 &v0, uint4 &v1) {
  if constexpr (INTER) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = Cvt<T>::pack2(a[i], b[i]);
    v0 = make_uint4(w[0], w[1], w[2], w[3]);
    v1 = make_uint4(w[4], w[5], w[6], w[7]);
  } else {
    v0 = pack8<T>(a);
    v1 = pack8<T>(b);
  }
}

// Turns the pairs (a, b) by (cos, dir * sin) of the lane's table entries.
__device__ __forceinline__ void qk_turn(float (&a)[8], float (&b)[8], const float4 *cs, int lanes,
                                        float dir) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 q = cs[i * lanes];
    const float c[2] = {q.x, q.y}, s[2] = {dir * q.z, dir * q.w};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float x = a[2 * i + e], y = b[2 * i + e];
      a[2 * i + e] = fmaf(x, c[e], -(y * s[e]));
      b[2 * i + e] = fmaf(y, c[e], x * s[e]);
    }
  }
}

// The value heads of the last blocks: a warp copies every v_warps-th row.
template <typename T>
__device__ void qk_copy_values(const QkParams &p, const T *from, long long f_ld, long long f_gs, T *to) {
  const int lane = threadIdx.x & 31;
  const unsigned warps = p.v_blocks * kQkWarps;
  const unsigned rows = (unsigned)p.tokens * p.groups;
  for (unsigned r = (blockIdx.x - p.blocks_qk) * kQkWarps + threadIdx.x / 32; r < rows; r += warps) {
    const unsigned g = r / p.tokens, t = r - g * p.tokens;
    const uint4 *src = reinterpret_cast<const uint4 *>(from + g * f_gs + t * f_ld) + p.v_first;
    uint4 *dst = reinterpret_cast<uint4 *>(to + g * p.y_gs + t * p.y_ld) + p.v_first;
    int i = lane;
    for (; i + 96 < p.v_vecs; i += 128) {
      const uint4 a = src[i], b = src[i + 32], c = src[i + 64], d = src[i + 96];
      dst[i] = a; dst[i + 32] = b; dst[i + 64] = c; dst[i + 96] = d;
    }
    for (; i < p.v_vecs; i += 32) dst[i] = src[i];
  }
}

// BWD: out = dx from x and dy; else out = y from x.  NORM: with gains.
template <typename T, int LPH, bool INTER, bool NORM, bool BWD>
__global__ void __launch_bounds__(kQkWarps * 32, BWD ? kQkBwdBlocks : kQkFwdBlocks)
    qk_rope_kernel(const QkParams p) {
  constexpr int HPW = 32 / LPH;
  constexpr bool kX = NORM || !BWD;                        // x is read
  __shared__ __align__(16) float4 cs_all[kQkWarps][4 * LPH];
  __shared__ __align__(16) float4 gain_all[NORM ? 4 * LPH : 1];   // as cs_all: (a, a, b, b)
  __shared__ float sums[BWD && NORM ? kQkWarps : 1][256];
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
  const int c = lane % LPH, sub = lane / LPH;
  const bool on = c < p.hd / 16, turns = c < p.rot / 16;
  const bool split = turns && !INTER;                      // partners rot/2 apart
  const int v0 = !on ? 0 : split ? 8 * c : 16 * c, v1 = split ? v0 + p.rot / 2 : v0 + 8;

  if constexpr (NORM) {
    if (warp == 0 && lane < LPH) {
      const T *g = static_cast<const T *>(p.gain[key]);
      float ga[8] = {}, gb[8] = {};                        // 0 beyond the head's elements
      if (on)
        qk_unpack<T, INTER>(*reinterpret_cast<const uint4 *>(g + v0),
                            *reinterpret_cast<const uint4 *>(g + v1), ga, gb);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        gain_all[i * LPH + c] = make_float4(ga[2 * i], ga[2 * i + 1], gb[2 * i], gb[2 * i + 1]);
    }
    __syncthreads();
  }
  const float4 *gain = gain_all + c, *cs = cs_all[warp] + c;
  float acc_a[8] = {}, acc_b[8] = {};                      // the gain's gradient

  const int chunk = w / K.warps;
  const int u0 = chunk * K.spc, n_slots = min(K.spc, p.groups * K.slots - u0);
  const int g0 = u0 / K.slots, s0 = u0 - g0 * K.slots;
  const int step = HPW * p.hd, dv = v1 - v0;
  const long long col = (long long)s0 * step + (K.first + sub) * p.hd + v0;
  const long long x_wrap = p.x_gs - (long long)K.slots * step, y_wrap = p.y_gs - (long long)K.slots * step;
  const int h_last = on ? K.heads - sub : 0;               // a head in slot s where s * HPW < h_last
  for (int token = chunk < K.chunks ? w - chunk * K.warps : p.tokens; token < p.tokens;
       token += K.warps) {
    // the next slot to fetch: its number within the group, its places
    int hs = s0 * HPW;
    const T *px = in_x + g0 * p.x_gs + token * p.x_ld + col;
    const T *pd = in_dy + g0 * p.y_gs + token * p.y_ld + col;
    T *po = out + g0 * p.y_gs + token * p.y_ld + col, *o = po;
    uint4 nx0, nx1, nd0, nd1;
    bool live, here;
    auto fetch = [&]() {
      live = hs < h_last;
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
      hs += HPW;
      px += step;
      pd += step;
      po += step;
      if (hs >= K.heads) {
        hs = 0;
        px += x_wrap;
        pd += y_wrap;
        po += y_wrap;
      }
    };
    fetch();
    if (p.rot) qk_angles(p, token, cs_all[warp], LPH, lane);
    for (int u = 0; u < n_slots; ++u) {
      {
        const uint4 x0 = nx0, x1 = nx1, d0 = nd0, d1 = nd1;
        T *to = o;
        here = live;
        if (u + 1 < n_slots) fetch();                      // the next slot's loads go out first
        float a[8], b[8];
        if constexpr (BWD) {
          qk_unpack<T, INTER>(d0, d1, a, b);
          if (turns) qk_turn(a, b, cs, LPH, -1.f);
        }
        if constexpr (NORM) {
          float xa[8], xb[8], ss = 0.f, sd = 0.f;
          qk_unpack<T, INTER>(x0, x1, xa, xb);
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(xa[i], xa[i], fmaf(xb[i], xb[i], ss));
          if constexpr (BWD) {
            // the gain's gradient takes dn x, then dn becomes d = dn g
            float ta[8], tb[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 g = gain[i * LPH];
              const float ga[2] = {g.x, g.y}, gb[2] = {g.z, g.w};
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int k = 2 * i + e;
                ta[k] = a[k] * xa[k];
                tb[k] = b[k] * xb[k];
                sd = fmaf(ta[k], ga[e], fmaf(tb[k], gb[e], sd));
                a[k] *= ga[e];
                b[k] *= gb[e];
              }
            }
#pragma unroll
            for (int o2 = LPH / 2; o2 > 0; o2 >>= 1) {
              ss += __shfl_xor_sync(0xffffffffu, ss, o2);
              sd += __shfl_xor_sync(0xffffffffu, sd, o2);
            }
            const float r = rsqrtf(fmaf(ss, p.inv_hd, p.eps));
            const float m = -r * r * r * (sd * p.inv_hd);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              acc_a[k] = fmaf(ta[k], r, acc_a[k]);
              acc_b[k] = fmaf(tb[k], r, acc_b[k]);
              a[k] = fmaf(a[k], r, xa[k] * m);
              b[k] = fmaf(b[k], r, xb[k] * m);
            }
          } else {
#pragma unroll
            for (int o2 = LPH / 2; o2 > 0; o2 >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o2);
            const float r = rsqrtf(fmaf(ss, p.inv_hd, p.eps));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 g = gain[i * LPH];
              a[2 * i] = xa[2 * i] * r * g.x;
              a[2 * i + 1] = xa[2 * i + 1] * r * g.y;
              b[2 * i] = xb[2 * i] * r * g.z;
              b[2 * i + 1] = xb[2 * i + 1] * r * g.w;
            }
          }
        } else if constexpr (!BWD) {
          qk_unpack<T, INTER>(x0, x1, a, b);
        }
        if (!BWD && turns) qk_turn(a, b, cs, LPH, 1.f);
        if (here) {
          uint4 q0, q1;
          qk_pack<T, INTER>(a, b, q0, q1);
          *reinterpret_cast<uint4 *>(to) = q0;
          *reinterpret_cast<uint4 *>(to + dv) = q1;
        }
      }
    }
  }
  if constexpr (BWD && NORM) {
    // the warp's head positions, then the block's warps, each in a fixed order
    float f[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {                          // in the order of v0 and v1
      f[INTER ? 2 * i : i] = acc_a[i];
      f[INTER ? 2 * i + 1 : 8 + i] = acc_b[i];
    }
#pragma unroll
    for (int o = LPH; o < 32; o <<= 1)
#pragma unroll
      for (int i = 0; i < 16; ++i) f[i] += __shfl_xor_sync(0xffffffffu, f[i], o);
    if (lane < LPH && on)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sums[warp][v0 + i] = f[i];
        sums[warp][v1 + i] = f[8 + i];
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
  if (heads > (1 << 20) || rows >= (1ll << 30)) return GPTL_E_SHAPE;
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

// Sizes, and the split of the work over `blocks` resident blocks.  Queries and
// keys get blocks of their own, in proportion to their slots (a token's angles
// cost `angles` of them), so that a warp keeps one gain and its gradient in
// registers.  A token's slots go to one warp, or in chunks to several where
// that evens out the tokens of a warp: the number of chunks is the one with
// the shortest longest warp.  Value heads come in blocks behind the others:
// with or without them, the sums have one order.
QkParams qk_params(const gptl_qk_desc &d, int v_heads, int blocks, double angles) {
  QkParams p{};
  const int hpw = 32 / qk_lanes(d.head_dim);
  const int heads[2] = {d.q_heads, d.k_heads};
  if (d.rot_dim == 0) angles = 0.25;
  double weight[2];
  for (int i = 0; i < 2; ++i) {
    QkKind &k = p.kind[i];
    k.heads = heads[i];
    k.first = i ? d.q_heads : 0;
    k.slots = (heads[i] + hpw - 1) / hpw;
    weight[i] = angles + (double)k.slots * d.groups;
  }
  for (int i = 0; i < 2; ++i) {
    QkKind &k = p.kind[i];
    const int all = k.slots * d.groups;
    long long nb = (long long)(blocks * weight[i] / (weight[0] + weight[1]));
    const long long most = ((long long)d.tokens * all + kQkWarps - 1) / kQkWarps;
    if (nb > most) nb = most;
    if (nb < 1) nb = 1;
    const long long warps = nb * kQkWarps;
    double best = 0;
    k.chunks = 0;
    for (int c = 1; c <= all && c <= warps && c <= 64; ++c) {
      const int spc = (all + c - 1) / c;
      if (c > 1 && spc == k.spc) continue;                 // the same chunks, some of them empty
      const long long each = warps / c;
      const double longest = (double)((d.tokens + each - 1) / each) * (angles + (double)spc);
      if (!k.chunks || longest < best) {
        best = longest;
        k.spc = spc;
        k.chunks = (all + spc - 1) / spc;
      }
    }
    k.warps = (int)(warps / k.chunks);
    if (i == 0) p.blocks_q = (int)nb;
    else p.blocks_qk = p.blocks_q + (int)nb;
  }
  p.v_vecs = v_heads * d.head_dim / 8;
  p.v_first = (d.q_heads + d.k_heads) * d.head_dim / 8;
  if (v_heads) {
    const long long rows = (long long)d.tokens * d.groups, want = 8ll * blocks;
    const long long nb = (rows + kQkWarps - 1) / kQkWarps;
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
  int rc = GPTL_OK;
  auto run = [&]<typename T, int LPH, bool INTER, bool NORM>() {
    auto kern = qk_rope_kernel<T, LPH, INTER, NORM, BWD>;
    kern<<<grid, kQkWarps * 32, 0, st>>>(p);
  };
  auto go = [&]<typename T, int LPH, bool INTER>() {
    if (norm) run.template operator()<T, LPH, INTER, true>();
    else run.template operator()<T, LPH, INTER, false>();
  };
  auto by_pairs = [&]<typename T, int LPH>() {
    if (interleaved) go.template operator()<T, LPH, true>();
    else go.template operator()<T, LPH, false>();
  };
  auto by_lanes = [&]<typename T>() {
    switch (qk_lanes(p.hd)) {
      case 1: by_pairs.template operator()<T, 1>(); break;
      case 2: by_pairs.template operator()<T, 2>(); break;
      case 4: by_pairs.template operator()<T, 4>(); break;
      case 8: by_pairs.template operator()<T, 8>(); break;
      default: by_pairs.template operator()<T, 16>(); break;
    }
  };
  if (dt == GPTL_FP16) by_lanes.template operator()<__half>();
  else by_lanes.template operator()<__nv_bfloat16>();
  GPTL_TRY(rc);
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
  QkParams p = qk_params(d, in_place ? 0 : d.v_heads, sms * kQkFwdBlocks, kQkFwdAngles);
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
  int most = sms * kQkBwdBlocks;
  if (most > kQkMaxBlocks) most = kQkMaxBlocks;
  QkParams p = qk_params(d, dy == dx ? 0 : d.v_heads, most, kQkBwdAngles);
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
  qk_gain_kernel<<<dim3((d.head_dim + 31) / 32, 2), dim3(32, 16), 0, st>>>(
      p.part, p.blocks_q, p.blocks_qk, d.head_dim, dgq, dgk);
  GPTL_CK(cudaGetLastError());
  prof_launched(st, GPTL_KIND_REDUCE);
  return GPTL_OK;
}

}  // extern "C"
