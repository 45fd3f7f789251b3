// Bias + dropout + residual, forward and backward, with a mask that is made
// from a counter wherever it is needed and never stored.
//
//   forward   y  = resid + keep (x + bias) / P(keep)
//   backward  dx = keep dy / P(keep),  dbias = column sums of dx
//
// The generator is Philox4x32-10 (J. Salmon, M. Moraes, R. Dror, D. Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", SC 2011): 128 random bits a
// call, of which an element takes 16, so one call serves the 8 elements of a
// 16-byte vector.  (32 bits an element would take two calls a vector, and the
// integer multiplies would bound the backward, which moves 4 bytes an element.)
//
// Bytes: 4 to 10 an element forward, 4 to 6 backward.  A 32-bit residual stream is
// bound by HBM.  16-bit streams are held up by the generator: a warp's vector takes
// about 200 instructions forward and 140 backward, over half of the issue slots, and a
// thread's next rows are loaded only after the present ones are stored.  A warp
// reads 512 contiguous bytes of a row; a thread keeps its 8 columns and walks
// down the rows, so the bias is read once and the bias gradient is summed in
// registers, in the order of the rows.
//
// B200, GPU time (share of the bytes at 6535 GB/s): forward 2048 x 10240 with a 32-bit
// residual 33 us (0.97), 8192 x 2560 fp16 27.2 (0.71), without a residual 24.4 (0.53);
// backward 8192 x 2560 fp16 18.0 us (0.71), with the bias gradient 21.6 (0.59: the second
// kernel and the first one's end), 2048 x 10240 from 32 bits with it 24.7 (0.78); 128 x 128
// 2.5 us, a launch's time.  Two rows in flight a thread at four blocks an SM: with four
// rows the backward spills more (22.7 us), with six blocks too (26.4); as it is, the form
// from 32 bits with the bias gradient spills 16 bytes.
//
// Included by libgptlayer.cu after gptlayer.cu, in the same translation unit.
#pragma once

#include "gptlayer_parts.h"

namespace gptl {

constexpr int kDropRows = 2;            // rows of a thread in flight
constexpr int kDropBlocksPerSm = 4;     // resident (64 registers a thread)

struct DropParams {
  const void *in;                       // x or dy
  const void *bias, *resid;
  void *out;
  float *part;                          // [gridDim.y][h] partial column sums
  const gptl_rng_state *rng;
  int rows, h, lanes;                   // lanes: threads side by side on a row
  unsigned site, drop;                  // drop: D << 16
  float scale;
};

__device__ __forceinline__ uint4 philox4x32_10(uint4 c, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint32_t h0 = __umulhi(0xD2511F53u, c.x), l0 = 0xD2511F53u * c.x;
    const uint32_t h1 = __umulhi(0xCD9E8D57u, c.z), l1 = 0xCD9E8D57u * c.z;
    c = make_uint4(h1 ^ c.y ^ k0, l1, h0 ^ c.w ^ k1, l0);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return c;
}

// f[e] *= scale where element e of block v is kept, 0 where it is dropped
// (selected, not multiplied: a dropped inf or NaN is gone).
__device__ __forceinline__ void drop8(float (&f)[8], const DropParams &p, uint32_t v, ulonglong2 st) {
  if (p.drop == 0) return;
  const uint4 w = philox4x32_10(
      make_uint4(v, p.site, (uint32_t)st.y, (uint32_t)(st.y >> 32)), (uint32_t)st.x,
      (uint32_t)(st.x >> 32));
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = (u[i] << 16) >= p.drop ? f[2 * i] * p.scale : 0.f;
    // the low half cannot lift u over a multiple of 2^16
    f[2 * i + 1] = u[i] >= p.drop ? f[2 * i + 1] * p.scale : 0.f;
  }
}

template <typename T> struct Raw8 { uint4 a; };
template <> struct Raw8<float> { float4 a, b; };

template <typename S>
__device__ __forceinline__ Raw8<S> raw8(const S *p) {
  Raw8<S> r;
  if constexpr (sizeof(S) == 4) {
    r.a = reinterpret_cast<const float4 *>(p)[0];
    r.b = reinterpret_cast<const float4 *>(p)[1];
  } else {
    r.a = *reinterpret_cast<const uint4 *>(p);
  }
  return r;
}
template <typename S, typename T>
__device__ __forceinline__ void raw8_f(const Raw8<S> &r, float (&f)[8]) {
  if constexpr (sizeof(S) == 4) {
    f[0] = r.a.x; f[1] = r.a.y; f[2] = r.a.z; f[3] = r.a.w;
    f[4] = r.b.x; f[5] = r.b.y; f[6] = r.b.z; f[7] = r.b.w;
  } else {
    unpack8<T>(r.a, f);
  }
}
template <typename S, typename T>
__device__ __forceinline__ void put8(S *p, const float (&f)[8]) {
  if constexpr (sizeof(S) == 4) store_vec8_f32(p, 0, f);
  else *reinterpret_cast<uint4 *>(p) = pack8<T>(f);
}

// T: cdt; TR: type of resid (T when there is none); TY: type of y.
template <typename T, typename TR, typename TY>
__global__ void __launch_bounds__(256) dropout_fwd_kernel(const DropParams p) {
  const int team = threadIdx.x / p.lanes, teams = blockDim.x / p.lanes;
  const int cv = blockIdx.x * p.lanes + threadIdx.x % p.lanes;
  if (cv >= p.h / 8) return;
  const T *x = static_cast<const T *>(p.in) + cv * 8;
  const TR *res = static_cast<const TR *>(p.resid) + cv * 8;
  TY *y = static_cast<TY *>(p.out) + cv * 8;
  ulonglong2 st = make_ulonglong2(0, 0);
  if (p.drop) st = make_ulonglong2(p.rng->seed, p.rng->offset);
  float bias[8] = {};
  if (p.bias) unpack8<T>(__ldg(static_cast<const uint4 *>(p.bias) + cv), bias);
  const long long step = (long long)gridDim.y * teams;
  for (long long r0 = (long long)blockIdx.y * teams + team; r0 < p.rows; r0 += kDropRows * step) {
    Raw8<T> xv[kDropRows];
    Raw8<TR> rv[kDropRows] = {};
#pragma unroll
    for (int i = 0; i < kDropRows; ++i) {
      const long long r = r0 + i * step;
      if (r >= p.rows) break;
      xv[i] = raw8<T>(x + r * p.h);
      if (p.resid) rv[i] = raw8<TR>(res + r * p.h);
    }
#pragma unroll
    for (int i = 0; i < kDropRows; ++i) {
      const long long r = r0 + i * step;
      if (r >= p.rows) break;
      float f[8], q[8];
      raw8_f<T, T>(xv[i], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] += bias[e];
      drop8(f, p, (uint32_t)(r * (p.h / 8) + cv), st);
      if (p.resid) {
        raw8_f<TR, T>(rv[i], q);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] += q[e];
      }
      put8<TY, T>(y + r * p.h, f);
    }
  }
}

template <typename T, typename TD, bool SUM>
__global__ void __launch_bounds__(256, kDropBlocksPerSm) dropout_bwd_kernel(const DropParams p) {
  if constexpr (SUM) grid_dependents_launch();
  const int team = threadIdx.x / p.lanes, teams = blockDim.x / p.lanes;
  const int cv = blockIdx.x * p.lanes + threadIdx.x % p.lanes;
  const bool on = cv < p.h / 8;
  const TD *dy = static_cast<const TD *>(p.in) + cv * 8;
  T *dx = static_cast<T *>(p.out) + cv * 8;
  ulonglong2 st = make_ulonglong2(0, 0);
  if (p.drop) st = make_ulonglong2(p.rng->seed, p.rng->offset);
  float acc[8] = {};
  const long long step = (long long)gridDim.y * teams;
  long long r0 = on ? (long long)blockIdx.y * teams + team : (long long)p.rows;
  for (; r0 < p.rows; r0 += kDropRows * step) {
    Raw8<TD> dv[kDropRows];
#pragma unroll
    for (int i = 0; i < kDropRows; ++i) {
      const long long r = r0 + i * step;
      if (r >= p.rows) break;
      dv[i] = raw8<TD>(dy + r * p.h);
    }
#pragma unroll
    for (int i = 0; i < kDropRows; ++i) {
      const long long r = r0 + i * step;
      if (r >= p.rows) break;
      float f[8];
      raw8_f<TD, T>(dv[i], f);
      drop8(f, p, (uint32_t)(r * (p.h / 8) + cv), st);
      if constexpr (SUM) {
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += f[e];
      }
      put8<T, T>(dx + r * p.h, f);
    }
  }
  if constexpr (SUM) {
    // the block's teams, in order; thread t adds columns t, t + 256, ... of the strip
    __shared__ float sm[256 * 8];
    const int width = p.lanes * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) sm[team * width + (threadIdx.x % p.lanes) * 8 + e] = acc[e];
    __syncthreads();
    for (int c = threadIdx.x; c < width; c += blockDim.x) {
      const int col = blockIdx.x * width + c;
      if (col >= p.h) break;
      float s = 0.f;
      for (int t = 0; t < teams; ++t) s += sm[t * width + c];
      p.part[(long long)blockIdx.y * p.h + col] = s;
    }
  }
}

// Adds the partial rows in order: 32 columns and 16 runs of rows a block.
__global__ void __launch_bounds__(512) drop_bias_kernel(const float *__restrict__ part, int splits, int h,
                                                        float *__restrict__ dbias) {
  __shared__ float sm[16][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  float s = 0.f;
  grid_dependency_wait();
  if (c < h) {
#pragma unroll 4
    for (int r = threadIdx.y; r < splits; r += 16) s += part[(long long)r * h + c];
  }
  sm[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && c < h) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += sm[i][threadIdx.x];
    dbias[c] = t;
  }
}

__global__ void rng_advance_kernel(gptl_rng_state *rng, unsigned long long n) { rng->offset += n; }

}  // namespace gptl

namespace {

constexpr int kDropBlocks = kDropBlocksPerSm * 148;   // blocks of a backward with dbias: one wave

// Threads side by side on a row (a power of two, at most a warp), and the
// strips of that many vectors that cover it.
int drop_lanes(int h) {
  int l = 1;
  while (l < 32 && l < h / 8) l *= 2;
  return l;
}

// Row splits of a launch.  With sums, few enough that the partial rows stay
// small beside the data: about kDropBlocks blocks in all.  Without, a split
// for every kDropRows rows of a team.  A function of the sizes alone, so that
// the scratch size is known without a device.
int drop_splits(int rows, int h, bool sums) {
  const int lanes = drop_lanes(h), teams = 256 / lanes;
  const int strips = (h / 8 + lanes - 1) / lanes;
  long long most = ((long long)rows + teams * kDropRows - 1) / (teams * kDropRows);
  if (sums) {
    const long long want = kDropBlocks / strips;
    if (most > want) most = want > 0 ? want : 1;
  }
  return (int)(most > 65535 ? 65535 : most);
}

bool drop_sizes(int rows, int h) {
  return rows > 0 && h > 0 && h % 8 == 0 && (long long)rows * h < (1ll << 35);
}

int check_drop(int rows, int h, gptl_dtype dt, float p, const gptl_rng_state *rng, DropParams *a) {
  if (dt != GPTL_FP16 && dt != GPTL_BF16) return GPTL_E_DTYPE;
  if (!drop_sizes(rows, h)) return GPTL_E_SHAPE;
  if (!(p >= 0.f && p < 1.f)) return GPTL_E_ARG;
  const int d = (int)floor((double)p * 65536.0 + 0.5);
  if (d >= 65536) return GPTL_E_ARG;
  if (d && !rng) return GPTL_E_NULL;
  if (reinterpret_cast<uintptr_t>(rng) & 7u) return GPTL_E_ALIGN;
  a->rng = rng;
  a->rows = rows;
  a->h = h;
  a->lanes = drop_lanes(h);
  a->drop = (unsigned)d << 16;
  a->scale = (float)(65536.0 / (65536 - d));
  return GPTL_OK;
}

}  // namespace

extern "C" {

int gptl_rng_advance(gptl_rng_state *rng, unsigned long long n, gptl_stream_t stream) {
  if (!rng) return GPTL_E_NULL;
  if (reinterpret_cast<uintptr_t>(rng) & 7u) return GPTL_E_ALIGN;
  GPTL_TRY(device_check());
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  prof_start(st);
  rng_advance_kernel<<<1, 1, 0, st>>>(rng, n);
  GPTL_CK(cudaGetLastError());
  prof_launched(st, GPTL_KIND_RNG);
  return GPTL_OK;
}

int gptl_dropout_add_fwd(int rows, int h, gptl_dtype dtype, const void *x, const void *bias,
                         const void *resid, int resid_f32, float p, const gptl_rng_state *rng,
                         unsigned site, void *y, int y_f32, gptl_stream_t stream) {
  if (!x || !y) return GPTL_E_NULL;
  DropParams a{};
  GPTL_TRY(check_drop(rows, h, dtype, p, rng, &a));
  if (!aligned16(x) || !aligned16(bias) || !aligned16(resid) || !aligned16(y)) return GPTL_E_ALIGN;
  if ((resid_f32 != 0 && resid_f32 != 1) || (y_f32 != 0 && y_f32 != 1)) return GPTL_E_ARG;
  const long long n = (long long)rows * h, ny = n * (y_f32 ? 4 : 2);
  if (!(y == x && !y_f32) && ranges_overlap(x, 2 * n, y, ny)) return GPTL_E_ARG;
  if (resid && !(y == resid && y_f32 == resid_f32) &&
      ranges_overlap(resid, n * (resid_f32 ? 4 : 2), y, ny))
    return GPTL_E_ARG;
  if (bias && ranges_overlap(bias, 2ll * h, y, ny)) return GPTL_E_ARG;
  GPTL_TRY(device_check());
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  a.in = x;
  a.bias = bias;
  a.resid = resid;
  a.out = y;
  a.site = site;
  const dim3 grid((h / 8 + a.lanes - 1) / a.lanes, drop_splits(rows, h, false));
  prof_start(st);
  auto go = [&]<typename T>() {
    const bool rf = resid && resid_f32;
    if (rf && y_f32) dropout_fwd_kernel<T, float, float><<<grid, 256, 0, st>>>(a);
    else if (rf) dropout_fwd_kernel<T, float, T><<<grid, 256, 0, st>>>(a);
    else if (y_f32) dropout_fwd_kernel<T, T, float><<<grid, 256, 0, st>>>(a);
    else dropout_fwd_kernel<T, T, T><<<grid, 256, 0, st>>>(a);
  };
  if (dtype == GPTL_FP16) go.template operator()<__half>();
  else go.template operator()<__nv_bfloat16>();
  GPTL_CK(cudaGetLastError());
  prof_launched(st, GPTL_KIND_DROPOUT_FWD);
  return GPTL_OK;
}

size_t gptl_dropout_scratch_bytes(int rows, int h) {
  if (!drop_sizes(rows, h)) return 0;
  return (size_t)drop_splits(rows, h, true) * (size_t)h * sizeof(float);
}

int gptl_dropout_add_bwd(int rows, int h, gptl_dtype dtype, const void *dy, int dy_f32, float p,
                         const gptl_rng_state *rng, unsigned site, void *dx, float *dbias,
                         void *scratch, gptl_stream_t stream) {
  if (!dy || !dx || (dbias && !scratch)) return GPTL_E_NULL;
  DropParams a{};
  GPTL_TRY(check_drop(rows, h, dtype, p, rng, &a));
  if (!aligned16(dy) || !aligned16(dx) || !aligned16(dbias) || (dbias && !aligned16(scratch)))
    return GPTL_E_ALIGN;
  if (dy_f32 != 0 && dy_f32 != 1) return GPTL_E_ARG;
  const long long n = (long long)rows * h;
  if (!(dx == dy && !dy_f32) && ranges_overlap(dy, n * (dy_f32 ? 4 : 2), dx, 2 * n)) return GPTL_E_ARG;
  GPTL_TRY(device_check());
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  a.in = dy;
  a.out = dx;
  a.site = site;
  a.part = static_cast<float *>(scratch);
  const int splits = drop_splits(rows, h, dbias != nullptr);
  const dim3 grid((h / 8 + a.lanes - 1) / a.lanes, splits);
  prof_start(st);
  auto go = [&]<typename T>() {
    auto by_sum = [&]<bool SUM>() {
      if (dy_f32) dropout_bwd_kernel<T, float, SUM><<<grid, 256, 0, st>>>(a);
      else dropout_bwd_kernel<T, T, SUM><<<grid, 256, 0, st>>>(a);
    };
    if (dbias) by_sum.template operator()<true>();
    else by_sum.template operator()<false>();
  };
  if (dtype == GPTL_FP16) go.template operator()<__half>();
  else go.template operator()<__nv_bfloat16>();
  GPTL_CK(cudaGetLastError());
  prof_launched(st, GPTL_KIND_DROPOUT_BWD);
  if (!dbias) return GPTL_OK;
  GPTL_TRY(launch_after(drop_bias_kernel, dim3((h + 31) / 32), dim3(32, 16), st, (const float *)a.part,
                        splits, h, dbias));
  prof_launched(st, GPTL_KIND_REDUCE);
  return GPTL_OK;
}

}  // extern "C"
