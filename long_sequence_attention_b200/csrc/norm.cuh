// Root-mean-square norm of a block's rows, with the residual's addition and bf16, fp32 or
// scaled E4M3 output.
//
// For each row, over its C columns,
//     h = x + r (r = 0 without a residual),  y = h * w / sqrt(mean(h^2) + eps),
// the stream h is rounded once to its type for the next layer, and y is rounded once from the
// unrounded fp32 h (so the norm does not see the stream's rounding).  E4M3 output follows the
// quantisers' rule per group of columns (a whole row, or 128 columns):
//     descale = max |y| / 448 (1 if the maximum is below 2^-119),  code = e4m3_rn_satfinite(y / descale).
//
// Bytes bound: each element is read once (x, r) and written once (h, y).  So a row stays in registers
// between the sum and the output: a CTA per row (or, up to 128 pieces of 16 bytes, 8 to 32 lanes of
// a warp), NV 16-byte pieces a thread.  Rows that are not whole aligned 16-byte pieces are held as
// single elements; rows too long for the registers are read again from the caches instead.  B200, rows of
// 5120 bf16 with a residual, 32760 of them: 172 us to E4M3 with a scale every 128 columns (6.8 TB/s), 197 us
// to bf16 (6.8 TB/s); one such row 2.2 us; 40000 rows of 1000 to bf16 50 us, of 1001 (single elements) 99 us.
#pragma once

#include <cuda_bf16.h>

#include "ptx.cuh"
#include "quant.cuh"

namespace dit {

// Groups whose largest magnitude is below this count as zeros: 448 over it would leave fp32's range.
constexpr float kE4m3Least = 1.504632769052528e-36f;   // 2^-119

struct NormParams {
  const void* x;
  long long x_stride;        // elements between rows of x; every other tensor is dense
  const void* residual;      // or null
  const void* weight;        // [C] or null (ones)
  void* out;
  void* stream_out;          // h in the input type, or null
  float* descales;           // E4M3: [rows, groups]
  long long rows;
  int C;
  int group;                 // E4M3: columns of one scale (C or 128)
  float eps;
};

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ void from_f32(float v, __nv_bfloat16& o) { o = __float2bfloat16(v); }
__device__ __forceinline__ void from_f32(float v, float& o) { o = v; }

__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0f;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) v += red[w];
  return v;
}

// A 16-byte piece of a row as fp32 values, and back.
template <typename T>
struct NormVec;
template <>
struct NormVec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void unpack(const uint4& a, float (&v)[8]) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[8]) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
};
template <>
struct NormVec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void unpack(const uint4& a, float (&v)[4]) {
    v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y); v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
};

// N results to the output row at element e: bf16, fp32 (OUT 0, 1) or E4M3 codes of y / d (OUT 2), the quotient taken as
// y times 448 / max |y| (rcp), correctly rounded: y carries roundings of that size anyhow.
template <int OUT, int N>
__device__ __forceinline__ void norm_store(void* out, long long e, const float (&y)[N], float rcp) {
  if constexpr (OUT == 0) {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) w[i] = pack_bf16x2(y[2 * i], y[2 * i + 1]);
    if constexpr (N == 8)
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out) + e) = make_uint4(w[0], w[1], w[2], w[3]);
    else
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + e) = make_uint2(w[0], w[1]);
  } else if constexpr (OUT == 1) {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      *reinterpret_cast<float4*>(static_cast<float*>(out) + e + i) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint32_t c = pack_e4m3x4(y[i] * rcp, y[i + 1] * rcp, y[i + 2] * rcp, y[i + 3] * rcp);
      *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(out) + e + i) = c;
    }
  }
}

constexpr int kNormMaxVecs = 4096;         // 512 threads of 8 pieces
constexpr int kNormWarpVecs = 128;         // a warp of 4 pieces

// LANES > 0: a row on LANES lanes of a warp (256 threads, 256 / LANES rows a CTA); LANES = 0: a row on the CTA.
// Thread i of the row's group holds pieces i, i + width, ...: 128 columns are 16 (bf16) or 32 (fp32) neighbouring
// lanes, so a scale of 128 columns is a few shuffles.
template <typename T, int OUT, int NV, int LANES>
__global__ void __launch_bounds__(LANES ? 256 : (NV <= 2 ? 1024 : 512), LANES || NV != 4 ? 1 : 2) rms_norm_vec_kernel(const NormParams p) {
  using V = NormVec<T>;
  constexpr int N = V::kN;
  __shared__ float red[2][33];
  const int lane = threadIdx.x & 31;
  const int width = LANES ? LANES : blockDim.x;
  const int at = LANES ? static_cast<int>(threadIdx.x) % (LANES ? LANES : 1) : static_cast<int>(threadIdx.x);
  const long long row = LANES ? blockIdx.x * (256LL / (LANES ? LANES : 1)) + threadIdx.x / (LANES ? LANES : 1) : blockIdx.x;
  const bool on = row < p.rows;
  const int nvec = p.C / N;
  const T* x = static_cast<const T*>(p.x) + row * p.x_stride;
  const long long base = row * p.C;
  const T* r = static_cast<const T*>(p.residual) + (p.residual ? base : 0);
  const T* w = static_cast<const T*>(p.weight);
  uint4 xv[NV], rv[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = at + i * width;
    xv[i] = rv[i] = make_uint4(0u, 0u, 0u, 0u);
    if (on && v < nvec) {
      xv[i] = *reinterpret_cast<const uint4*>(x + v * N);
      if (p.residual) rv[i] = *reinterpret_cast<const uint4*>(r + v * N);
    }
  }
  float h[NV][N];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float a[N], b[N];
    V::unpack(xv[i], a);
    V::unpack(rv[i], b);
#pragma unroll
    for (int e = 0; e < N; ++e) {
      h[i][e] = a[e] + b[e];
      ss = fmaf(h[i][e], h[i][e], ss);
    }
    const int v = at + i * width;
    if (p.stream_out && on && v < nvec)
      *reinterpret_cast<uint4*>(static_cast<T*>(p.stream_out) + base + v * N) = V::pack(h[i]);
  }
#pragma unroll
  for (int o = (LANES ? LANES : 32) / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if constexpr (LANES == 0) {
    const int nw = blockDim.x >> 5;
    if (nw > 1) {
      if (lane == 0) red[0][threadIdx.x >> 5] = ss;
      __syncthreads();
      ss = lane < nw ? red[0][lane] : 0.0f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
  }
  const float inv = __frsqrt_rn(ss / static_cast<float>(p.C) + p.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = at + i * width;
    if (w) {
      float b[N];
      V::unpack(v < nvec ? __ldg(reinterpret_cast<const uint4*>(w + v * N)) : make_uint4(0u, 0u, 0u, 0u), b);
#pragma unroll
      for (int e = 0; e < N; ++e) h[i][e] = h[i][e] * inv * b[e];
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) h[i][e] *= inv;
    }
  }
  float d = 1.0f, rcp = 1.0f;
  if (OUT == 2 && p.group == p.C) {              // one scale a row
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (at + i * width < nvec) m = fmaxf(m, fabsf(h[i][e]));
#pragma unroll
    for (int o = (LANES ? LANES : 32) / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if constexpr (LANES == 0) {
      const int nw = blockDim.x >> 5;
      if (nw > 1) {
        if (lane == 0) red[1][threadIdx.x >> 5] = m;
        __syncthreads();
        m = lane < nw ? red[1][lane] : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      }
    }
    d = m >= kE4m3Least ? __fdiv_rn(m, 448.0f) : 1.0f;
    rcp = m >= kE4m3Least ? __fdiv_rn(448.0f, m) : 1.0f;
    if (on && at == 0) p.descales[row] = d;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = at + i * width;
    if (OUT == 2 && p.group != p.C) {            // one scale every 128 columns
      constexpr int kGroup = 128 / N;
      float m = 0.0f;
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (v < nvec) m = fmaxf(m, fabsf(h[i][e]));
#pragma unroll
      for (int o = (LANES && LANES < kGroup ? LANES : kGroup) / 2; o > 0; o >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      d = m >= kE4m3Least ? __fdiv_rn(m, 448.0f) : 1.0f;
      rcp = m >= kE4m3Least ? __fdiv_rn(448.0f, m) : 1.0f;
      if (on && v < nvec && v % kGroup == 0) p.descales[row * ((p.C + 127) / 128) + v / kGroup] = d;
    }
    if (on && v < nvec) norm_store<OUT, N>(p.out, base + v * N, h[i], rcp);
  }
}

// Any alignment and width up to 128 * NG * 32 columns: a CTA per row, each warp NG runs of 128 columns, four elements
// of a run a lane (32 apart, so that a warp's accesses are dense); a scale of 128 columns is a warp's.
template <typename T, int OUT, int NG>
__global__ void __launch_bounds__(1024) rms_norm_cols_kernel(const NormParams p) {
  __shared__ float red[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const long long row = blockIdx.x, base = row * p.C;
  const T* x = static_cast<const T*>(p.x) + row * p.x_stride;
  const T* r = static_cast<const T*>(p.residual) + (p.residual ? base : 0);
  const T* w = static_cast<const T*>(p.weight);
  float h[NG][4], wv[NG][4];
  float ss = 0.0f;
#pragma unroll
  for (int g = 0; g < NG; ++g)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = (warp + g * nw) * 128 + e * 32 + lane;
      h[g][e] = 0.0f;
      wv[g][e] = 1.0f;
      if (c < p.C) {
        h[g][e] = to_f32(x[c]) + (p.residual ? to_f32(r[c]) : 0.0f);
        if (w) wv[g][e] = to_f32(w[c]);
      }
      ss = fmaf(h[g][e], h[g][e], ss);
    }
#pragma unroll
  for (int g = 0; g < NG; ++g)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = (warp + g * nw) * 128 + e * 32 + lane;
      if (p.stream_out && c < p.C) from_f32(h[g][e], static_cast<T*>(p.stream_out)[base + c]);
    }
  const float inv = __frsqrt_rn(block_sum(ss, red[0]) / static_cast<float>(p.C) + p.eps);
  float m[NG], row_m = 0.0f;
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    m[g] = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      h[g][e] = h[g][e] * inv * wv[g][e];
      m[g] = fmaxf(m[g], (warp + g * nw) * 128 + e * 32 + lane < p.C ? fabsf(h[g][e]) : 0.0f);
    }
    row_m = fmaxf(row_m, m[g]);
  }
  float d = 1.0f, rcp = 1.0f;
  if (OUT == 2 && p.group == p.C) {
    row_m = block_max(row_m, red[1]);
    d = row_m >= kE4m3Least ? __fdiv_rn(row_m, 448.0f) : 1.0f;
    rcp = row_m >= kE4m3Least ? __fdiv_rn(448.0f, row_m) : 1.0f;
    if (threadIdx.x == 0) p.descales[row] = d;
  }
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const int c0 = (warp + g * nw) * 128;
    if (OUT == 2 && p.group != p.C) {
      float a = m[g];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
      d = a >= kE4m3Least ? __fdiv_rn(a, 448.0f) : 1.0f;
      rcp = a >= kE4m3Least ? __fdiv_rn(448.0f, a) : 1.0f;
      if (lane == 0 && c0 < p.C) p.descales[row * ((p.C + 127) / 128) + c0 / 128] = d;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = c0 + e * 32 + lane;
      if (c >= p.C) continue;
      if constexpr (OUT == 0) static_cast<__nv_bfloat16*>(p.out)[base + c] = __float2bfloat16(h[g][e]);
      else if constexpr (OUT == 1) static_cast<float*>(p.out)[base + c] = h[g][e];
      else static_cast<uint8_t*>(p.out)[base + c] = static_cast<uint8_t>(pack_e4m3x2(h[g][e] * rcp, 0.0f) & 0xFFu);
    }
  }
}

constexpr int kNormThreads = 256;

// One CTA per row, the row read twice (the second time from L1 / L2).
// OUT: 0 = bf16, 1 = fp32, 2 = E4M3.
template <typename T, int OUT>
__global__ void __launch_bounds__(kNormThreads) rms_norm_kernel(const NormParams p) {
  __shared__ float red[kNormThreads / 32];
  const T* w = static_cast<const T*>(p.weight);
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + row * p.x_stride;
    const T* r = p.residual ? static_cast<const T*>(p.residual) + row * p.C : nullptr;
    T* so = p.stream_out ? static_cast<T*>(p.stream_out) + row * p.C : nullptr;
    auto h_at = [&](int c) { return to_f32(x[c]) + (r ? to_f32(r[c]) : 0.0f); };
    float ss = 0.0f;
    for (int c = threadIdx.x; c < p.C; c += kNormThreads) {
      const float h = h_at(c);
      ss = fmaf(h, h, ss);
    }
    const float inv = __frsqrt_rn(block_sum(ss, red) / static_cast<float>(p.C) + p.eps);
    auto y_at = [&](int c) { return h_at(c) * inv * (w ? to_f32(w[c]) : 1.0f); };
    const long long base = row * p.C;
    if constexpr (OUT == 2) {
      const int ng = (p.C + p.group - 1) / p.group;
      for (int g = 0; g < ng; ++g) {
        const int c1 = min(p.C, (g + 1) * p.group);
        float m = 0.0f;
        for (int c = g * p.group + threadIdx.x; c < c1; c += kNormThreads) m = fmaxf(m, fabsf(y_at(c)));
        const float amax = block_max(m, red);
        const float d = amax >= kE4m3Least ? __fdiv_rn(amax, 448.0f) : 1.0f;
        if (threadIdx.x == 0) p.descales[row * ng + g] = d;
        for (int c = g * p.group + threadIdx.x; c < c1; c += kNormThreads)
          static_cast<uint8_t*>(p.out)[base + c] =
              static_cast<uint8_t>(pack_e4m3x2(__fdiv_rn(y_at(c), d), 0.0f) & 0xFFu);
      }
    } else {
      for (int c = threadIdx.x; c < p.C; c += kNormThreads) {
        if constexpr (OUT == 1) static_cast<float*>(p.out)[base + c] = y_at(c);
        else static_cast<__nv_bfloat16*>(p.out)[base + c] = __float2bfloat16(y_at(c));
      }
    }
    __syncthreads();   // the stream may overwrite x or r in place: only after every read of them
    if (so)
      for (int c = threadIdx.x; c < p.C; c += kNormThreads) {
        const float h = h_at(c);
        from_f32(h, so[c]);
      }
    __syncthreads();
  }
}

}  // namespace dit
