// Root-mean-square norm of a block's rows, with the residual's addition and bf16, fp32 or
// scaled E4M3 output.
//
// For each row, over its C columns,
//     h = x + r (r = 0 without a residual),  y = h * w / sqrt(mean(h^2) + eps),
// the stream h is rounded once to its type for the next layer, and y is rounded once from the
// unrounded fp32 h (so the norm does not see the stream's rounding).  E4M3 output follows the
// quantisers' rule per group of columns (a whole row, or 128 columns):
//     descale = max |y| / 448 (1 if the maximum is 0),  code = e4m3_rn_satfinite(y / descale).
//
// Bytes bound: each element is read once (x, r) and written once (h, y).
#pragma once

#include <cuda_bf16.h>

#include "ptx.cuh"
#include "quant.cuh"

namespace dit {

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
    const float inv = rsqrtf(block_sum(ss, red) / static_cast<float>(p.C) + p.eps);
    auto y_at = [&](int c) { return h_at(c) * inv * (w ? to_f32(w[c]) : 1.0f); };
    const long long base = row * p.C;
    if constexpr (OUT == 2) {
      const int ng = (p.C + p.group - 1) / p.group;
      for (int g = 0; g < ng; ++g) {
        const int c1 = min(p.C, (g + 1) * p.group);
        float m = 0.0f;
        for (int c = g * p.group + threadIdx.x; c < c1; c += kNormThreads) m = fmaxf(m, fabsf(y_at(c)));
        const float amax = block_max(m, red);
        const float d = amax > 0.0f ? __fdiv_rn(amax, 448.0f) : 1.0f;
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
