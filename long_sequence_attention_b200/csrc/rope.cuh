// Rotary positions of queries and keys, with their per-head root-mean-square norm, read from
// the projection's token-major output and written head-major for the attention kernels, in
// bf16 or as the E4M3 128-row blocks of the block-scaled attention.
//
// Pair i of a head's first `rot` elements (neighbours (2i, 2i+1), or (i, i + rot/2)) turns by
// the angle position * freq_i:
//     (a, b) -> magnitude * (a cos - b sin, b cos + a sin);  elements past rot pass unchanged.
// Each pair belongs to one position axis (1 for text, up to 3 for t, y, x grids).
//
// Angles in whole turns, 64-bit fixed point: F = freq / 2 pi * 2^64 mod 2^64, and position * F
// in 64-bit integer arithmetic drops whole turns exactly, so far positions lose nothing; the
// top 32 bits are the angle in units of 2^-32 turns, and sincospi takes it from there.
//
// Bytes bound: q and k are read once and written once.
#pragma once

#include <cuda_bf16.h>

#include "norm.cuh"
#include "ptx.cuh"
#include "quant.cuh"

namespace dit {

constexpr int kMaxRopeAxes = 3;

struct RopeParams {
  const __nv_bfloat16* x[2];            // q, k
  long long sb[2], ss[2], sh[2];        // element strides of batch, token, head (D is dense)
  void* out[2];                         // [B, heads, S, D]
  float* descales[2];                   // E4M3: [B, heads, ceil(S / 128)]
  const __nv_bfloat16* weight[2];       // [D], or null: no norm
  int heads[2];
  const int* pos;                       // [B or 1, S, axes]
  long long pos_sb;                     // elements between batches of pos (0: shared)
  const double* freqs;                  // [rot / 2] radians per position
  int axes;
  int axis_end[kMaxRopeAxes];           // pairs [axis_end[a - 1], axis_end[a]) belong to axis a
  int B, S, D, rot;
  int interleaved;
  float eps, magnitude;
};

// 2^64 times a frequency in turns per position, whole turns dropped (any finite frequency).
__device__ __forceinline__ unsigned long long rope_turns(double freq) {
  const double t = freq * 0.15915494309189535;                  // turns per position
  const double f = t - floor(t);                                // exact; in [0, 1]
  return f < 1.0 ? __double2ull_rz(f * 18446744073709551616.0) : 0ull;
}

__device__ __forceinline__ void rope_cos_sin(int pos, unsigned long long turns, float magnitude, float& c, float& s) {
  const unsigned long long t = static_cast<unsigned long long>(static_cast<long long>(pos)) * turns;
  const int hi = static_cast<int>(t >> 32);                     // the fraction of a turn, in [-1/2, 1/2) * 2^32
  sincospif(static_cast<float>(hi) * 4.6566128730773926e-10f, &s, &c);   // 2^-31: half turns
  c *= magnitude;
  s *= magnitude;
}

// One head row by one warp: load, norm, rotate; the D results in y (shared memory of the warp).
__device__ __forceinline__ void rope_row(const RopeParams& p, int which, long long b, int h, int s, float* row,
                                         float* y) {
  const int lane = threadIdx.x & 31;
  const __nv_bfloat16* x = p.x[which] + b * p.sb[which] + s * p.ss[which] + h * p.sh[which];
  float ssum = 0.0f;
  for (int d = lane; d < p.D; d += 32) {
    const float v = __bfloat162float(x[d]);
    row[d] = v;
    ssum = fmaf(v, v, ssum);
  }
  if (p.weight[which] != nullptr) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ssum += __shfl_xor_sync(0xffffffffu, ssum, o);
    const float inv = rsqrtf(ssum / p.D + p.eps);
    for (int d = lane; d < p.D; d += 32) row[d] *= inv * __bfloat162float(p.weight[which][d]);
  }
  __syncwarp();
  const int* pos = p.pos + b * p.pos_sb + static_cast<long long>(s) * p.axes;
  const int pairs = p.rot / 2;
  for (int i = lane; i < pairs; i += 32) {
    int axis = 0;
    while (axis + 1 < p.axes && i >= p.axis_end[axis]) ++axis;
    float c, sn;
    rope_cos_sin(pos[axis], rope_turns(p.freqs[i]), p.magnitude, c, sn);
    const int ia = p.interleaved ? 2 * i : i, ib = p.interleaved ? 2 * i + 1 : i + pairs;
    const float a = row[ia], bb = row[ib];
    y[ia] = a * c - bb * sn;
    y[ib] = bb * c + a * sn;
  }
  for (int d = p.rot + lane; d < p.D; d += 32) y[d] = row[d];
  __syncwarp();
}

constexpr int kRopeWarps = 8;
constexpr int kRopeBlockRows = 128;
constexpr int kRopeSmem = (kRopeWarps + kRopeBlockRows) * 128 * 4;

// One CTA per 128 tokens of one head of q or k: its rows in shared memory, then bf16 out, or
// their absolute maximum and the E4M3 codes.
template <bool E4M3>
__global__ void __launch_bounds__(32 * kRopeWarps) rope_kernel(const RopeParams p) {
  extern __shared__ float sm[];
  __shared__ float red[kRopeWarps];
  const int warp = threadIdx.x >> 5;
  float* row = sm + warp * 128;
  float* y = sm + kRopeWarps * 128;
  const int nblk = (p.S + kRopeBlockRows - 1) / kRopeBlockRows;
  const int heads = p.heads[0] + p.heads[1];
  const int blk = blockIdx.x % nblk;
  const int hh = static_cast<int>((blockIdx.x / nblk) % heads);
  const long long b = blockIdx.x / nblk / heads;
  const int which = hh >= p.heads[0];
  const int h = which ? hh - p.heads[0] : hh;
  const int s0 = blk * kRopeBlockRows, rows = min(kRopeBlockRows, p.S - s0);
  for (int i = warp; i < rows; i += kRopeWarps) rope_row(p, which, b, h, s0 + i, row, y + i * p.D);
  __syncthreads();
  const long long bh = b * p.heads[which] + h;
  const long long base = (bh * p.S + s0) * p.D;
  const int n = rows * p.D;
  if constexpr (E4M3) {
    float m = 0.0f;
    for (int i = threadIdx.x; i < n; i += blockDim.x) m = fmaxf(m, fabsf(y[i]));
    const float amax = block_max(m, red);
    const float d = amax > 0.0f ? __fdiv_rn(amax, 448.0f) : 1.0f;
    if (threadIdx.x == 0) p.descales[which][bh * nblk + blk] = amax > 0.0f ? d : 0.0f;
    for (int i = threadIdx.x; i < n; i += blockDim.x)
      static_cast<uint8_t*>(p.out[which])[base + i] =
          static_cast<uint8_t>(pack_e4m3x2(__fdiv_rn(y[i], d), 0.0f) & 0xFFu);
  } else {
    for (int i = threadIdx.x; i < n; i += blockDim.x)
      static_cast<__nv_bfloat16*>(p.out[which])[base + i] = __float2bfloat16(y[i]);
  }
}

}  // namespace dit
