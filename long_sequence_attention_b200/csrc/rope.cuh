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
// Bytes bound: q and k are read once and written once.  Eight elements a lane, 16 (D = 128) or 8 lanes a head
// row; a lane's eight are four whole pairs in either layout (two runs of four, half the rotated part
// apart, in the half layout), so nothing crosses lanes but the norm's sum.  A thread keeps its token and walks over
// heads, so the angles are formed once for many heads.
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

// cos and sin of position * freq times the magnitude.  The nearest quarter turn is taken off in integers
// first, so that the rest, at most an eighth of a turn, keeps more of its bits in fp32.
__device__ __forceinline__ void rope_cos_sin(int pos, unsigned long long turns, float magnitude, float& c, float& s) {
  const unsigned long long t = static_cast<unsigned long long>(static_cast<long long>(pos)) * turns;
  const uint32_t hi = static_cast<uint32_t>(t >> 32);           // in 2^-32 turns
  const uint32_t quarter = (hi + 0x20000000u) >> 30;
  const int rest = static_cast<int>(hi - (quarter << 30));      // in [-2^29, 2^29)
  float cr, sr;
  sincospif(static_cast<float>(rest) * 4.6566128730773926e-10f, &sr, &cr);   // 2^-31: half turns
  const float x = (quarter & 1u) ? sr : cr, y = (quarter & 1u) ? cr : sr;
  c = ((quarter + 1u) & 2u) ? -x * magnitude : x * magnitude;
  s = (quarter & 2u) ? -y * magnitude : y * magnitude;
}

// A lane's part of a head: elements lo .. lo + 3 and hi .. hi + 3; pairs 4 lane .. 4 lane + 3.
struct RopeLane {
  int lo, hi;
  bool split;                    // half layout, inside the rotated part: two 8-byte accesses
  bool turn[4];                  // pair k is rotated
  float c[4], s[4];
};

template <int D, bool INTER>
__device__ __forceinline__ RopeLane rope_lane(const RopeParams& p, int lane, const int* pos, bool on) {
  RopeLane r;
  const int pairs = p.rot / 2;
  r.split = !INTER && lane * 4 < pairs;
  r.lo = r.split ? 4 * lane : 8 * lane;
  r.hi = r.split ? 4 * lane + pairs : 8 * lane + 4;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int i = 4 * lane + k;
    r.turn[k] = i < pairs;
    r.c[k] = 1.0f;
    r.s[k] = 0.0f;
    if (on && r.turn[k]) {
      int axis = 0;
#pragma unroll
      for (int a = 0; a + 1 < kMaxRopeAxes; ++a)
        if (a + 1 < p.axes && i >= p.axis_end[a]) axis = a + 1;
      rope_cos_sin(__ldg(pos + axis), rope_turns(__ldg(p.freqs + i)), p.magnitude, r.c[k], r.s[k]);
    }
  }
  return r;
}

template <bool INTER>
__device__ __forceinline__ uint4 rope_load(const __nv_bfloat16* x, const RopeLane& r) {
  if (INTER) return __ldg(reinterpret_cast<const uint4*>(x + r.lo));
  const uint2 a = __ldg(reinterpret_cast<const uint2*>(x + r.lo)), b = __ldg(reinterpret_cast<const uint2*>(x + r.hi));
  return make_uint4(a.x, a.y, b.x, b.y);
}

// Norm (where w is given) and rotation of a lane's eight elements.
template <int D, bool INTER>
__device__ __forceinline__ void rope_apply(const RopeLane& r, const uint4& raw, bool norm, const float (&w)[8], float eps,
                                           float (&y)[8]) {
  float v[8];
  NormVec<__nv_bfloat16>::unpack(raw, v);
  if (norm) {
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
#pragma unroll
    for (int o = D / 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float inv = __frsqrt_rn(ss * (1.0f / D) + eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] * inv * w[i];
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int ia = INTER ? 2 * k : k, ib = INTER ? 2 * k + 1 : k + 4;
    if (INTER) {
      const float a = v[ia], b = v[ib];
      y[ia] = r.turn[k] ? a * r.c[k] - b * r.s[k] : a;
      y[ib] = r.turn[k] ? b * r.c[k] + a * r.s[k] : b;
    } else {
      const float a = v[ia], b = v[ib];
      y[ia] = r.split ? a * r.c[k] - b * r.s[k] : a;
      y[ib] = r.split ? b * r.c[k] + a * r.s[k] : b;
    }
  }
}

__device__ __forceinline__ void rope_weights(const __nv_bfloat16* w, const RopeLane& r, float (&v)[8]) {
  if (w == nullptr) return;
  const uint2 a = __ldg(reinterpret_cast<const uint2*>(w + r.lo)), b = __ldg(reinterpret_cast<const uint2*>(w + r.hi));
  NormVec<__nv_bfloat16>::unpack(make_uint4(a.x, a.y, b.x, b.y), v);
}

// bf16 out.  A CTA takes 256 * 8 / D tokens (of all batches, one after another) and heads_per heads of q and k
// together; four heads' loads are in flight at a time.
constexpr int kRopeThreads = 256;
constexpr int kRopeUnroll = 4;

template <int D, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p, int heads_per) {
  constexpr int kLanes = D / 8;
  const long long n = static_cast<long long>(blockIdx.x) * (kRopeThreads / kLanes) + threadIdx.x / kLanes;
  const bool on = n < static_cast<long long>(p.B) * p.S;
  const long long b = on ? n / p.S : 0;
  const int s = on ? static_cast<int>(n - b * p.S) : 0;
  const int lane = threadIdx.x % kLanes;
  const RopeLane r = rope_lane<D, INTER>(p, lane, p.pos + b * p.pos_sb + static_cast<long long>(s) * p.axes, on);
  const int first = blockIdx.y * heads_per, last = min(first + heads_per, p.heads[0] + p.heads[1]);
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const int shift = which ? p.heads[0] : 0;
    const int h0 = max(first - shift, 0), h1 = min(last - shift, p.heads[which]);
    if (h0 >= h1) continue;
    const bool norm = p.weight[which] != nullptr;
    float w[8];
    rope_weights(p.weight[which], r, w);
    const __nv_bfloat16* x = p.x[which] + b * p.sb[which] + s * p.ss[which];
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out[which]) + (b * p.heads[which] * p.S + s) * D;
    const long long step = static_cast<long long>(p.S) * D;
#pragma unroll 1
    for (int h = h0; h < h1; h += kRopeUnroll) {
      uint4 raw[kRopeUnroll];
#pragma unroll
      for (int i = 0; i < kRopeUnroll; ++i)
        raw[i] = on && h + i < h1 ? rope_load<INTER>(x + (h + i) * p.sh[which], r) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int i = 0; i < kRopeUnroll; ++i) {
        float y[8];
        rope_apply<D, INTER>(r, raw[i], norm, w, p.eps, y);
        if (on && h + i < h1) {
          const uint4 o = NormVec<__nv_bfloat16>::pack(y);
          __nv_bfloat16* dst = out + (h + i) * step;
          if (INTER) {
            *reinterpret_cast<uint4*>(dst + r.lo) = o;
          } else {
            *reinterpret_cast<uint2*>(dst + r.lo) = make_uint2(o.x, o.y);
            *reinterpret_cast<uint2*>(dst + r.hi) = make_uint2(o.z, o.w);
          }
        }
      }
    }
  }
}

// E4M3 out.  A CTA takes a block of 128 tokens and heads_per heads, one head at a time: the block stays in
// registers between its maximum and its codes, and the next head's loads are under way meanwhile.
constexpr int kRopeBlockRows = 128;
constexpr int kRopeBlockThreads = 512;

template <int D, bool INTER>
__global__ void __launch_bounds__(kRopeBlockThreads, 1) rope_e4m3_kernel(const RopeParams p, int heads_per) {
  constexpr int kLanes = D / 8, kRows = kRopeBlockThreads / kLanes, kPass = kRopeBlockRows / kRows;
  __shared__ float red[2][kRopeBlockThreads / 32];
  const int nblk = (p.S + kRopeBlockRows - 1) / kRopeBlockRows;
  const long long b = blockIdx.x / nblk;
  const int blk = blockIdx.x % nblk;
  const int s0 = blk * kRopeBlockRows + threadIdx.x / kLanes;
  const int lane = threadIdx.x % kLanes;
  RopeLane r[kPass];
#pragma unroll
  for (int i = 0; i < kPass; ++i) {
    const int s = s0 + i * kRows;
    r[i] = rope_lane<D, INTER>(p, lane, p.pos + b * p.pos_sb + static_cast<long long>(s) * p.axes, s < p.S);
  }
  const int first = blockIdx.y * heads_per, last = min(first + heads_per, p.heads[0] + p.heads[1]);
  int flip = 0;
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const int shift = which ? p.heads[0] : 0;
    const int h0 = max(first - shift, 0), h1 = min(last - shift, p.heads[which]);
    if (h0 >= h1) continue;
    const bool norm = p.weight[which] != nullptr;
    float w[8];
    rope_weights(p.weight[which], r[0], w);
    const __nv_bfloat16* x = p.x[which] + b * p.sb[which] + s0 * p.ss[which];
    const long long step = kRows * p.ss[which];
    uint4 raw[kPass];
    auto load = [&](int h) {
#pragma unroll
      for (int i = 0; i < kPass; ++i)
        raw[i] = s0 + i * kRows < p.S ? rope_load<INTER>(x + h * p.sh[which] + i * step, r[i]) : make_uint4(0u, 0u, 0u, 0u);
    };
    load(h0);
#pragma unroll 1
    for (int h = h0; h < h1; ++h) {
      float y[kPass][8];
      float m = 0.0f;
#pragma unroll
      for (int i = 0; i < kPass; ++i) {
        rope_apply<D, INTER>(r[i], raw[i], norm, w, p.eps, y[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(y[i][e]));
      }
      if (h + 1 < h1) load(h + 1);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      if ((threadIdx.x & 31) == 0) red[flip][threadIdx.x >> 5] = m;
      __syncthreads();
      m = red[flip][threadIdx.x & (kRopeBlockThreads / 32 - 1)];
#pragma unroll
      for (int o = kRopeBlockThreads / 64; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      flip ^= 1;                                  // (two buffers: one barrier a head is enough)
      const float d = m > 0.0f ? __fdiv_rn(m, 448.0f) : 1.0f;
      const float rcp = __frcp_rn(d);
      const long long bh = b * p.heads[which] + h;
      if (threadIdx.x == 0) p.descales[which][bh * nblk + blk] = m > 0.0f ? d : 0.0f;
      uint8_t* out = static_cast<uint8_t*>(p.out[which]) + (bh * p.S + s0) * D;
#pragma unroll
      for (int i = 0; i < kPass; ++i) {
        if (s0 + i * kRows >= p.S) break;
        uint32_t c[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
          c[e] = pack_e4m3x4(quot_e4m3(y[i][4 * e], d, rcp), quot_e4m3(y[i][4 * e + 1], d, rcp),
                             quot_e4m3(y[i][4 * e + 2], d, rcp), quot_e4m3(y[i][4 * e + 3], d, rcp));
        uint8_t* dst = out + static_cast<long long>(i) * kRows * D;
        if (INTER) {
          *reinterpret_cast<uint2*>(dst + r[i].lo) = make_uint2(c[0], c[1]);
        } else {
          *reinterpret_cast<uint32_t*>(dst + r[i].lo) = c[0];
          *reinterpret_cast<uint32_t*>(dst + r[i].hi) = c[1];
        }
      }
    }
  }
}

}  // namespace dit
