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
// in 64-bit integer arithmetic drops whole turns exactly, so far positions lose nothing.  Of the
// fraction the nearest quarter turn comes off in integers too; cosine and sine of the rest, at most an
// eighth of a turn, are polynomials (fit_rope_poly.py), within 1.1 * 2^-24 absolutely.
//
// Bytes bound: q and k are read once and written once.  Sixteen elements a lane, D / 16 lanes a head row; a
// lane's sixteen are two runs of eight and hold eight whole pairs in either layout, so nothing crosses lanes but
// the norm's sum, and pairs of pairs go through packed fp32 instructions.  Angles are formed once for many heads: a thread keeps its token, or (E4M3) a CTA keeps its
// block's in shared memory, and walks over heads.
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

// cos and sin of position * freq times the magnitude.
__device__ __forceinline__ void rope_cos_sin(int pos, unsigned long long turns, float magnitude, float& c, float& s) {
  const unsigned long long t = static_cast<unsigned long long>(static_cast<long long>(pos)) * turns;
  const uint32_t hi = static_cast<uint32_t>(t >> 32);           // in 2^-32 turns
  const uint32_t quarter = (hi + 0x20000000u) >> 30;
  const int rest = static_cast<int>(hi - (quarter << 30));      // in [-2^29, 2^29)
  const float xi = static_cast<float>(rest);                    // 24 of its bits,
  const float dx = static_cast<float>(rest - static_cast<int>(xi)) * 1.4629180792671596e-09f;   // and pi 2^-31 times the rest
  const float x = xi * 4.6566128730773926e-10f;                 // 2^-31: half turns, |x| <= 1/4
  const float u = x * x;
  float q = fmaf(0.08099587261676788f, u, -0.5992013812065125f);
  q = fmaf(q, u, 2.5501625537872314f);
  q = fmaf(q, u, -5.167712688446045f);
  q = fmaf(q, u, -8.742277657347586e-08f);                      // pi less its fp32 value, which comes last
  float sp = fmaf(x, 3.1415927410125732f, x * q);
  float cp = fmaf(0.23126092553138733f, u, -1.3350359201431274f);
  cp = fmaf(cp, u, 4.058706760406494f);
  cp = fmaf(cp, u, -4.934802055358887f);
  cp = fmaf(cp, u, 1.0f);
  const float s0 = sp;
  sp = fmaf(cp, dx, sp);
  cp = fmaf(-s0, dx, cp);
  const float a = (quarter & 1u) ? sp : cp, b = (quarter & 1u) ? cp : sp;
  c = ((quarter + 1u) & 2u) ? -a * magnitude : a * magnitude;
  s = (quarter & 2u) ? -b * magnitude : b * magnitude;
}

// The turns and the axis of every pair, in shared memory.
struct RopeTable {
  unsigned long long turns[64];
  int axis[64];
};
__device__ __forceinline__ void rope_fill(const RopeParams& p, RopeTable& tab) {
  for (int i = threadIdx.x; i < p.rot / 2; i += blockDim.x) {
    tab.turns[i] = rope_turns(p.freqs[i]);
    int axis = 0;
#pragma unroll
    for (int a = 0; a + 1 < kMaxRopeAxes; ++a)
      if (a + 1 < p.axes && i >= p.axis_end[a]) axis = a + 1;
    tab.axis[i] = axis;
  }
  __syncthreads();
}

// Where a lane's elements lie: two runs of eight, lo .. and hi .., neighbouring lanes next to each other.  Interleaved:
// four pairs in each.  Half layout, inside the rotated part: the first elements of eight pairs and their second ones.
// `first` and `second` are the pairs that the runs' four (interleaved) or the lane's eight (half) begin with.
struct RopeLane {
  int lo, hi, first, second;
  uint32_t turn;                 // bit k: the lane's pair k is rotated
};
template <int D, bool INTER>
__device__ __forceinline__ RopeLane rope_lane(int rot, int lane) {
  RopeLane r;
  const int pairs = rot / 2;
  const bool split = !INTER && 8 * lane < pairs;
  r.lo = split || INTER ? 8 * lane : 16 * lane;
  r.hi = split ? 8 * lane + pairs : (INTER ? D / 2 + 8 * lane : 16 * lane + 8);
  r.first = INTER ? 4 * lane : 8 * lane;
  r.second = INTER ? D / 4 + 4 * lane : 8 * lane + 4;
  r.turn = 0u;
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if ((k < 4 ? r.first + k : r.second + k - 4) < pairs) r.turn |= 1u << k;
  return r;
}

struct RopeRaw { uint4 x, y; };
__device__ __forceinline__ RopeRaw rope_load(const __nv_bfloat16* x, const RopeLane& r) {
  return RopeRaw{__ldg(reinterpret_cast<const uint4*>(x + r.lo)), __ldg(reinterpret_cast<const uint4*>(x + r.hi))};
}

// A lane's pairs as packed fp32: a[k] = first elements of its pairs 2k and 2k + 1, b[k] their second ones.
template <bool INTER>
__device__ __forceinline__ void rope_unpack(const RopeRaw& raw, uint64_t (&a)[4], uint64_t (&b)[4]) {
  const uint32_t w[8] = {raw.x.x, raw.x.y, raw.x.z, raw.x.w, raw.y.x, raw.y.y, raw.y.z, raw.y.w};
  auto lo = [](uint32_t v) { return __uint_as_float(v << 16); };
  auto hi = [](uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); };
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (INTER) {
      a[k] = f2_pack(lo(w[2 * k]), lo(w[2 * k + 1]));
      b[k] = f2_pack(hi(w[2 * k]), hi(w[2 * k + 1]));
    } else {
      a[k] = f2_pack(lo(w[k]), hi(w[k]));
      b[k] = f2_pack(lo(w[4 + k]), hi(w[4 + k]));
    }
  }
}

// Norm (where weights are given, as raw) and rotation.
template <int D, bool INTER>
__device__ __forceinline__ void rope_apply(const RopeLane& r, const RopeRaw& raw, bool norm, const RopeRaw& weight, float eps,
                                           const uint64_t (&c)[4], const uint64_t (&s)[4], uint64_t (&ya)[4],
                                           uint64_t (&yb)[4]) {
  uint64_t a[4], b[4];
  rope_unpack<INTER>(raw, a, b);
  if (norm) {
    uint64_t q = 0ull;
#pragma unroll
    for (int k = 0; k < 4; ++k) q = f2_fma(a[k], a[k], f2_fma(b[k], b[k], q));
    float q0, q1;
    f2_unpack(q, q0, q1);
    float ss = q0 + q1;
#pragma unroll
    for (int o = D / 32; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float inv = __frsqrt_rn(ss * (1.0f / D) + eps);
    const uint64_t inv2 = f2_pack(inv, inv);
    uint64_t wa[4], wb[4];
    rope_unpack<INTER>(weight, wa, wb);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      a[k] = f2_mul(f2_mul(a[k], inv2), wa[k]);
      b[k] = f2_mul(f2_mul(b[k], inv2), wb[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    ya[k] = f2_sub(f2_mul(a[k], c[k]), f2_mul(b[k], s[k]));
    yb[k] = f2_fma(a[k], s[k], f2_mul(b[k], c[k]));
  }
  if (r.turn != 0xFFu) {         // elements past rot pass unchanged
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float a0, a1, b0, b1, y0, y1, z0, z1;
      f2_unpack(a[k], a0, a1);
      f2_unpack(b[k], b0, b1);
      f2_unpack(ya[k], y0, y1);
      f2_unpack(yb[k], z0, z1);
      const bool t0 = (r.turn >> (2 * k)) & 1u, t1 = (r.turn >> (2 * k + 1)) & 1u;
      ya[k] = f2_pack(t0 ? y0 : a0, t1 ? y1 : a1);
      yb[k] = f2_pack(t0 ? z0 : b0, t1 ? z1 : b1);
    }
  }
}

// A lane's angles (0 where nothing turns).
__device__ __forceinline__ void rope_angles(const RopeParams& p, const RopeTable& tab, const RopeLane& r, const int* pos, bool on,
                                            float (&c)[8], float (&s)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    c[k] = s[k] = 0.0f;
    const int i = k < 4 ? r.first + k : r.second + k - 4;
    if (on && ((r.turn >> k) & 1u)) rope_cos_sin(__ldg(pos + tab.axis[i]), tab.turns[i], p.magnitude, c[k], s[k]);
  }
}

// bf16 out.  A CTA takes 256 * 16 / D tokens (of all batches, one after another) and heads_per heads of q and k
// together, four heads' loads in flight at a time (B200, 40 + 40 heads x 32760 x 128, normed: 221 us, 6.07 TB/s; two
// heads and three CTAs on an SM 242).
constexpr int kRopeThreads = 256;
constexpr int kRopeUnroll = 4;

template <int D, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 2) rope_kernel(const RopeParams p, int heads_per) {
  constexpr int kLanes = D / 16;
  __shared__ RopeTable tab;
  rope_fill(p, tab);
  const long long n = static_cast<long long>(blockIdx.x) * (kRopeThreads / kLanes) + threadIdx.x / kLanes;
  const bool on = n < static_cast<long long>(p.B) * p.S;
  const long long b = on ? n / p.S : 0;
  const int s = on ? static_cast<int>(n - b * p.S) : 0;
  const int lane = threadIdx.x % kLanes;
  const RopeLane r = rope_lane<D, INTER>(p.rot, lane);
  uint64_t c2[4], s2[4];
  {
    float c[8], sn[8];
    rope_angles(p, tab, r, p.pos + b * p.pos_sb + static_cast<long long>(s) * p.axes, on, c, sn);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      c2[k] = f2_pack(c[2 * k], c[2 * k + 1]);
      s2[k] = f2_pack(sn[2 * k], sn[2 * k + 1]);
    }
  }
  const int first = blockIdx.y * heads_per, last = min(first + heads_per, p.heads[0] + p.heads[1]);
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const int shift = which ? p.heads[0] : 0;
    const int h0 = max(first - shift, 0), h1 = min(last - shift, p.heads[which]);
    if (h0 >= h1) continue;
    const bool norm = p.weight[which] != nullptr;
    RopeRaw w = {};
    if (norm) w = rope_load(p.weight[which], r);
    const long long sh = p.sh[which], step = static_cast<long long>(p.S) * D;
    const __nv_bfloat16* x = p.x[which] + b * p.sb[which] + s * p.ss[which] + h0 * sh;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out[which]) + ((b * p.heads[which] + h0) * p.S + s) * D;
#pragma unroll 1
    for (int h = h0; h < h1; h += kRopeUnroll) {
      RopeRaw raw[kRopeUnroll];
#pragma unroll
      for (int i = 0; i < kRopeUnroll; ++i) {
        raw[i] = RopeRaw{};
        if (on && h + i < h1) raw[i] = rope_load(x + i * sh, r);
      }
#pragma unroll
      for (int i = 0; i < kRopeUnroll; ++i) {
        uint64_t ya[4], yb[4];
        rope_apply<D, INTER>(r, raw[i], norm, w, p.eps, c2, s2, ya, yb);
        uint32_t o[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float a0, a1, b0, b1;
          f2_unpack(ya[k], a0, a1);
          f2_unpack(yb[k], b0, b1);
          if (INTER) {
            o[2 * k] = pack_bf16x2(a0, b0);
            o[2 * k + 1] = pack_bf16x2(a1, b1);
          } else {
            o[k] = pack_bf16x2(a0, a1);
            o[4 + k] = pack_bf16x2(b0, b1);
          }
        }
        if (on && h + i < h1) {
          *reinterpret_cast<uint4*>(out + i * step + r.lo) = make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4*>(out + i * step + r.hi) = make_uint4(o[4], o[5], o[6], o[7]);
        }
      }
      x += kRopeUnroll * sh;
      out += kRopeUnroll * step;
    }
  }
}

// E4M3 out.  A CTA takes a block of 128 tokens and heads_per heads, one head at a time, one row piece of sixteen
// elements a thread: it keeps its angles and, between the block's maximum and its codes, its results in registers.
// The next heads' loads are under way into shared memory (asynchronous copies that only the thread that made them
// reads back, so that they need no barrier); one barrier a head, for the maximum.  Issue slots bound it (about 165
// instructions for sixteen elements), not bytes: 2 x 4429 x 48 x 128 take 47 us, 3.5 TB/s; with the angles in shared
// memory and four row pieces a thread 49, with two heads' results in registers at a time more.
constexpr int kRopeBlockRows = 128;
constexpr int kRopeStages = 3;
template <int D>
struct RopeBlock {
  static constexpr int kLanes = D / 16, kThreads = kRopeBlockRows * kLanes;
  static constexpr int kStage = kRopeBlockRows * D * 2;
  static constexpr int kSmem = kRopeStages * kStage;
  static constexpr int kCtas = 1024 / kThreads;                 // on an SM (registers: 1024 threads of 64)
};

__device__ __forceinline__ void copy_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <int D, bool INTER>
__global__ void __launch_bounds__(RopeBlock<D>::kThreads, RopeBlock<D>::kCtas) rope_e4m3_kernel(const RopeParams p, int heads_per) {
  using R = RopeBlock<D>;
  constexpr int kWarps = R::kThreads / 32;
  extern __shared__ uint4 stages[];
  __shared__ RopeTable tab;
  __shared__ float red[2][kWarps];
  rope_fill(p, tab);
  const int nblk = (p.S + kRopeBlockRows - 1) / kRopeBlockRows;
  const long long b = blockIdx.x / nblk;
  const int blk = blockIdx.x % nblk;
  const int s = blk * kRopeBlockRows + threadIdx.x / R::kLanes;
  const bool on = s < p.S;
  const RopeLane r = rope_lane<D, INTER>(p.rot, threadIdx.x % R::kLanes);
  const int first = blockIdx.y * heads_per, last = min(first + heads_per, p.heads[0] + p.heads[1]);
  // running places of the next head to load and of the next to write, which go from q's heads to k's
  const __nv_bfloat16* x;
  uint8_t* out;
  float* descale;
  auto seek_x = [&](int which, int h) { x = p.x[which] + b * p.sb[which] + s * p.ss[which] + h * p.sh[which]; };
  auto seek_out = [&](int which, int h) {
    const long long bh = b * p.heads[which] + h;
    out = static_cast<uint8_t*>(p.out[which]) + (bh * p.S + s) * D;
    descale = p.descales[which] + bh * nblk + blk;
  };
  const int q_heads = p.heads[0];
  seek_x(first >= q_heads, first >= q_heads ? first - q_heads : first);
  seek_out(first >= q_heads, first >= q_heads ? first - q_heads : first);
  uint4* const mine = stages + threadIdx.x;
  int to_load = first, load_slot = 0;
  auto load = [&] {
    if (on && to_load < last) {
      uint4* dst = mine + load_slot * (R::kStage / 16);
      copy_async16(dst, x + r.lo);
      copy_async16(dst + R::kThreads, x + r.hi);
    }
    copy_async_commit();
    x += to_load < q_heads ? p.sh[0] : p.sh[1];
    if (++to_load == q_heads && p.heads[1] > 0) seek_x(1, 0);
    load_slot = load_slot == kRopeStages - 1 ? 0 : load_slot + 1;
  };
#pragma unroll
  for (int k = 0; k < kRopeStages; ++k) load();
  uint64_t c2[4], s2[4];
  {
    float c[8], sn[8];
    rope_angles(p, tab, r, p.pos + b * p.pos_sb + static_cast<long long>(s) * p.axes, on, c, sn);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      c2[k] = f2_pack(c[2 * k], c[2 * k + 1]);
      s2[k] = f2_pack(sn[2 * k], sn[2 * k + 1]);
    }
  }
  RopeRaw w = {};
  bool norm = false;
  auto weights = [&](int which) {
    norm = p.weight[which] != nullptr;
    if (norm) w = rope_load(p.weight[which], r);
  };
  weights(first >= q_heads);
  int slot = 0, flip = 0;
#pragma unroll 1
  for (int hh = first; hh < last; ++hh) {
    if (hh == q_heads && hh != first) {
      weights(1);
      seek_out(1, 0);
    }
    copy_async_wait<kRopeStages - 1>();
    RopeRaw raw = {};
    if (on) raw = RopeRaw{mine[slot * (R::kStage / 16)], mine[slot * (R::kStage / 16) + R::kThreads]};
    slot = slot == kRopeStages - 1 ? 0 : slot + 1;
    uint64_t ya[4], yb[4];
    rope_apply<D, INTER>(r, raw, norm, w, p.eps, c2, s2, ya, yb);
    load();
    float m = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float a0, a1, b0, b1;
      f2_unpack(ya[k], a0, a1);
      f2_unpack(yb[k], b0, b1);
      m = fmax3(m, fabsf(a0), fabsf(a1));
      m = fmax3(m, fabsf(b0), fabsf(b1));
    }
    // (of values >= 0 the bits order as the values do: one instruction for the warp's maximum)
    m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
    if ((threadIdx.x & 31) == 0) red[flip][threadIdx.x >> 5] = m;
    __syncthreads();
    m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(red[flip][threadIdx.x & (kWarps - 1)])));
    const float d = m >= kE4m3Least ? __fdiv_rn(m, 448.0f) : 1.0f;     // (two buffers: one barrier a head is enough)
    const float rcp = m >= kE4m3Least ? __fdiv_rn(448.0f, m) : 1.0f;   // (1 / d with one rounding less)
    if (threadIdx.x == 0) *descale = m >= kE4m3Least ? d : 0.0f;
    flip ^= 1;
    const uint64_t rcp2 = f2_pack(rcp, rcp);
    uint32_t c[4];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      float a0, a1, a2, a3, b0, b1, b2, b3;
      f2_unpack(f2_mul(ya[2 * q], rcp2), a0, a1);
      f2_unpack(f2_mul(ya[2 * q + 1], rcp2), a2, a3);
      f2_unpack(f2_mul(yb[2 * q], rcp2), b0, b1);
      f2_unpack(f2_mul(yb[2 * q + 1], rcp2), b2, b3);
      if (INTER) {
        c[2 * q] = pack_e4m3x4(a0, b0, a1, b1);
        c[2 * q + 1] = pack_e4m3x4(a2, b2, a3, b3);
      } else {
        c[q] = pack_e4m3x4(a0, a1, a2, a3);
        c[2 + q] = pack_e4m3x4(b0, b1, b2, b3);
      }
    }
    if (on) {
      *reinterpret_cast<uint2*>(out + r.lo) = make_uint2(c[0], c[1]);
      *reinterpret_cast<uint2*>(out + r.hi) = make_uint2(c[2], c[3]);
    }
    out += static_cast<long long>(p.S) * D;
    descale += nblk;
  }
  copy_async_wait<0>();
}

}  // namespace dit
