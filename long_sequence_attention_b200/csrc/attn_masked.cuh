// Attention with capped scores, a distance bias and causal, prefix and document masks, shared
// key / value heads, and the few-query form of a step against a long cache.
//
// Query i of sequence b stands at position pos = q_start[b] + i among the keys j:
//     s_ij = scale * q_i . k_j;   s_ij = cap * tanh(s_ij / cap)   (cap > 0)
//     s_ij = s_ij - slope_h * |pos - j|                            (slopes given)
//     allowed(i, j) = (not causal or j <= pos or j < prefix[b])
//                     and (no documents or (q_doc[i] = kv_doc[j] and q_doc[i] >= 0))
//     out_i = sum over allowed j of softmax_j(s_ij) v_j,  lse_i = log sum over allowed exp(s_ij);
//     no allowed key: out_i = 0, lse_i = -inf.
#pragma once

#include <cuda_bf16.h>

#include "ptx.cuh"

namespace dit {

struct MaskedParams {
  const __nv_bfloat16 *q, *k, *v;   // [B, H, S_q, D], [B, H_kv, S_kv, D] x 2
  __nv_bfloat16* out;               // [B, H, S_q, D]
  float* lse;                       // [B, H, S_q] or null
  int B, H, H_kv, S_q, S_kv;
  float scale, cap;                 // cap 0: scores not capped
  const float* slopes;              // [H] or null
  int causal;
  const int* q_start;               // [B] or null: S_kv - S_q
  const int* prefix;                // [B] or null: 0
  const int* q_doc;                 // [B, S_q], with kv_doc, or null
  const int* kv_doc;                // [B, S_kv]
  unsigned long long timeout_ns;
};

// One warp per query row: 32 keys at a time, one per lane, with a running maximum and sum; the
// lanes then share the output's D elements.  A key that the row may not attend to is never
// multiplied, whatever its row of V holds.
constexpr int kMaskedRowWarps = 4;

template <int D>
__global__ void __launch_bounds__(32 * kMaskedRowWarps) attn_masked_row_kernel(const MaskedParams p) {
  __shared__ float sq[kMaskedRowWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long rows = static_cast<long long>(p.B) * p.H * p.S_q;
  for (long long r = static_cast<long long>(blockIdx.x) * kMaskedRowWarps + warp; r < rows;
       r += static_cast<long long>(gridDim.x) * kMaskedRowWarps) {
    const int i = static_cast<int>(r % p.S_q);
    const int h = static_cast<int>((r / p.S_q) % p.H);
    const long long b = r / p.S_q / p.H;
    const long long kv0 = (b * p.H_kv + h / (p.H / p.H_kv)) * p.S_kv * D;
    for (int d = lane; d < D; d += 32) sq[warp][d] = __bfloat162float(p.q[r * D + d]);
    __syncwarp();
    const int pos = (p.q_start ? p.q_start[b] : p.S_kv - p.S_q) + i;
    const int lim = p.causal ? max(pos + 1, p.prefix ? p.prefix[b] : 0) : p.S_kv;   // keys j < lim
    const int doc = p.q_doc ? p.q_doc[b * p.S_q + i] : 0;
    const float slope = p.slopes ? p.slopes[h] : 0.0f;
    float m = -INFINITY, l = 0.0f, acc[D / 32] = {};
    const int n = doc < 0 ? 0 : min(lim, p.S_kv);
    for (int j0 = 0; j0 < n; j0 += 32) {
      const int j = j0 + lane;
      float s = -INFINITY;
      if (j < n && (!p.kv_doc || p.kv_doc[b * p.S_kv + j] == doc)) {
        const __nv_bfloat16* kr = p.k + kv0 + static_cast<long long>(j) * D;
        s = 0.0f;
        for (int d = 0; d < D; ++d) s = fmaf(sq[warp][d], __bfloat162float(kr[d]), s);
        s *= p.scale;
        if (p.cap > 0.0f) s = p.cap * tanhf(s / p.cap);
        if (p.slopes) s -= slope * fabsf(static_cast<float>(pos - j));
      }
      float mt = s;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
      const float mn = fmaxf(m, mt);
      if (mn == -INFINITY) continue;
      const float pj = __expf(s - mn), alpha = __expf(m - mn);
      m = mn;
      float ps = pj;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, o);
      l = l * alpha + ps;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) acc[e] *= alpha;
      for (int t = 0; t < 32 && j0 + t < n; ++t) {
        const float pt = __shfl_sync(0xffffffffu, pj, t);
        const float st = __shfl_sync(0xffffffffu, s, t);
        if (st == -INFINITY) continue;
        const __nv_bfloat16* vr = p.v + kv0 + static_cast<long long>(j0 + t) * D;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) acc[e] = fmaf(pt, __bfloat162float(vr[e * 32 + lane]), acc[e]);
      }
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
    for (int e = 0; e < D / 32; ++e)
      p.out[r * D + e * 32 + lane] = __float2bfloat16(m == -INFINITY ? 0.0f : acc[e] * (l != l ? l : inv));
    if (lane == 0 && p.lse) p.lse[r] = m == -INFINITY ? -INFINITY : m + logf(l);
    __syncwarp();
  }
}

}  // namespace dit
