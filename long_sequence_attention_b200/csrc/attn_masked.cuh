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
//
// The kernel keeps the pipeline of the dense forward (attn_fwd.cuh: TMA producer, one thread that
// issues every tcgen05.mma, two softmax warpgroups, P over S in TMEM) around another walk:
//   * The query heads of a key / value head lie next to each other in memory, so they make one run
//     of query rows cut into tiles of 128 without regard to heads, which fills the tiles of few
//     queries; where a head's rows fill its tiles well enough, each head is a run of its own.
//   * Units differ in length, so a CTA takes its next one from a counter when it gets there (the TMA
//     thread fetches it early and passes it on through shared memory), the longest first.
//   * Every role walks the same list of KV tiles of its unit: the tiles up to the last key that
//     a row of the unit may see, without those that hold no document of its rows (bits that a
//     small kernel writes before).  Tiles that every row sees whole take the dense path (the
//     speculative softmax); the others are masked per row and take the exact maximum first.
//   * Long form: a unit is 256 rows as two Q tiles that share each K and V tile.
//   * Split form, for few rows against many keys: a unit is one 128-row Q tile and a share of its
//     KV tiles; the two streams take alternate tiles, each with its own running maximum, sum
//     and O, and the partial results (fp32) are joined by their LSEs in a second kernel.
//   * The two idle warps of the dense form look through the V rows of masked tiles: a non-finite
//     value would reach every row of the tile (0 * inf), so it is zeroed in shared memory and
//     its key flagged; the rows that may see that key become NaN, the others never notice.
#pragma once

#include <cuda_bf16.h>

#include "attn_fwd.cuh"
#include "ptx.cuh"

namespace dit {

struct MaskedParams {
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
  int run_heads, runs;              // query heads of a run (H / H_kv, or 1), runs = B * H / run_heads
  int rows;                         // query rows of a run: run_heads * S_q
  int n_blk;                        // units of a run's rows: ceil(rows / 256), split form ceil(rows / 128)
  int n_split;                      // split form: shares of the KV tiles
  int n_units;
  unsigned int* next_unit;          // units handed out beyond the first of every CTA (zero at launch); null: in steps
  uint2* words;                     // [B, n_blk, ceil(S_kv / 4096)] {needed, whole} tile bits, or null
  float* part_o;                    // split form: [2 n_split, B * H * S_q, D]
  float* part_lse;                  // split form: [2 n_split, B * H * S_q]
  unsigned long long timeout_ns;
};

constexpr int kMaskedTile = 128;    // keys of a KV tile

// What one unit computes: query rows r0.. of a run, KV tiles [j0, j1) of key head kv = b * H_kv + key head.
struct MaskedUnit {
  int run, kv, b, r0, start, pre;
  int j0, j1, jc;                   // jc: where the walk starts
  int n_whole;                      // keys [0, n_whole) are left by every row's causal / prefix mask
  const uint2* words;
};

// First key past those that a query at this position may see (documents aside).
__device__ __forceinline__ int masked_limit(const MaskedParams& p, int pos, int pre) {
  return p.causal ? min(max(max(pos + 1, pre), 0), p.S_kv) : p.S_kv;
}

template <bool SPLIT>
__device__ __forceinline__ MaskedUnit masked_unit(const MaskedParams& p, int u) {
  constexpr int kRows = SPLIT ? 128 : 256;
  MaskedUnit w;
  int blk, share = 0;
  if constexpr (SPLIT) {
    share = u % p.n_split;
    blk = (u / p.n_split) % p.n_blk;
    w.run = u / p.n_split / p.n_blk;
  } else {
    // the last rows (of a causal mask: the longest lists) of every run first
    blk = p.n_blk - 1 - u / p.runs;
    w.run = u % p.runs;
  }
  const int per_b = p.H / p.run_heads;
  w.b = w.run / per_b;
  w.kv = w.b * p.H_kv + (w.run % per_b) * p.run_heads / (p.H / p.H_kv);
  w.r0 = blk * kRows;
  w.start = p.q_start ? __ldg(p.q_start + w.b) : p.S_kv - p.S_q;
  w.pre = p.prefix ? __ldg(p.prefix + w.b) : 0;
  const int last = min(w.r0 + kRows, p.rows) - 1;
  const bool one_head = w.r0 / p.S_q == last / p.S_q;
  const int lo = one_head ? w.r0 % p.S_q : 0, hi = one_head ? last % p.S_q : p.S_q - 1;
  w.n_whole = masked_limit(p, w.start + lo, w.pre);
  const int n = (masked_limit(p, w.start + hi, w.pre) + kMaskedTile - 1) / kMaskedTile;
  w.j0 = 0;
  w.j1 = n;
  if constexpr (SPLIT) {
    const int per = (n + p.n_split - 1) / p.n_split;
    w.j0 = min(n, share * per);
    w.j1 = min(n, w.j0 + per);
  }
  // With a distance bias the walk starts at the last row's own position, where its scores are largest, and
  // goes outwards; otherwise it starts at the end, where the masks of a causal or ragged unit lie.  Either way the
  // first tile, which takes the exact path anyhow, settles the running maximum.
  w.jc = w.j1 - 1;
  if (p.slopes != nullptr) w.jc = min(max((w.start + hi) / kMaskedTile, w.j0), w.j1 - 1);
  w.words = p.words
                ? p.words + (static_cast<size_t>(w.b) * p.n_blk + blk) * ((p.S_kv + 32 * kMaskedTile - 1) / (32 * kMaskedTile))
                : nullptr;
  return w;
}

// Walk over a unit's KV tiles, jc down to j0 and then jc + 1 up to j1 - 1; every role of the CTA sees the same
// sequence.
struct MaskedTiles {
  const uint2* words;
  int j, j0, j1, jc, n_whole;
  int at = -1;
  bool down = true;
  uint32_t need = 0u, whole = 0u;
  __device__ __forceinline__ explicit MaskedTiles(const MaskedUnit& w)
      : words(w.words), j(w.jc), j0(w.j0), j1(w.j1), jc(w.jc), n_whole(w.n_whole) {}
  // The next tile and whether some row masks some of its keys; false at the end.
  __device__ __forceinline__ bool next(int& tile, bool& part) {
    while (true) {
      if (down ? j < j0 : j >= j1) {
        if (!down) return false;
        down = false;
        j = jc + 1;
        continue;
      }
      part = (j + 1) * kMaskedTile > n_whole;
      if (words != nullptr) {
        if ((j >> 5) != at) {
          at = j >> 5;
          const uint2 x = words[at];
          need = x.x;
          whole = x.y;
        }
        const uint32_t m = down ? need & (0xFFFFFFFFu >> (31 - (j & 31))) : need & (0xFFFFFFFFu << (j & 31));
        if (m == 0u) {
          j = down ? (at << 5) - 1 : (at + 1) << 5;
          continue;
        }
        j = (at << 5) + (down ? 31 - __clz(m) : __ffs(m) - 1);
        if (down ? j < j0 : j >= j1) continue;
        part = (j + 1) * kMaskedTile > n_whole || !((whole >> (j & 31)) & 1u);
      }
      tile = j;
      j += down ? -1 : 1;
      return true;
    }
  }
  // Tiles of the whole walk.
  __device__ __forceinline__ int count() const {
    if (words == nullptr || j1 <= j0) return max(j1 - j0, 0);
    int n = 0;
    for (int w = j0 >> 5; w * 32 < j1; ++w) {
      uint32_t m = words[w].x;
      if (w == j0 >> 5) m &= 0xFFFFFFFFu << (j0 & 31);
      if (j1 - w * 32 < 32) m &= (1u << (j1 - w * 32)) - 1u;
      n += __popc(m);
    }
    return n;
  }
};

// Documents: bit j of a unit's words says whether KV tile j holds a key whose document lies
// between the smallest and largest document of the unit's rows (needed), and whether all of both
// are one document (whole).  One CTA per (b, unit of rows); reads S_kv + 256 ids, a few KB that stay in L2.
template <int kRows>
__global__ void __launch_bounds__(256) masked_tiles_kernel(const MaskedParams p) {
  __shared__ int red[3][8];
  const int blk = blockIdx.x % p.n_blk, b = blockIdx.x / p.n_blk;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_words = (p.S_kv + 32 * kMaskedTile - 1) / (32 * kMaskedTile);
  const int r = blk * kRows + threadIdx.x;
  int lo = 0x7FFFFFFF, hi = -1, pad = 0;
  if (static_cast<int>(threadIdx.x) < kRows && r < p.rows) {
    const int id = p.q_doc[static_cast<size_t>(b) * p.S_q + r % p.S_q];
    pad = id < 0;
    if (!pad) lo = hi = id;
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  pad = __reduce_max_sync(0xffffffffu, pad);
  if (lane == 0) { red[0][warp] = lo; red[1][warp] = hi; red[2][warp] = pad; }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) { lo = min(lo, red[0][i]); hi = max(hi, red[1][i]); pad = max(pad, red[2][i]); }
  const bool q_one = lo == hi && !pad;
  const int* kd = p.kv_doc + static_cast<size_t>(b) * p.S_kv;
  uint2* words = p.words + static_cast<size_t>(blockIdx.x) * n_words;
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.next_unit != nullptr) *p.next_unit = 0u;
  // 32 tiles at a time, four to a warp: sixteen loads of a lane in flight
  __shared__ uint2 part[8];
  for (int w = 0; w < n_words; ++w) {
    uint2 x = make_uint2(0u, 0u);
    int id[4][4];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const long long k = (w * 32LL + warp * 4 + t) * kMaskedTile + i * 32 + lane;
        id[t][i] = k < p.S_kv ? __ldg(kd + k) : -1;
      }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      int klo = 0x7FFFFFFF, khi = -1, kpad = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        kpad |= id[t][i] < 0;
        klo = min(klo, id[t][i] < 0 ? 0x7FFFFFFF : id[t][i]);
        khi = max(khi, id[t][i]);
      }
      klo = __reduce_min_sync(0xffffffffu, klo);
      khi = __reduce_max_sync(0xffffffffu, khi);
      kpad = __any_sync(0xffffffffu, kpad != 0);
      if (khi >= lo && klo <= hi && hi >= 0 && khi >= 0) x.x |= 1u << (warp * 4 + t);
      if (q_one && klo == khi && klo == lo && !kpad) x.y |= 1u << (warp * 4 + t);
    }
    if (lane == 0) part[warp] = x;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
      for (int i = 1; i < 8; ++i) { x.x |= part[i].x; x.y |= part[i].y; }
      words[w] = x;
    }
    __syncthreads();
  }
}

template <int D, bool SPLIT>
struct MaskedCfg {
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kBlkBytes = 128 * 128;
  static constexpr int kNBlk = D / 64;
  static constexpr int kQTiles = SPLIT ? 1 : 2;
  // D = 128: 2 Q + 2 K + 2 V tiles, or 1 + 3 + 3; D = 64: 2 + 5 + 5, or 1 + 6 + 6 (tiles of 16 KB)
  static constexpr int kStages = D == 128 ? (SPLIT ? 3 : 2) : (SPLIT ? 6 : 5);
  static constexpr int kThreads = 384;
  static constexpr int kRegsLaunch = 168, kRegsSoftmax = 216, kRegsCtl = 72;
  static_assert(2 * 128 * kRegsSoftmax + 128 * kRegsCtl <= kThreads * kRegsLaunch, "register split");
  static constexpr int kMmaWarp = 8, kTmaWarp = 9, kVWarp = 10;
  static constexpr int kColS0 = 0, kColS1 = 128, kColO0 = 256, kColO1 = 256 + D;
  // P, O and l are floating point, so a running maximum 2^40 below the true one costs no precision (dense form:
  // 2^8): loud scores then hardly ever leave the speculative path
  static constexpr float kRescaleLog2 = 40.0f, kSumBound = 1099511627776.0f;
  static constexpr int kOffK = kQTiles * kTileBytes;
  static constexpr int kOffV = kOffK + kStages * kTileBytes;
  static constexpr int kOffIds = kOffV + kStages * kTileBytes;      // documents of the tile's keys, per V stage
  static constexpr int kOffBad = kOffIds + kStages * 512;           // 128 bits of flagged keys, per V stage
  static constexpr int kOffBar = kOffBad + kStages * 16;
  static constexpr int kUnitSlots = 4;                              // units handed on and not yet taken by every role
  static constexpr int kUnitReaders = 1 + 2 + 8;                    // MMA, V and softmax warps
  static constexpr int kNumBars = 2 + 5 * kStages + 6 + 1 + 2 * kUnitSlots;
  static constexpr int kOffMisc = kOffBar + 8 * kNumBars;
  static constexpr int kSmemBytes = kOffMisc + 16 + 8 * kUnitSlots + 1024;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
};

// tanh(x) = x p(x^2) for |x| <= 1, relative error 6e-7 (fit_tanh_poly.py), on the FMA pipe.
__device__ __forceinline__ uint64_t tanh_poly2(uint64_t x) {
  const uint64_t t = f2_mul(x, x);
  uint64_t r = f2_fma(f2_pack(-0.003067060373723507f, -0.003067060373723507f), t,
                      f2_pack(0.016743116080760956f, 0.016743116080760956f));
  r = f2_fma(r, t, f2_pack(-0.051605675369501114f, -0.051605675369501114f));
  r = f2_fma(r, t, f2_pack(0.13281433284282684f, 0.13281433284282684f));
  r = f2_fma(r, t, f2_pack(-0.3332904279232025f, -0.3332904279232025f));
  r = f2_fma(r, t, f2_pack(0.9999994039535522f, 0.9999994039535522f));
  return f2_mul(x, r);
}

// tanh by the exponential, any x: 1 - 2 / (1 + e^2x), within 3e-7 absolutely.
__device__ __forceinline__ float tanh_any(float x) {
  return 1.0f - __fdividef(2.0f, 1.0f + ex2_approx(x * 2.8853900817779268f));
}

// N scores s -> tanh(s * c), in place (the caller's unit becomes the cap).  The polynomial where every
// |s * c| <= 1 in the warp, the usual case: capping is meant for rare large scores.
template <int N>
__device__ __forceinline__ void cap_scores(uint32_t (&s)[N], float c) {
  float m[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < N; i += 8)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      m[k] = fmax3(m[k], fabsf(__uint_as_float(s[i + 2 * k])), fabsf(__uint_as_float(s[i + 2 * k + 1])));
  const bool far = !(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * c <= 1.0f);
  if (!__any_sync(0xffffffffu, far)) {
    const uint64_t c2 = f2_pack(c, c);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      float a, b;
      f2_unpack(tanh_poly2(f2_mul(f2_pack(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), c2)), a, b);
      s[i] = __float_as_uint(a);
      s[i + 1] = __float_as_uint(b);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = __float_as_uint(tanh_any(__uint_as_float(s[i]) * c));
  }
}

// MOD: what is done to the scores, fixed at compile time because the softmax's registers are full: 0 nothing,
// 1 the cap, 2 the distance bias and, where given, the cap.
template <int D, bool SPLIT, int MOD>
__global__ void __launch_bounds__(384, 1)
    attn_masked_kernel(const __grid_constant__ MapSet<1> maps, const MaskedParams p) {
  using C = MaskedCfg<D, SPLIT>;
  constexpr int NS = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* bar_q_full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* bar_q_empty = bar_q_full + 1;
  uint64_t* bar_k_full = bar_q_full + 2;              // [NS]
  uint64_t* bar_k_empty = bar_k_full + NS;            // [NS]
  uint64_t* bar_v_full = bar_k_empty + NS;            // [NS] V has landed
  uint64_t* bar_v_clean = bar_v_full + NS;            // [NS] and holds finite values where it is masked
  uint64_t* bar_v_empty = bar_v_clean + NS;           // [NS]
  uint64_t* bar_s_full = bar_v_empty + NS;            // [2]
  uint64_t* bar_p_full = bar_s_full + 2;              // [2]
  uint64_t* bar_o_final = bar_p_full + 2;             // [2]
  uint64_t* bar_drain = bar_o_final + 2;
  uint64_t* bar_u_full = bar_drain + 1;               // [kUnitSlots]
  uint64_t* bar_u_empty = bar_u_full + C::kUnitSlots; // [kUnitSlots]
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  volatile int* units = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 16);   // [slot] {unit, tiles}
  int* ids = reinterpret_cast<int*>(smem + C::kOffIds);
  uint32_t* bad = reinterpret_cast<uint32_t*>(smem + C::kOffBad);
  uint8_t* sQ = smem;
  uint8_t* sK = smem + C::kOffK;
  uint8_t* sV = smem + C::kOffV;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint64_t tmo = p.timeout_ns;

  if (threadIdx.x == C::kTmaWarp * 32) {
    mbar_init(bar_q_full, 1);
    mbar_init(bar_q_empty, 1);
    for (int s = 0; s < NS; ++s) {
      mbar_init(bar_k_full + s, 1);
      mbar_init(bar_k_empty + s, 1);
      mbar_init(bar_v_full + s, 1);
      mbar_init(bar_v_clean + s, 2);
      mbar_init(bar_v_empty + s, 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar_s_full + t, 1);
      mbar_init(bar_p_full + t, 4);
      mbar_init(bar_o_final + t, 1);
    }
    mbar_init(bar_drain, 1);
    for (int s = 0; s < C::kUnitSlots; ++s) {
      mbar_init(bar_u_full + s, 1);
      mbar_init(bar_u_empty + s, C::kUnitReaders);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;

  // Q tiles of a unit that hold rows (long form; in the split form both streams use the one tile)
  auto q_tiles = [&](const MaskedUnit& w) { return SPLIT ? 1 : (p.rows - w.r0 > 128 ? 2 : 1); };

  // The i-th unit of this CTA, as the TMA thread passed it on (n_units or more: no further one); < 0: gave up.
  // Every reading warp frees the slot once.  (The MMA thread takes the number of tiles along with it, because its
  // registers, 72 less the descriptors of every K step, have no room for the walk.)
  auto unit_of = [&](int i) {
    const int slot = i % C::kUnitSlots;
    if (!mbar_wait(bar_u_full + slot, (i / C::kUnitSlots) & 1, abort_flag, tmo, 0x2D)) return -1;
    return units[2 * slot];
  };
  auto unit_taken = [&](int i) { mbar_arrive(bar_u_empty + i % C::kUnitSlots); };

  if (warp >= 8) {
    regs_dec<C::kRegsCtl>();
    if (warp == C::kTmaWarp) {
      // ---------------------------------------------------------------- TMA producer
      if (lane == 0) {
        tma_prefetch_desc(&maps.q[0]);
        tma_prefetch_desc(&maps.k[0]);
        tma_prefetch_desc(&maps.v[0]);
        int g = 0, nq = 0, k_issued = 0, v_issued = 0;      // running tile and Q counts
        bool ok = true;
        int u = blockIdx.x;
        for (int i = 0; ok; ++i) {
          const int slot = i % C::kUnitSlots;
          if (i >= C::kUnitSlots && !(ok = mbar_wait(bar_u_empty + slot, ((i / C::kUnitSlots) + 1) & 1, abort_flag, tmo, 0x2E)))
            break;
          const bool last = u >= p.n_units;
          const MaskedUnit w = masked_unit<SPLIT>(p, last ? 0 : u);
          MaskedTiles it(w);
          units[2 * slot] = u;
          units[2 * slot + 1] = it.count();
          mbar_arrive(bar_u_full + slot);
          if (last) break;
          u = p.next_unit ? static_cast<int>(gridDim.x + atomicAdd(p.next_unit, 1u)) : u + static_cast<int>(gridDim.x);
          int j;
          bool part, first = true;
          while (ok && it.next(j, part)) {
            if (first) {
              first = false;
              if (nq > 0 && !(ok = mbar_wait(bar_q_empty, (nq - 1) & 1, abort_flag, tmo, 0x20))) break;
              const int nt = q_tiles(w);
              mbar_arrive_expect_tx(bar_q_full, nt * C::kTileBytes);
              for (int t = 0; t < nt; ++t)
                for (int b = 0; b < C::kNBlk; ++b)
                  tma_load_4d(sQ + t * C::kTileBytes + b * C::kBlkBytes, &maps.q[0], bar_q_full, b * 64,
                              w.r0 + t * 128, w.run, 0);
              ++nq;
            }
            const int st = g % NS;
            if (g >= NS && !(ok = mbar_wait(bar_k_empty + st, ((g / NS) + 1) & 1, abort_flag, tmo, 0x21))) break;
            mbar_arrive_expect_tx(bar_k_full + st, C::kTileBytes);
            for (int b = 0; b < C::kNBlk; ++b)
              tma_load_4d(sK + st * C::kTileBytes + b * C::kBlkBytes, &maps.k[0], bar_k_full + st, b * 64,
                          j * kMaskedTile, w.kv, 0);
            k_issued = g + 1;
            if (g >= NS && !(ok = mbar_wait(bar_v_empty + st, ((g / NS) + 1) & 1, abort_flag, tmo, 0x22))) break;
            mbar_arrive_expect_tx(bar_v_full + st, C::kTileBytes);
            for (int b = 0; b < C::kNBlk; ++b)
              tma_load_4d(sV + st * C::kTileBytes + b * C::kBlkBytes, &maps.v[0], bar_v_full + st, b * 64,
                          j * kMaskedTile, w.kv, 0);
            v_issued = ++g;
          }
        }
        // the last load of every stage must land before the CTA may exit
        if (nq > 0) mbar_wait_drain(bar_q_full, (nq - 1) & 1, tmo);
        for (int r = 0; r < NS; ++r) {
          if (k_issued > r) mbar_wait_drain(bar_k_full + r, ((k_issued - 1 - r) / NS) & 1, tmo);
          if (v_issued > r) mbar_wait_drain(bar_v_full + r, ((v_issued - 1 - r) / NS) & 1, tmo);
        }
      }
    } else if (warp == C::kMmaWarp) {
      // ---------------------------------------------------------------- MMA issuer
      if (lane == 0) {
        constexpr uint32_t id_s = instr_desc(1u, false, 128, 128);
        constexpr uint32_t id_o = instr_desc(1u, true, 128, D);
        const uint64_t dq = smem_desc_sw128(smem_u32(sQ), 16, 1024);
        const uint64_t dk = smem_desc_sw128(smem_u32(sK), 16, 1024);
        const uint64_t dv = smem_desc_sw128(smem_u32(sV), C::kBlkBytes, 1024);
        const uint32_t qk_hi = static_cast<uint32_t>(dq >> 32), v_hi = static_cast<uint32_t>(dv >> 32);
        const uint32_t q_lo = static_cast<uint32_t>(dq), k_lo = static_cast<uint32_t>(dk),
                       v_lo = static_cast<uint32_t>(dv);
        auto issue_s = [&](int t, int st) {
          const uint32_t a0 = q_lo + (((SPLIT ? 0 : t) * C::kTileBytes) >> 4);
          const uint32_t b0 = k_lo + ((st * C::kTileBytes) >> 4);
          const uint32_t d = tmem_base + (t ? C::kColS1 : C::kColS0);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk * 32 / 128) * C::kBlkBytes + (kk * 32) % 128) >> 4;
            mma_ss_lohi(false, d, a0 + off, qk_hi, b0 + off, qk_hi, id_s, kk > 0 ? 1u : 0u);
          }
        };
        auto issue_pv = [&](int t, int st, bool acc) {
          const uint32_t b0 = v_lo + ((st * C::kTileBytes) >> 4);
          const uint32_t a_tm = tmem_base + (t ? C::kColS1 : C::kColS0);
          const uint32_t d = tmem_base + (t ? C::kColO1 : C::kColO0);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ts_lohi(false, d, a_tm + kk * 8, b0 + ((kk * 16 * 128) >> 4), v_hi, id_o, (acc || kk > 0) ? 1u : 0u);
        };
        bool ok = true;
        int g = 0, nq = 0;                       // running tile and Q counts
        int np[2] = {0, 0};                      // P tiles taken from each stream
        auto wait_v = [&](int gt) {
          return mbar_wait(bar_v_clean + gt % NS, (gt / NS) & 1, abort_flag, tmo, 0x24);
        };
        auto wait_p = [&](int t) {
          const bool r = mbar_wait(bar_p_full + t, np[t] & 1, abort_flag, tmo, 0x25);
          ++np[t];
          return r;
        };
        for (int i = 0; ok; ++i) {
          const int u = unit_of(i);
          if (u < 0 || u >= p.n_units) break;
          const int tiles = units[2 * (i % C::kUnitSlots) + 1];
          unit_taken(i);
          const int nt = SPLIT || p.rows - (p.n_blk - 1 - u / p.runs) * 256 <= 128 ? 1 : 2;
          int n = 0;                             // tiles of this unit so far
          while (n < tiles) {
            if (n == 0) {
              if (!(ok = mbar_wait(bar_q_full, nq & 1, abort_flag, tmo, 0x26))) break;
              ++nq;
            }
            const int st = g % NS;
            if (!(ok = mbar_wait(bar_k_full + st, (g / NS) & 1, abort_flag, tmo, 0x23))) break;
            tc_fence_after();
            if constexpr (SPLIT) {
              // stream t takes every other tile; its previous one is two back
              const int t = n & 1;
              if (n >= 2) {
                if (!(ok = wait_v(g - 2) && wait_p(t))) break;
                tc_fence_after();
                issue_pv(t, (g - 2) % NS, n >= 4);
                tc_commit(bar_v_empty + (g - 2) % NS);
              }
              issue_s(t, st);
              tc_commit(bar_s_full + t);
            } else {
              const int vs = (g - 1 + NS) % NS;
              if (n > 0) {
                if (!(ok = wait_v(g - 1) && wait_p(0))) break;
                tc_fence_after();
                issue_pv(0, vs, n > 1);
                if (nt == 1) tc_commit(bar_v_empty + vs);
              }
              issue_s(0, st);
              tc_commit(bar_s_full + 0);
              if (nt == 2) {
                if (n > 0) {
                  if (!(ok = wait_p(1))) break;
                  tc_fence_after();
                  issue_pv(1, vs, n > 1);
                  tc_commit(bar_v_empty + vs);
                }
                issue_s(1, st);
                tc_commit(bar_s_full + 1);
              }
            }
            tc_commit(bar_k_empty + st);
            ++g;
            ++n;
          }
          if (!ok) break;
          if (n == 0) continue;
          tc_commit(bar_q_empty);                // every S MMA of this unit is issued
          if constexpr (SPLIT) {
            for (int e = n >= 2 ? n - 2 : 0; ok && e < n; ++e) {
              const int t = e & 1, gt = g - n + e;
              if (!(ok = wait_v(gt) && wait_p(t))) break;
              tc_fence_after();
              issue_pv(t, gt % NS, e >= 2);
              tc_commit(bar_o_final + t);
              tc_commit(bar_v_empty + gt % NS);
            }
          } else {
            const int vs = (g - 1) % NS;
            ok = wait_v(g - 1);
            for (int t = 0; ok && t < nt; ++t) {
              if (!(ok = wait_p(t))) break;
              tc_fence_after();
              issue_pv(t, vs, n > 1);
              tc_commit(bar_o_final + t);
            }
            if (ok) tc_commit(bar_v_empty + vs);
          }
        }
        // Every MMA this thread issued must finish before TMEM is released.
        tc_commit(bar_drain);
        mbar_wait_drain(bar_drain, 0, tmo);
      }
    } else {
      // ---------------------------------------------------------------- V rows of masked tiles
      // warp 10 keys 0-63, warp 11 keys 64-127: document ids for the softmax, non-finite values zeroed
      const int half = warp - C::kVWarp;
      bool ok = true;
      int g = 0;
      for (int i = 0; ok; ++i) {
        const int u = unit_of(i);
        __syncwarp();
        if (__any_sync(0xffffffffu, u < 0 || u >= p.n_units)) break;
        if (lane == 0) unit_taken(i);
        const MaskedUnit w = masked_unit<SPLIT>(p, u);
        MaskedTiles it(w);
        int j;
        bool part;
        while (it.next(j, part)) {
          const int st = g % NS;
          int id0 = -1, id1 = -1;
          if (part && w.words != nullptr) {
            const int k = j * kMaskedTile + half * 64 + lane;
            const int* kd = p.kv_doc + static_cast<size_t>(w.b) * p.S_kv;
            if (k < p.S_kv) id0 = __ldg(kd + k);
            if (k + 32 < p.S_kv) id1 = __ldg(kd + k + 32);
          }
          ok = __all_sync(0xffffffffu, mbar_wait(bar_v_full + st, (g / NS) & 1, abort_flag, tmo, 0x27));
          if (!ok) break;
          if (part) {
            if (w.words != nullptr) {
              ids[st * 128 + half * 64 + lane] = id0;
              ids[st * 128 + half * 64 + 32 + lane] = id1;
            }
            if (lane < 2) bad[st * 4 + half * 2 + lane] = 0u;
            __syncwarp();
            // row r of a 64-column block is the 128 bytes at r * 128 (the swizzle moves 16-byte pieces
            // within a row); exponent bits all ones: (x & 0x7F80) + 0x80 carries into bit 15
#pragma unroll 1
            for (int b = 0; b < C::kNBlk; ++b) {
              uint4* base = reinterpret_cast<uint4*>(sV + st * C::kTileBytes + b * C::kBlkBytes + half * 8192);
#pragma unroll 4
              for (int i = 0; i < 16; ++i) {
                const uint4 x = base[i * 32 + lane];
                const uint32_t e = ((x.x & 0x7F807F80u) + 0x00800080u) | ((x.y & 0x7F807F80u) + 0x00800080u) |
                                   ((x.z & 0x7F807F80u) + 0x00800080u) | ((x.w & 0x7F807F80u) + 0x00800080u);
                if (e & 0x80008000u) {
                  auto clean = [](uint32_t v) {
                    if ((v & 0x7F80u) == 0x7F80u) v &= 0xFFFF0000u;
                    if ((v & 0x7F800000u) == 0x7F800000u) v &= 0x0000FFFFu;
                    return v;
                  };
                  base[i * 32 + lane] = make_uint4(clean(x.x), clean(x.y), clean(x.z), clean(x.w));
                  const int r = i * 4 + (lane >> 3);             // key within this half
                  atomicOr(&bad[st * 4 + half * 2 + (r >> 5)], 1u << (r & 31));
                }
              }
            }
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_v_clean + st);
          ++g;
        }
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax warpgroups
    regs_inc<C::kRegsSoftmax>();
    const int t = warp >> 2;                     // Q tile, or stream of the split form
    const int quad = warp & 3;
    const int row = quad * 32 + lane;            // row within the tile == TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t tS = tmem_base + lane_off + (t ? C::kColS1 : C::kColS0);
    const uint32_t tO = tmem_base + lane_off + (t ? C::kColO1 : C::kColO0);
    // one unit of the scores that the softmax sees, in natural-log and in log2 units: raw q.k, or
    // tanh(q.k * scale / cap)
    const bool capped = MOD == 1 || (MOD == 2 && p.cap > 0.0f);
    const float unit = capped ? p.cap : p.scale;
    const float cl = unit * 1.4426950408889634f;
    const float cap_c = capped ? p.scale / p.cap : 0.0f;
    bool ok = true;
    int g = 0, ns = 0, no = 0;                   // running tiles of the CTA, S tiles and O's of this stream

    for (int i = 0; ok; ++i) {
      const int u = unit_of(i);
      __syncwarp();
      if (__any_sync(0xffffffffu, u < 0 || u >= p.n_units)) break;
      if (lane == 0) unit_taken(i);
      const MaskedUnit w = masked_unit<SPLIT>(p, u);
      MaskedTiles it(w);
      const bool mine = SPLIT || t < q_tiles(w);
      const int r = w.r0 + (SPLIT ? 0 : t * 128) + row;
      const bool valid_row = r < p.rows;
      const bool warp_rows = __any_sync(0xffffffffu, valid_row);
      const int token = r % p.S_q, head = w.run % (p.H / p.run_heads) * p.run_heads + r / p.S_q;
      const int pos = w.start + token;
      int lim = p.S_kv, doc = -1;
      float slope = 0.0f;
      if (valid_row) {
        lim = masked_limit(p, pos, w.pre);
        if (w.words != nullptr) {
          doc = __ldg(p.q_doc + static_cast<size_t>(w.b) * p.S_q + token);
          if (doc < 0) lim = 0;
        }
        if (MOD == 2 && p.slopes != nullptr) slope = __ldg(p.slopes + head) / unit;
      }
      float m_use = valid_row ? -INFINITY : 0.0f, l = 0.0f;      // (rows past the end ride along with zero scores)
      bool poison = false, started = false;       // started: every row of the warp has seen a key
      int n = 0, own = 0, j;                     // tiles of the unit, and of this stream
      bool part;
      while (__any_sync(0xffffffffu, it.next(j, part))) {
        const int st = g % NS, gp = (g / NS) & 1;
        ++g;
        ++n;
        if (!mine || (SPLIT && ((n - 1) & 1) != t)) continue;
        ok = __all_sync(0xffffffffu, mbar_wait(bar_s_full + t, ns & 1, abort_flag, tmo, 0x28 + t));
        if (!ok) break;
        ++ns;
        tc_fence_after();
        const bool masked = __any_sync(0xffffffffu, part);   // (votes: the compiler then knows the branches uniform)
        if (warp_rows) {
          uint32_t pw[64];
          float sum = 0.0f, alpha = 1.0f;
          bool need = false;
          // Distance bias, -slope |d - c| at column c with d = position - first key.  Where every row of the warp lies
          // on one side of the tile it is linear in c: a multiply-add with `tilt`, and the rest, `off`, is one
          // number for the row.
          const int d = pos - j * kMaskedTile;
          float tilt = 0.0f, off = 0.0f;
          bool edit = masked;                    // scores rewritten in TMEM first (see below)
          if (MOD == 2) {
            const bool left = __all_sync(0xffffffffu, !valid_row || d >= 127);
            const bool right = __all_sync(0xffffffffu, !valid_row || d <= 0);
            if (!left && !right) edit = true;
            tilt = left ? slope : -slope;
            if (!edit) off = -tilt * static_cast<float>(d);
          }
          if (edit) {
            // Masked tiles, and those that lie on both sides of a row: cap, bias and masks in passes of 32 columns,
            // written back over S.  The rest of the loop then sees plain scores, and its registers, which hold
            // a whole row of S, are spared the masks' state.
            if (masked) {
              ok = __all_sync(0xffffffffu, mbar_wait(bar_v_clean + st, gp, abort_flag, tmo, 0x2A));
              if (!ok) break;
            }
            const int valid = masked ? lim - j * kMaskedTile : kMaskedTile;
            const bool docs = masked && p.words != nullptr;
#pragma unroll 1
            for (int c0 = 0; c0 < kMaskedTile; c0 += 32) {
              uint32_t x[32];
              tmem_ld32_sync(tS + c0, x);
              if (capped) cap_scores(x, cap_c);
              if (MOD == 2) {
                const float df = static_cast<float>(d - c0);
#pragma unroll
                for (int c = 0; c < 32; ++c)
                  x[c] = __float_as_uint(fmaf(-slope, fabsf(df - static_cast<float>(c)), __uint_as_float(x[c])));
              }
              if (docs) {
                const int4* idp = reinterpret_cast<const int4*>(ids + st * 128 + c0);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                  const int4 id = idp[c];
                  if (id.x != doc) x[4 * c] = 0xFF800000u;
                  if (id.y != doc) x[4 * c + 1] = 0xFF800000u;
                  if (id.z != doc) x[4 * c + 2] = 0xFF800000u;
                  if (id.w != doc) x[4 * c + 3] = 0xFF800000u;
                }
              }
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (c >= valid - c0) x[c] = 0xFF800000u;
              if (masked) {
                for (uint32_t m = bad[st * 4 + (c0 >> 5)]; m != 0u; m &= m - 1u) {
                  const int c = c0 + __ffs(m) - 1;
                  poison |= c < valid && (!docs || ids[st * 128 + c] == doc);
                }
              }
              tmem_st32(tS + c0, x);
            }
            tmem_st_wait();
          }
          uint32_t s[128];
          auto scores = [&] {
            tmem_ld128_sync(tS, s);
            if (MOD != 0 && !edit) {
              if (capped) cap_scores(s, cap_c);
              if (MOD == 2) {
#pragma unroll
                for (int c = 0; c < 128; ++c) s[c] = __float_as_uint(fmaf(tilt, static_cast<float>(c), __uint_as_float(s[c])));
              }
            }
          };
          scores();
          bool slow = masked || !started;
          if (!slow) {
            // speculative pass, as in the dense form: the running maximum, kept when the row sums stay bounded
            exp_pass<false, 0>(s, cl, (m_use - off) * cl, pw, sum);
            slow = __any_sync(0xffffffffu, !(sum <= C::kSumBound));
            if (slow) scores();
          }
          if (slow) {
            const float m_new = fmaxf(m_use, row_max128(s) + off);
            need = (m_new - m_use) * cl > C::kRescaleLog2;     // true on a row's first visible tile
            if (need) {
              alpha = ex2_approx((m_use - m_new) * cl);        // 0 when m_use = -inf
              m_use = m_new;
            }
            started = __all_sync(0xffffffffu, m_use != -INFINITY);
            // (a row that has seen no key yet keeps m_use = -inf: exponents of -inf, p = 0)
            exp_pass<false, 0>(s, cl, m_use == -INFINITY ? 0.0f : (m_use - off) * cl, pw, sum);
          }
          tmem_st32(tS, *reinterpret_cast<uint32_t(*)[32]>(&pw[0]));
          tmem_st32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&pw[32]));
          tmem_st_wait();
          // O_t is quiescent here: the P.V of this stream's previous tile completed before S was signalled
          if (own > 0 && __any_sync(0xffffffffu, need)) {
#pragma unroll 1
            for (int cc = 0; cc < D / 32; ++cc) {
              uint32_t o[32];
              tmem_ld32_sync(tO + cc * 32, o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st32(tO + cc * 32, o);
            }
            tmem_st_wait();
          }
          l = fmaf(l, alpha, sum);
        }
        ++own;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_p_full + t);
      }
      if (!ok) break;
      if (!mine) continue;

      // ---------------------------------------------------------------- epilogue
      if (own > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(bar_o_final + t, no & 1, abort_flag, tmo, 0x2B + t));
        if (!ok) break;
        ++no;
        tc_fence_after();
      }
      if (!warp_rows) continue;
      if (poison) l = __int_as_float(0x7FC00000);
      const bool empty = own == 0 || l == 0.0f;                  // no key was visible
      const float inv = empty ? 0.0f : 1.0f / l;
      const float lse = empty ? -INFINITY : unit * m_use + logf(l);
      const size_t row_idx = static_cast<size_t>(w.run) * p.rows + r;
      if constexpr (SPLIT) {
        const size_t n_rows = static_cast<size_t>(p.runs) * p.rows;
        const size_t at = static_cast<size_t>(2 * (u % p.n_split) + t) * n_rows + row_idx;
        if (valid_row) p.part_lse[at] = lse;
        if (own > 0)
#pragma unroll 1
          for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t o[32];
            tmem_ld32_sync(tO + cc * 32, o);
            if (valid_row && !empty) {
              float4* dst = reinterpret_cast<float4*>(p.part_o + at * D + cc * 32);
#pragma unroll
              for (int i = 0; i < 8; ++i)
                dst[i] = make_float4(__uint_as_float(o[4 * i]) * inv, __uint_as_float(o[4 * i + 1]) * inv,
                                     __uint_as_float(o[4 * i + 2]) * inv, __uint_as_float(o[4 * i + 3]) * inv);
            }
          }
      } else {
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t o[32];
          if (own > 0) tmem_ld32_sync(tO + cc * 32, o);
          uint32_t x[16];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            x[i] = empty ? 0u : pack_bf16x2(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
          if (valid_row) {
            uint4* dst = reinterpret_cast<uint4*>(p.out + row_idx * D + cc * 32);
#pragma unroll
            for (int i = 0; i < 4; ++i) dst[i] = make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
          }
        }
        if (valid_row && p.lse != nullptr) p.lse[row_idx] = lse;
      }
      // The O reads above end with tcgen05.wait::ld; the next unit's first P.V (which overwrites O_t)
      // is issued only after this warpgroup publishes that unit's first P_t.
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// Join of the split form's partial results: w_c = exp(lse_c - M) / L, M the largest lse and L the sum of
// weights, out = sum w_c O_c.  One warp per row; the partials of empty shares are not read.
template <int D>
__global__ void __launch_bounds__(128) masked_join_kernel(const MaskedParams p) {
  const int lane = threadIdx.x & 31;
  const long long n_rows = static_cast<long long>(p.B) * p.H * p.S_q;
  const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (row >= n_rows) return;
  const int n = 2 * p.n_split;
  float M = -INFINITY;
  bool nan = false;
  for (int c = lane; c < n; c += 32) {
    const float x = p.part_lse[c * n_rows + row];
    nan |= x != x;
    M = fmaxf(M, x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (__any_sync(0xffffffffu, nan)) M = __int_as_float(0x7FC00000);
  float L = 0.0f, acc[D / 32] = {};
  if (M != -INFINITY) {
    for (int c0 = 0; c0 < n; c0 += 32) {
      const float wl = c0 + lane < n ? __expf(p.part_lse[(c0 + lane) * n_rows + row] - M) : 0.0f;
      const int m = min(32, n - c0);
#pragma unroll 4
      for (int k = 0; k < m; ++k) {
        const float wk = __shfl_sync(0xffffffffu, wl, k);
        L += wk;
        if (wk != 0.0f) {
          const float* o = p.part_o + ((c0 + k) * n_rows + row) * D + lane * (D / 32);
#pragma unroll
          for (int e = 0; e < D / 32; ++e) acc[e] = fmaf(wk, o[e], acc[e]);
        }
      }
    }
  }
  const float inv = M == -INFINITY ? 0.0f : 1.0f / L;
  uint32_t x[D / 64];
#pragma unroll
  for (int e = 0; e < D / 64; ++e) x[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + row * D) + lane * (D / 64);
#pragma unroll
  for (int e = 0; e < D / 64; ++e) dst[e] = x[e];
  if (lane == 0 && p.lse != nullptr) p.lse[row] = M == -INFINITY ? -INFINITY : M + logf(L);
}

}  // namespace dit
