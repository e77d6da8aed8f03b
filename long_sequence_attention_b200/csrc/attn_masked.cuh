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
//   * Long form: a unit is 256 rows as two Q tiles that share each K and V tile.  Units differ in
//     length, so a CTA takes its next one from a counter when it gets there, the longest first.
//   * Split form, for few rows against many keys: a unit is one 128-row Q tile and a share of its
//     KV tiles; the two streams take alternate tiles, each with its own running maximum, sum
//     and O, and the partial results (fp32) are joined by their LSEs in a second kernel.
//   * The TMA thread walks over the KV tiles of its unit, leaves out those that no row sees (past the last
//     visible key; without a document of the rows, by bits that a small kernel writes before), and passes a
//     note on each through shared memory to the other roles: per Q tile, whether it sees none of the
//     tile (then that stream skips it), some of it, or all.  Neighbouring whole tiles share a note.
//   * Tiles that some row sees in part come first.  They take one loop of the softmax, which masks S and
//     takes the exact maximum; the whole tiles take another, the dense form's speculative one, whose
//     registers are then free of the masks' state.  A row's mask is 128 bits: the keys below its limit, and
//     those of its document, which a warp finds for all rows of one document at once (a ballot of 32 keys'
//     ids a word).  Only 16-column pieces that some row of the warp does not see whole are touched.
//   * The two idle warps of the dense form look through the V rows of tiles that are masked for some row: a
//     non-finite value would reach every row of the tile (0 * inf), so it is zeroed in shared memory
//     and its key flagged; the rows that may see that key become NaN, the others never notice.
//
// What bounds it: the hand-offs and the softmax of a tile, as in the dense form (205 us for 24 x 4608 x 128; here,
// without masks, 219), with two softmax warps on a scheduler; a masked tile costs a stream 3.1 us where a whole one
// costs 1.65 (D = 64), of which the mask's bits take 0.5 and their application 0.5.  B200, 24 x 4608 x 128: causal
// 149 us, bias 248, bias and causal 163 (6 key heads), capped 305; 8(4) x 16896 x 128 causal after a prefix of 512:
// 488 us, 1200 TFLOP/s of the pairs that the mask leaves; 2 x 24 x 4429 x 64 in seven documents 158 us; one query of
// 4 x 40(8) heads x 32760 keys 90 us, 5.7 TB/s.
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
  float2 cap_k[6];                  // coefficients of the cap's polynomial in s, twice each (see cap_fold)
  float cap_c, cap_limit;           // scale / cap; largest (s c)^2 that the polynomial is used for, < 0: never
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
  int* cost;                        // documents, more units than CTAs: [B, n_blk] tiles of each unit of rows
  int* order;                       // and (b, unit of rows) by falling cost, as b * n_blk + unit; or null
  uint4* words;                     // [B, n_blk, ceil(S_kv / 4096)] {seen, whole} tile bits of Q tiles 0 and 1, or null
  float* part_o;                    // split form: [2 n_split, B * H * S_q, D]
  float* part_lse;                  // split form: [2 n_split, B * H * S_q]
  unsigned long long timeout_ns;
};

constexpr int kMaskedTile = 128;    // keys of a KV tile

// First key past those that a query at this position may see (documents aside).
__device__ __forceinline__ int masked_limit(const MaskedParams& p, int pos, int pre) {
  return p.causal ? min(max(max(pos + 1, pre), 0), p.S_kv) : p.S_kv;
}

// Query rows r0.. of run `run`, of sequence b; its share of the KV tiles (split form).
struct MaskedUnit {
  int run, b, r0, blk, share;
};

// Units are handed out for all runs of a sequence at a time, the blocks of rows with the longest walks first: by
// `order`, else (causal masks) the last rows first.
template <bool SPLIT>
__device__ __forceinline__ MaskedUnit masked_unit(const MaskedParams& p, int u) {
  MaskedUnit w;
  w.share = SPLIT ? u % p.n_split : 0;
  if (SPLIT) u /= p.n_split;
  const int per_b = p.H / p.run_heads, at = u / per_b;
  if (p.order != nullptr) {
    const int x = p.order[at];
    w.b = x / p.n_blk;
    w.blk = x - w.b * p.n_blk;
  } else {
    w.b = at % p.B;
    w.blk = p.n_blk - 1 - at / p.B;
  }
  w.run = w.b * per_b + u % per_b;
  w.r0 = w.blk * (SPLIT ? 128 : 256);
  return w;
}

// A note on n KV tiles of a unit (|n| neighbours; n < 0: downwards), from the TMA thread to the other roles; with the
// unit's run, rows and share.  masked: some row does not see some key.  x, low bits: the first tile; 3 bits for each Q tile (the
// split form: both the same); then what the note is.
constexpr int kNoteTile = (1 << 23) - 1;           // S_kv <= 2^30
constexpr int kNoteNone = 1, kNoteRange = 2, kNoteDocs = 4;   // sees nothing; some keys past a row's limit; ids to compare
constexpr int kNoteShift = 23;                     // Q tile t's bits at kNoteShift + 3 t
constexpr int kNoteWhole = 1 << 29;                // (a whole tile: no row masks a key, and it lies to one side of every row)
constexpr int kNoteLast = 1 << 30;                 // the unit's last note
constexpr int kNoteEmpty = static_cast<int>(1u << 31);   // no tile: a unit whose rows see nothing, or (run < 0) the end

__device__ __forceinline__ int note_class(int note, int t) { return (note >> (kNoteShift + 3 * t)) & 7; }

// The TMA thread's walk.  Ranges of tiles without a document mask: [js, je) lie on both sides of some row (distance
// bias only), [jw, j1) hold a key past some row's limit, the others are whole.  Order: the first two kinds, then
// (documents) the other tiles that a row sees in part, then the whole ones, downwards below js and upwards above
// je.  So with a bias it goes outwards from the rows' own positions, where the scores are largest, and the first
// tile, which takes the exact path anyhow, settles the running maximum.
template <bool SPLIT>
struct MaskedWalk {
  const uint4* words;
  int j0, j1, js, je, jw;
  int end[2], whole[2];              // of each Q tile: first key that no row sees, first key that some row does not see
  int seg, j, stop;
  bool up, two;                      // two: rows in both Q tiles
  int at;
  uint4 x;

  __device__ __forceinline__ MaskedWalk(const MaskedParams& p, const MaskedUnit& w, int start, int pre) {
    int lo[2], hi[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int r = w.r0 + (SPLIT ? 0 : t * 128), last = min(r + 128, p.rows) - 1;
      end[t] = whole[t] = 0;
      lo[t] = hi[t] = 0;
      if (r >= p.rows) continue;     // no rows: sees nothing
      const bool one_head = r / p.S_q == last / p.S_q;
      lo[t] = start + (one_head ? r % p.S_q : 0);
      hi[t] = start + (one_head ? last % p.S_q : p.S_q - 1);
      end[t] = masked_limit(p, hi[t], pre);
      whole[t] = masked_limit(p, lo[t], pre);
    }
    two = !SPLIT && p.rows - w.r0 > 128;
    const int n = (max(end[0], end[1]) + kMaskedTile - 1) / kMaskedTile;
    j0 = 0;
    j1 = n;
    if constexpr (SPLIT) {
      const int per = (n + p.n_split - 1) / p.n_split;
      j0 = min(n, w.share * per);
      j1 = min(n, j0 + per);
    }
    jw = min(max((two ? min(whole[0], whole[1]) : whole[0]) / kMaskedTile, j0), j1);
    js = je = jw;
    if (p.slopes != nullptr) {
      const int a = two ? min(lo[0], lo[1]) : lo[0], b = two ? max(hi[0], hi[1]) : hi[0];
      js = min(max(a >= 0 ? a / kMaskedTile : 0, j0), j1);
      je = min(max(b >= 0 ? b / kMaskedTile + 1 : 0, js), j1);
      js = min(js, jw);
      jw = max(jw, je);
    }
    words = p.words ? p.words + (static_cast<size_t>(w.b) * p.n_blk + w.blk) *
                                    ((p.S_kv + 32 * kMaskedTile - 1) / (32 * kMaskedTile))
                    : nullptr;
    at = -1;
    seg = -1;
    j = 0;
    stop = 1;
    up = false;
  }

  // Segments: 0 [js, je) down, 1 [jw, j1) down; documents: 2 [j0, js) down and 3 [je, jw) up in part; 4, 5 the same, whole.
  __device__ __forceinline__ bool next(int& note, int& run, bool& masked) {
    while (true) {
      if (up ? j >= stop : j < stop) {
        if (++seg == 2 && words == nullptr) seg = 4;
        if (seg > 5) return false;
        up = seg & 1 && seg > 1;
        if (seg == 0) { j = je - 1; stop = js; }
        else if (seg == 1) { j = j1 - 1; stop = jw; }
        else if (up) { j = je; stop = jw; }
        else { j = js - 1; stop = j0; }
        continue;
      }
      if (words != nullptr) {
        if ((j >> 5) != at) {
          at = j >> 5;
          x = words[at];
        }
        uint32_t m = x.x | x.z;
        if (seg >= 2) m &= seg < 4 ? ~(x.y & x.w) : (x.y & x.w);
        m &= up ? 0xFFFFFFFFu << (j & 31) : 0xFFFFFFFFu >> (31 - (j & 31));
        if (m == 0u) {
          j = up ? (at + 1) << 5 : (at << 5) - 1;
          continue;
        }
        j = (at << 5) + (up ? __ffs(m) - 1 : 31 - __clz(m));
        if (up ? j >= stop : j < stop) continue;
      }
      int n = j;
      const int bit = j & 31;
      run = up ? 1 : -1;
      if (seg >= 4) {                // whole tiles: as many as follow one another (documents: within a word)
        int len = up ? stop - j : j - stop + 1;
        if (words != nullptr) {
          const uint32_t m = ~(x.y & x.w);
          len = min(len, up ? (m >> bit ? __ffs(m >> bit) - 1 : 32 - bit)
                            : (m << (31 - bit) ? __clz(m << (31 - bit)) : bit + 1));
        }
        run = up ? len : -len;
      }
      j += run;
      int none = 0;
      masked = false;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int k = n & kNoteTile;
        int c = 0;
        if (k * kMaskedTile >= end[t]) c = kNoteNone;
        else if ((k + 1) * kMaskedTile > whole[t]) c = kNoteRange;
        if (words != nullptr) {
          const uint32_t seen = t ? x.z : x.x, all = t ? x.w : x.y;
          if (!((seen >> bit) & 1u)) c = kNoteNone;
          else if (!((all >> bit) & 1u) && c != kNoteNone) c |= kNoteDocs;
        }
        none += c == kNoteNone;
        masked |= c != 0 && (t == 0 || SPLIT || two);
        n |= c << (kNoteShift + 3 * t);
      }
      if (none == 2) continue;
      note = n | (seg >= 4 ? kNoteWhole : 0);
      return true;
    }
  }
};

// Documents: bit j of a unit's words says, for each of its Q tiles, whether KV tile j holds a key whose document
// lies between the smallest and largest document of the Q tile's rows (seen), and whether all of both are one
// document (whole).  One CTA per (b, unit of rows); reads S_kv + 256 ids, a few KB that stay in L2.
template <bool SPLIT>
__global__ void __launch_bounds__(256) masked_tiles_kernel(const MaskedParams p) {
  __shared__ int red[3][8];
  __shared__ uint4 part[8];
  grid_dep_launch();
  const int blk = blockIdx.x % p.n_blk, b = blockIdx.x / p.n_blk;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_words = (p.S_kv + 32 * kMaskedTile - 1) / (32 * kMaskedTile);
  const int r = SPLIT ? blk * 128 + static_cast<int>(threadIdx.x & 127) : blk * 256 + static_cast<int>(threadIdx.x);
  int lo = 0x7FFFFFFF, hi = -1, pad = 0;
  if (r < p.rows) {
    const int id = p.q_doc[static_cast<size_t>(b) * p.S_q + r % p.S_q];
    pad = id < 0;
    if (!pad) lo = hi = id;
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  pad = __reduce_max_sync(0xffffffffu, pad);
  if (lane == 0) { red[0][warp] = lo; red[1][warp] = hi; red[2][warp] = pad; }
  __syncthreads();
  int qlo[2], qhi[2];
  bool one[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    qlo[t] = 0x7FFFFFFF;
    qhi[t] = -1;
    int q_pad = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      qlo[t] = min(qlo[t], red[0][4 * t + i]);
      qhi[t] = max(qhi[t], red[1][4 * t + i]);
      q_pad = max(q_pad, red[2][4 * t + i]);
    }
    one[t] = qlo[t] == qhi[t] && !q_pad;
  }
  const bool absent = !SPLIT && blk * 256 + 128 >= p.rows;   // no second Q tile: it does not keep tiles from being whole
  const int* kd = p.kv_doc + static_cast<size_t>(b) * p.S_kv;
  uint4* words = p.words + static_cast<size_t>(blockIdx.x) * n_words;
  // tiles past the causal limit of the unit's last row do not count
  int n_tiles = 0, cost = 0;
  {
    const int last = min((blk + 1) * (SPLIT ? 128 : 256), p.rows) - 1, first = blk * (SPLIT ? 128 : 256);
    const int hi = first / p.S_q == last / p.S_q ? last % p.S_q : p.S_q - 1;
    n_tiles = (masked_limit(p, (p.q_start ? p.q_start[b] : p.S_kv - p.S_q) + hi, p.prefix ? p.prefix[b] : 0) + kMaskedTile - 1) /
              kMaskedTile;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.next_unit != nullptr) *p.next_unit = 0u;
  // 32 tiles at a time, four to a warp: sixteen loads of a lane in flight
  for (int w = 0; w < n_words; ++w) {
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
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
      int klo = 0x7FFFFFFF, khi = -1;
      bool kpad = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        kpad |= id[t][i] < 0;
        klo = min(klo, id[t][i] < 0 ? 0x7FFFFFFF : id[t][i]);
        khi = max(khi, id[t][i]);
      }
      klo = __reduce_min_sync(0xffffffffu, klo);
      khi = __reduce_max_sync(0xffffffffu, khi);
      kpad = __any_sync(0xffffffffu, kpad);
      const uint32_t bit = 1u << (warp * 4 + t);
      if (khi >= qlo[0] && klo <= qhi[0] && qhi[0] >= 0 && khi >= 0) x.x |= bit;
      if (one[0] && klo == khi && klo == qlo[0] && !kpad) x.y |= bit;
      if (khi >= qlo[1] && klo <= qhi[1] && qhi[1] >= 0 && khi >= 0) x.z |= bit;
      if (absent || (one[1] && klo == khi && klo == qlo[1] && !kpad)) x.w |= bit;
    }
    if (lane == 0) part[warp] = x;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
      for (int i = 1; i < 8; ++i) { x.x |= part[i].x; x.y |= part[i].y; x.z |= part[i].z; x.w |= part[i].w; }
      words[w] = x;
      const int left = n_tiles - w * 32;
      if (left > 0) cost += __popc((x.x | x.z) & (left < 32 ? (1u << left) - 1u : 0xFFFFFFFFu));
    }
    __syncthreads();
  }
  if (threadIdx.x == 0 && p.cost != nullptr) p.cost[blockIdx.x] = cost;
}

// Units by falling cost: a counting sort over 256 classes, one CTA.  (Units of one class come in any order: it
// changes who computes what when, not what.)
__global__ void __launch_bounds__(1024) masked_order_kernel(const MaskedParams p) {
  __shared__ int most, at[256];
  grid_dep_launch();
  const int n = p.B * p.n_blk;
  if (threadIdx.x == 0) most = 0;
  if (threadIdx.x < 256) at[threadIdx.x] = 0;
  __syncthreads();
  grid_dep_wait();
  int m = 0;
  for (int i = threadIdx.x; i < n; i += 1024) m = max(m, p.cost[i]);
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) atomicMax(&most, m);
  __syncthreads();
  const int shift = max(0, 32 - __clz(most) - 8);
  for (int i = threadIdx.x; i < n; i += 1024) atomicAdd(&at[p.cost[i] >> shift], 1);
  __syncthreads();
  if (threadIdx.x < 32) {                         // first place of each class, the largest class first
    int c[8], sum = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      c[k] = sum;
      sum += at[255 - (threadIdx.x * 8 + k)];
    }
    int before = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, before, o);
      if (static_cast<int>(threadIdx.x) >= o) before += y;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) at[255 - (threadIdx.x * 8 + k)] = before - sum + c[k];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += 1024) p.order[atomicAdd(&at[p.cost[i] >> shift], 1)] = i;
}

template <int D, bool SPLIT>
struct MaskedCfg {
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kBlkBytes = 128 * 128;
  static constexpr int kNBlk = D / 64;
  static constexpr int kQTiles = SPLIT ? 1 : 2;
  // Q tiles of the next unit while this one's are in use, where there is room: its first S then need not wait for them
  static constexpr int kQBufs = D == 64 && !SPLIT ? 2 : 1;
  // D = 128: 2 Q + 2 K + 2 V tiles, or 1 + 3 + 3; D = 64: 4 + 4 + 4, or 1 + 6 + 6 (tiles of 16 KB)
  static constexpr int kStages = D == 128 ? (SPLIT ? 3 : 2) : (SPLIT ? 6 : 4);
  static constexpr int kThreads = 384;
  static constexpr int kRegsLaunch = 168, kRegsSoftmax = 216, kRegsCtl = 72;
  static_assert(2 * 128 * kRegsSoftmax + 128 * kRegsCtl <= kThreads * kRegsLaunch, "register split");
  static constexpr int kMmaWarp = 8, kTmaWarp = 9, kVWarp = 10;
  static constexpr int kColS0 = 0, kColS1 = 128, kColO0 = 256, kColO1 = 256 + D;
  // P, O and l are floating point, so a running maximum 2^40 below the true one costs no precision (dense form:
  // 2^8): loud scores then hardly ever leave the speculative path
  static constexpr float kRescaleLog2 = 40.0f, kSumBound = 1099511627776.0f;
  static constexpr int kOffK = kQBufs * kQTiles * kTileBytes;
  static constexpr int kOffV = kOffK + kStages * kTileBytes;
  static constexpr int kOffIds = kOffV + kStages * kTileBytes;      // documents of the tile's keys, per V stage
  static constexpr int kOffBad = kOffIds + kStages * 512;           // 128 bits of flagged keys, per V stage
  static constexpr int kOffBar = kOffBad + kStages * 16;
  static constexpr int kNotes = 4;                                   // notes not yet read by every role
  static constexpr int kNoteReaders = 1 + 8;                        // MMA and softmax warps
  static constexpr int kVNotes = 2;                                 // notes on masked tiles for the V warps
  static constexpr int kNumBars = 2 * kQBufs + 5 * kStages + 6 + 1 + 2 * kNotes + 2 * kVNotes;
  static constexpr int kOffMisc = kOffBar + 8 * kNumBars;
  static constexpr int kSmemBytes = kOffMisc + 16 + 32 * kNotes + 16 * kVNotes + 1024;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
};

// Capping, tanh(x) with x = s c, c = scale / cap: x p(x^2) with p of degree 5 where every |x| <= 1 in the warp's tile
// (fit_tanh_poly.py; relative error 6e-7), the usual case, since a cap is meant for rare large scores; else by
// exponentials.  The polynomial runs on the FMA pipe, whose packed instructions take it 2 cycles each, while the
// special-function unit is busy with the softmax's exponentials; c is folded into the coefficients, k[i] = p_i
// c^(2i + 1), which saves one instruction a pair.  They come as kernel parameters, doubled for the packed
// instructions, and so take no registers.  Powers of a small c leave fp32's range: from 5e-4 down |x| <= 1/4 is
// asked for, where c^9 and c^11 do not matter, and below 5e-6 (c^7) the exponentials take over.
inline void cap_fold(MaskedParams& p) {
  const double poly[6] = {0.9999994039535522, -0.3332904279232025,  0.13281433284282684,
                          -0.051605675369501114, 0.016743116080760956, -0.003067060373723507};
  const double c = p.cap > 0.0f ? static_cast<double>(p.scale) / p.cap : 0.0;
  double f = c;
  for (int i = 0; i < 6; ++i, f *= c * c) p.cap_k[i] = make_float2(static_cast<float>(poly[i] * f), static_cast<float>(poly[i] * f));
  p.cap_c = static_cast<float>(c);
  p.cap_limit = c > 5e-4 && c < 1e3 ? 1.0f : (c > 5e-6 && c < 1e3 ? 0.0625f : -1.0f);
}
__device__ __forceinline__ uint64_t cap_coef(const MaskedParams& p, int i) { return f2_pack(p.cap_k[i].x, p.cap_k[i].y); }

// tanh of a pair of scores; t = the pair's squares.
__device__ __forceinline__ uint64_t cap_pair(uint64_t x, const MaskedParams& p, uint64_t& t) {
  t = f2_mul(x, x);
  uint64_t r = cap_coef(p, 5);
#pragma unroll
  for (int i = 4; i >= 0; --i) r = f2_fma(r, t, cap_coef(p, i));
  return f2_mul(x, r);
}

// By the exponential, any x: 1 - 2 / (1 + e^2x), within 3e-7 absolutely.
__device__ __forceinline__ float tanh_any(float x) {
  return 1.0f - __fdividef(2.0f, 1.0f + ex2_approx(x * 2.8853900817779268f));
}

// Scores s -> tanh(s c) in place by the polynomial (the caller's unit becomes the cap); returns the largest s^2.
__device__ __forceinline__ float cap_poly(uint32_t (&s)[128], const MaskedParams& p) {
  float m[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 64; ++i) {
    uint64_t t;
    float a, b, t0, t1;
    f2_unpack(cap_pair(f2_pack(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), p, t), a, b);
    f2_unpack(t, t0, t1);
    m[i & 3] = fmax3(m[i & 3], t0, t1);
    s[2 * i] = __float_as_uint(a);
    s[2 * i + 1] = __float_as_uint(b);
  }
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// The same and the exponentials in one pass, so that the one's FMA work runs under the other's special-function work:
// p = 2^(cl * tanh(s c) - mc), the P words and the row sum; returns the largest s^2.
__device__ __forceinline__ float cap_exp_pass(const uint32_t (&s)[128], const MaskedParams& p, float cl, float mc,
                                              uint32_t (&pw)[64], float& sum) {
  float m[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  const uint64_t cl2 = f2_pack(cl, cl), nmc2 = f2_pack(-mc, -mc);
  uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
  for (int i = 0; i < 64; ++i) {
    uint64_t t;
    float a, b, t0, t1;
    f2_unpack(f2_fma(cap_pair(f2_pack(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), p, t), cl2, nmc2), a, b);
    f2_unpack(t, t0, t1);
    m[i & 3] = fmax3(m[i & 3], t0, t1);
    a = ex2_approx(a);
    b = ex2_approx(b);
    acc[i & 3] = f2_add(acc[i & 3], f2_pack(a, b));
    pw[i] = pack_bf16x2(a, b);
  }
  float lo, hi;
  f2_unpack(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), lo, hi);
  sum = lo + hi;
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// MOD: what is done to the scores, fixed at compile time because the softmax's registers are full: 1 the cap, 2 the
// distance bias (3 both).
template <int D, bool SPLIT, int MOD>
__global__ void __launch_bounds__(384, 1)
    attn_masked_kernel(const __grid_constant__ MapSet<1> maps, const MaskedParams p) {
  using C = MaskedCfg<D, SPLIT>;
  constexpr int NS = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* bar_q_full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  constexpr int NQ = C::kQBufs;
  uint64_t* bar_q_empty = bar_q_full + NQ;            // [NQ] (and bar_q_full)
  uint64_t* bar_k_full = bar_q_empty + NQ;            // [NS]
  uint64_t* bar_k_empty = bar_k_full + NS;            // [NS]
  uint64_t* bar_v_full = bar_k_empty + NS;            // [NS] V has landed
  uint64_t* bar_v_clean = bar_v_full + NS;            // [NS] and holds finite values where it is masked
  uint64_t* bar_v_empty = bar_v_clean + NS;           // [NS]
  uint64_t* bar_s_full = bar_v_empty + NS;            // [2]
  uint64_t* bar_p_full = bar_s_full + 2;              // [2]
  uint64_t* bar_o_final = bar_p_full + 2;             // [2]
  uint64_t* bar_drain = bar_o_final + 2;
  uint64_t* bar_n_full = bar_drain + 1;               // [kNotes]
  uint64_t* bar_n_empty = bar_n_full + C::kNotes;     // [kNotes]
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  uint64_t* bar_w_full = bar_n_empty + C::kNotes;     // [kVNotes]
  uint64_t* bar_w_empty = bar_w_full + C::kVNotes;    // [kVNotes]
  // [kNotes] {x, run, rows, share, n, masked, start, prefix}, [kVNotes] {x, b, running tile, -}
  volatile int* notes = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 16);
  volatile int* v_notes = notes + 8 * C::kNotes;
  int* ids = reinterpret_cast<int*>(smem + C::kOffIds);
  uint32_t* bad = reinterpret_cast<uint32_t*>(smem + C::kOffBad);
  uint8_t* sQ = smem;
  uint8_t* sK = smem + C::kOffK;
  uint8_t* sV = smem + C::kOffV;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint64_t tmo = p.timeout_ns;

  if (SPLIT) grid_dep_launch();                  // the join may take its place as soon as CTAs leave
  if (threadIdx.x == C::kTmaWarp * 32) {
    for (int s = 0; s < NQ; ++s) {
      mbar_init(bar_q_full + s, 1);
      mbar_init(bar_q_empty + s, 1);
    }
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
    for (int s = 0; s < C::kNotes; ++s) {
      mbar_init(bar_n_full + s, 1);
      mbar_init(bar_n_empty + s, C::kNoteReaders);
    }
    for (int s = 0; s < C::kVNotes; ++s) {
      mbar_init(bar_w_full + s, 1);
      mbar_init(bar_w_empty + s, 2);
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

  // The i-th note.  Every reading warp frees its slot once (note_read).  Giving up reads as the end.
  struct Note { int x, run, n, masked; };
  auto note_at = [&](int i) {
    volatile int* e = notes + 8 * (i % C::kNotes);
    if (!mbar_wait(bar_n_full + i % C::kNotes, (i / C::kNotes) & 1, abort_flag, tmo, 0x2D)) return Note{kNoteEmpty, -1, 0, 0};
    return Note{e[0], e[1], e[4], e[5]};
  };
  auto note_read = [&](int i) { mbar_arrive(bar_n_empty + i % C::kNotes); };

  if (warp >= 8) {
    regs_dec<C::kRegsCtl>();
    if (warp == C::kTmaWarp) {
      // ---------------------------------------------------------------- TMA producer
      if (lane == 0) {
        tma_prefetch_desc(&maps.q[0]);
        tma_prefetch_desc(&maps.k[0]);
        tma_prefetch_desc(&maps.v[0]);
        grid_dep_wait();                         // (the tile bits and the unit counter of this call)
        int g = 0, nq = 0, nn = 0, nv = 0, k_issued = 0, v_issued = 0;   // running tile, Q and note counts
        bool ok = true;
        MaskedUnit w;
        int start = 0, pre = 0;
        auto put = [&](int x, int run, int n, bool masked) {
          const int slot = nn % C::kNotes;
          if (nn >= C::kNotes && !mbar_wait(bar_n_empty + slot, ((nn / C::kNotes) + 1) & 1, abort_flag, tmo, 0x2E)) return false;
          volatile int* e = notes + 8 * slot;
          e[0] = x;
          e[1] = run;
          e[2] = w.r0;
          e[3] = w.share;
          e[4] = n;
          e[5] = masked;
          e[6] = start;
          e[7] = pre;
          mbar_arrive(bar_n_full + slot);
          ++nn;
          return true;
        };
        auto put_v = [&](int x, int b) {
          const int slot = nv % C::kVNotes;
          if (nv >= C::kVNotes && !mbar_wait(bar_w_empty + slot, ((nv / C::kVNotes) + 1) & 1, abort_flag, tmo, 0x2F)) return false;
          v_notes[4 * slot] = x;
          v_notes[4 * slot + 1] = b;
          v_notes[4 * slot + 2] = g;
          mbar_arrive(bar_w_full + slot);
          ++nv;
          return true;
        };
        int u = blockIdx.x;
        while (ok && u < p.n_units) {
          w = masked_unit<SPLIT>(p, u);
          start = p.q_start ? __ldg(p.q_start + w.b) : p.S_kv - p.S_q;
          pre = p.prefix ? __ldg(p.prefix + w.b) : 0;
          const int u_next = p.next_unit ? static_cast<int>(gridDim.x + atomicAdd(p.next_unit, 1u))
                                         : u + static_cast<int>(gridDim.x);
          MaskedWalk<SPLIT> walk(p, w, start, pre);
          const int kv = w.b * p.H_kv + (w.run % (p.H / p.run_heads)) * p.run_heads / (p.H / p.H_kv);
          int ahead = 0, ahead_run = 0;
          bool ahead_masked = false;
          bool more = walk.next(ahead, ahead_run, ahead_masked);
          if (!more) {
            ok = put(kNoteEmpty, w.run, 0, false);
          }
          bool q_here = false;
          while (ok && more) {
            const int note = ahead;
            int run = ahead_run;
            const bool masked = ahead_masked;
            more = walk.next(ahead, ahead_run, ahead_masked);
            if (!(ok = put(note | (more ? 0 : kNoteLast), w.run, run, masked))) break;
            const int step = run < 0 ? -1 : 1;
            for (int j = note & kNoteTile; run != 0; j += step, run -= step) {
              const int st = g % NS;
              if (g >= NS && !(ok = mbar_wait(bar_k_empty + st, ((g / NS) + 1) & 1, abort_flag, tmo, 0x21))) break;
              mbar_arrive_expect_tx(bar_k_full + st, C::kTileBytes);
              for (int b = 0; b < C::kNBlk; ++b)
                tma_load_4d(sK + st * C::kTileBytes + b * C::kBlkBytes, &maps.k[0], bar_k_full + st, b * 64,
                            j * kMaskedTile, kv, 0);
              k_issued = g + 1;
              if (!q_here) {                     // after the first K, which need not wait for the last unit's S
                q_here = true;
                const int qb = nq % NQ;
                if (nq >= NQ && !(ok = mbar_wait(bar_q_empty + qb, ((nq / NQ) + 1) & 1, abort_flag, tmo, 0x20))) break;
                const int nt = SPLIT || p.rows - w.r0 <= 128 ? 1 : 2;
                mbar_arrive_expect_tx(bar_q_full + qb, nt * C::kTileBytes);
                for (int t = 0; t < nt; ++t)
                  for (int b = 0; b < C::kNBlk; ++b)
                    tma_load_4d(sQ + (qb * C::kQTiles + t) * C::kTileBytes + b * C::kBlkBytes, &maps.q[0], bar_q_full + qb,
                                b * 64, w.r0 + t * 128, w.run, 0);
                ++nq;
              }
              if (g >= NS && !(ok = mbar_wait(bar_v_empty + st, ((g / NS) + 1) & 1, abort_flag, tmo, 0x22))) break;
              // (only now: the V warps wait on bar_v_full of masked tiles alone, and the phase before this tile's has to
              // be over when they do, or they would take that one for it)
              if (masked && !(ok = put_v(note, w.b))) break;
              mbar_arrive_expect_tx(bar_v_full + st, C::kTileBytes);
              for (int b = 0; b < C::kNBlk; ++b)
                tma_load_4d(sV + st * C::kTileBytes + b * C::kBlkBytes, &maps.v[0], bar_v_full + st, b * 64,
                            j * kMaskedTile, kv, 0);
              v_issued = ++g;
            }
          }
          u = u_next;
        }
        if (ok) ok = put(kNoteEmpty, -1, 0, false);
        if (ok) put_v(kNoteEmpty, -1);
        // the last load of every stage must land before the CTA may exit
        for (int r = 0; r < NQ; ++r)
          if (nq > r) mbar_wait_drain(bar_q_full + r, ((nq - 1 - r) / NQ) & 1, tmo);
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
        auto issue_s = [&](int t, int st, int qb) {
          const uint32_t a0 = q_lo + (((qb * C::kQTiles + (SPLIT ? 0 : t)) * C::kTileBytes) >> 4);
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
        // V of running tile gt: as it landed, or, of a masked tile, as the V warps left it.  They see masked tiles
        // only; for the others this thread turns bar_v_clean in their place, so that its phases stay in step.
        auto wait_v = [&](int gt, bool masked) {
          const int vs = gt % NS, ph = (gt / NS) & 1;
          if (masked) return mbar_wait(bar_v_clean + vs, ph, abort_flag, tmo, 0x24);
          if (!mbar_wait(bar_v_full + vs, ph, abort_flag, tmo, 0x24)) return false;
          mbar_arrive(bar_v_clean + vs);
          mbar_arrive(bar_v_clean + vs);
          return true;
        };
        auto wait_p = [&](int t) {
          const bool r = mbar_wait(bar_p_full + t, np[t] & 1, abort_flag, tmo, 0x25);
          ++np[t];
          return r;
        };
        for (int i = 0; ok;) {
          Note e = note_at(i);
          if (e.run < 0) break;
          if (e.x & kNoteEmpty) {
            note_read(i++);
            continue;
          }
          const int qb = nq % NQ;
          if (!(ok = mbar_wait(bar_q_full + qb, (nq / NQ) & 1, abort_flag, tmo, 0x26))) break;
          ++nq;
          int n = 0;                             // tiles of this unit so far
          int prev = 0, begun = 0;               // streams that own the previous tile, that have begun their O
          bool prev_masked = false, prev2_masked = false;
          while (true) {
            note_read(i++);
            const int own = (note_class(e.x, 0) != kNoteNone ? 1 : 0) | (note_class(e.x, 1) != kNoteNone ? 2 : 0);
            for (int left = e.n < 0 ? -e.n : e.n; left > 0; --left) {
              const int st = g % NS;
              if (!(ok = mbar_wait(bar_k_full + st, (g / NS) & 1, abort_flag, tmo, 0x23))) break;
              tc_fence_after();
              if constexpr (SPLIT) {
                // stream t takes every other tile; its previous one is two back
                const int t = n & 1;
                if (n >= 2) {
                  if (!(ok = wait_v(g - 2, prev2_masked) && wait_p(t))) break;
                  tc_fence_after();
                  issue_pv(t, (g - 2) % NS, n >= 4);
                  tc_commit(bar_v_empty + (g - 2) % NS);
                }
                issue_s(t, st, qb);
                tc_commit(bar_s_full + t);
                prev2_masked = prev_masked;
              } else {
                const int vs = (g - 1 + NS) % NS;
                if (prev && !(ok = wait_v(g - 1, prev_masked))) break;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                  if (prev & (1 << t)) {
                    if (!(ok = wait_p(t))) break;
                    tc_fence_after();
                    issue_pv(t, vs, begun & (1 << t));
                    begun |= 1 << t;
                  }
                  if (t == 1 && prev) tc_commit(bar_v_empty + vs);
                  if (own & (1 << t)) {
                    issue_s(t, st, qb);
                    tc_commit(bar_s_full + t);
                  }
                }
                if (!ok) break;
                prev = own;
              }
              prev_masked = e.masked;
              tc_commit(bar_k_empty + st);
              ++g;
              ++n;
            }
            if (!ok || (e.x & kNoteLast)) break;
            e = note_at(i);
            if (!(ok = e.run >= 0)) break;
          }
          if (!ok) break;
          tc_commit(bar_q_empty + qb);           // every S MMA of this unit is issued
          if constexpr (SPLIT) {
            for (int k = n >= 2 ? n - 2 : 0; ok && k < n; ++k) {
              const int t = k & 1, gt = g - n + k;
              if (!(ok = wait_v(gt, k == n - 1 ? prev_masked : prev2_masked) && wait_p(t))) break;
              tc_fence_after();
              issue_pv(t, gt % NS, k >= 2);
              tc_commit(bar_o_final + t);
              tc_commit(bar_v_empty + gt % NS);
            }
          } else {
            const int vs = (g - 1) % NS;
            ok = wait_v(g - 1, prev_masked);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (ok && (prev & (1 << t))) {
                if ((ok = wait_p(t))) {
                  tc_fence_after();
                  issue_pv(t, vs, begun & (1 << t));
                  begun |= 1 << t;
                }
              }
              if (ok && (begun & (1 << t))) tc_commit(bar_o_final + t);
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
      for (int i = 0; ok; ++i) {
        const int slot = i % C::kVNotes;
        ok = __all_sync(0xffffffffu, mbar_wait(bar_w_full + slot, (i / C::kVNotes) & 1, abort_flag, tmo, 0x30));
        if (!ok) break;
        const int x = v_notes[4 * slot], b = v_notes[4 * slot + 1], g = v_notes[4 * slot + 2];
        __syncwarp();
        if (__any_sync(0xffffffffu, b < 0)) break;
        if (lane == 0) mbar_arrive(bar_w_empty + slot);
        const bool docs = p.words != nullptr && ((note_class(x, 0) | note_class(x, 1)) & kNoteDocs);
        {
          const int st = g % NS;
          int id0 = -1, id1 = -1;
          if (docs) {
            const int k = (x & kNoteTile) * kMaskedTile + half * 64 + lane;
            const int* kd = p.kv_doc + static_cast<size_t>(b) * p.S_kv;
            if (k < p.S_kv) id0 = max(__ldg(kd + k), -1);
            if (k + 32 < p.S_kv) id1 = max(__ldg(kd + k + 32), -1);
          }
          ok = __all_sync(0xffffffffu, mbar_wait(bar_v_full + st, (g / NS) & 1, abort_flag, tmo, 0x27));
          if (!ok) break;
          {
            if (docs) {
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
              for (int r4 = 0; r4 < 16; ++r4) {
                const uint4 q = base[r4 * 32 + lane];
                const uint32_t e = ((q.x & 0x7F807F80u) + 0x00800080u) | ((q.y & 0x7F807F80u) + 0x00800080u) |
                                   ((q.z & 0x7F807F80u) + 0x00800080u) | ((q.w & 0x7F807F80u) + 0x00800080u);
                if (e & 0x80008000u) {
                  auto clean = [](uint32_t v) {
                    if ((v & 0x7F80u) == 0x7F80u) v &= 0xFFFF0000u;
                    if ((v & 0x7F800000u) == 0x7F800000u) v &= 0x0000FFFFu;
                    return v;
                  };
                  base[r4 * 32 + lane] = make_uint4(clean(q.x), clean(q.y), clean(q.z), clean(q.w));
                  const int r = r4 * 4 + (lane >> 3);             // key within this half
                  atomicOr(&bad[st * 4 + half * 2 + (r >> 5)], 1u << (r & 31));
                }
              }
            }
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_v_clean + st);
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
    const bool capped = (MOD & 1) && p.cap > 0.0f;             // (split form: one kernel for every change)
    const float unit = capped ? p.cap : p.scale;
    const float cl = unit * 1.4426950408889634f;
    // (s c)^2 within the polynomial's range, for the largest s^2 of each row of the warp
    auto cap_fits = [&](float t) { return t * p.cap_c * p.cap_c <= p.cap_limit; };
    // S of this stream's tile, capped
    auto load_s = [&](uint32_t (&s)[128]) {
      tmem_ld128_sync(tS, s);
      if (capped) {
        if (p.cap_limit > 0.0f) {
          const float t = cap_poly(s, p);
          if (__all_sync(0xffffffffu, cap_fits(t))) return;
          tmem_ld128_sync(tS, s);
        }
#pragma unroll
        for (int k = 0; k < 128; ++k) s[k] = __float_as_uint(tanh_any(__uint_as_float(s[k]) * p.cap_c));
      }
    };
    bool ok = true;
    int g = 0, ns = 0, no = 0;                   // running tiles of the CTA, S tiles and O's of this stream

    // A row of a unit: its place in its run, its position among the keys, the first key past those it may see, its
    // document (-2: no key's; padding's is -1) and its slope in the scores' unit.
    struct Row { int run, share, r, pos, lim, doc; float slope; };
    auto row_of = [&](int i, int run) {
      volatile int* info = notes + 8 * (i % C::kNotes);
      Row q;
      q.run = run;
      q.share = info[3];
      q.r = info[2] + (SPLIT ? 0 : t * 128) + row;
      const int per_b = p.H / p.run_heads, b = run / per_b, token = q.r % p.S_q;
      q.pos = info[6] + token;
      q.lim = p.S_kv;
      q.doc = -2;
      q.slope = 0.0f;
      if (run >= 0 && q.r < p.rows) {
        if (p.words != nullptr) q.doc = max(__ldg(p.q_doc + static_cast<size_t>(b) * p.S_q + token), -2);
        if (q.doc == -1) q.doc = -2;
        q.lim = masked_limit(p, q.pos, info[7]);
        if ((MOD & 2) && p.slopes != nullptr)
          q.slope = __ldg(p.slopes + (run - b * per_b) * p.run_heads + q.r / p.S_q) / unit;
      }
      return q;
    };

    int i = 0;
    Note e = note_at(i);
    __syncwarp();
    Row q = row_of(i, e.run);
    while (ok && !__any_sync(0xffffffffu, e.run < 0)) {
      const int run = q.run, share = q.share, r = q.r, pos = q.pos, lim = q.lim, doc = q.doc;
      const float slope = q.slope;
      const bool valid_row = r < p.rows;
      const bool warp_rows = __any_sync(0xffffffffu, valid_row);
      float m_use = valid_row ? -INFINITY : 0.0f, l = 0.0f;      // (rows past the end ride along with zero scores)
      bool poison = false, started = false;       // started: every row of the warp has seen a key
      int n = 0, own = 0;                         // tiles of the unit, and of this stream

      // One tile's S: the next of this stream, if it owns the tile.
      auto take = [&] {
        const bool mine = SPLIT ? (n & 1) == t : note_class(e.x, t) != kNoteNone;
        ++n;
        ++g;
        if (!mine) return false;
        ok = __all_sync(0xffffffffu, mbar_wait(bar_s_full + t, ns & 1, abort_flag, tmo, 0x28 + t));
        ++ns;
        tc_fence_after();
        return ok;
      };
      // P to TMEM, O to the new maximum, the row sum; then the tile is the MMA thread's.
      auto give = [&](uint32_t (&pw)[64], float sum, float alpha, bool need) {
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
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
            tmem_st32(tO + cc * 32, o);
          }
          tmem_st_wait();
        }
        l = fmaf(l, alpha, sum);
      };
      auto publish = [&] {
        ++own;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_p_full + t);
      };
      // The next note of this unit, false after its last.
      auto advance = [&] {
        __syncwarp();
        if (lane == 0) note_read(i);
        ++i;
        if (e.x & kNoteLast) return false;
        e = note_at(i);
        ok = __all_sync(0xffffffffu, e.run >= 0);
        return ok;
      };
      // Distance bias of a tile to one side of the row: slope times the distance is linear in the column; a multiply-add
      // with `tilt` for each, and the rest is one number for the row, returned.
      auto tilt_scores = [&](uint32_t (&s)[128], int d) {
        const float tilt = d > 0 ? slope : -slope;
#pragma unroll
        for (int c = 0; c < 128; ++c) s[c] = __float_as_uint(fmaf(tilt, static_cast<float>(c), __uint_as_float(s[c])));
        return -tilt * static_cast<float>(d);
      };
      auto exact = [&](uint32_t (&s)[128], float off, uint32_t (&pw)[64], float& sum, float& alpha, bool& need) {
        const float m_new = fmaxf(m_use, row_max128(s) + off);
        need = (m_new - m_use) * cl > C::kRescaleLog2;           // true on a row's first visible tile
        if (need) {
          alpha = ex2_approx((m_use - m_new) * cl);              // 0 when m_use = -inf
          m_use = m_new;
        }
        started = __all_sync(0xffffffffu, m_use != -INFINITY);
        // (a row that has seen no key yet keeps m_use = -inf: exponents of -inf, p = 0)
        exp_pass<false, 0>(s, cl, m_use == -INFINITY ? 0.0f : (m_use - off) * cl, pw, sum);
      };

      bool more = !(e.x & kNoteEmpty);
      if (!more) {
        __syncwarp();
        if (lane == 0) note_read(i);
        ++i;
      }
      // ---- tiles that some row of the unit sees in part, or that lie on both sides of a row
      while (more && !__any_sync(0xffffffffu, e.x & kNoteWhole)) {
        if (take()) {
          if (warp_rows) {
            const int cls = note_class(e.x, t), j = e.x & kNoteTile, st = (g - 1) % NS;
            uint32_t see[4];                     // the row's keys of this tile
            {
              const int valid = cls & kNoteRange ? lim - j * kMaskedTile : kMaskedTile;
#pragma unroll
              for (int k = 0; k < 4; ++k)
                see[k] = valid >= 32 * k + 32 ? 0xFFFFFFFFu : (valid <= 32 * k ? 0u : (1u << (valid - 32 * k)) - 1u);
            }
            if (e.masked) {
              ok = __all_sync(0xffffffffu, mbar_wait(bar_v_clean + st, ((g - 1) / NS) & 1, abort_flag, tmo, 0x2A));
              if (!ok) break;
              if (cls & kNoteDocs) {
                int id[4];
                uint32_t same[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                for (int k = 0; k < 4; ++k) id[k] = ids[st * 128 + 32 * k + lane];
                for (uint32_t todo = __ballot_sync(0xffffffffu, doc >= 0); todo != 0u;) {
                  const int one = __shfl_sync(0xffffffffu, doc, __ffs(todo) - 1);
#pragma unroll
                  for (int k = 0; k < 4; ++k) {
                    const uint32_t w = __ballot_sync(0xffffffffu, id[k] == one);
                    if (doc == one) same[k] = w;
                  }
                  todo &= ~__ballot_sync(0xffffffffu, doc == one);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) see[k] &= same[k];
              }
#pragma unroll
              for (int k = 0; k < 4; ++k) poison |= (see[k] & bad[st * 4 + k]) != 0u;
            }
            uint32_t s[128], pw[64];
            float sum = 0.0f, alpha = 1.0f;
            bool need = false;
            load_s(s);
            if (MOD & 2) {
              const float df = static_cast<float>(pos - j * kMaskedTile);
#pragma unroll
              for (int c = 0; c < 128; ++c)
                s[c] = __float_as_uint(fmaf(-slope, fabsf(df - static_cast<float>(c)), __uint_as_float(s[c])));
            }
#pragma unroll
            for (int c0 = 0; c0 < 128; c0 += 16) {
              const uint32_t w = (see[c0 >> 5] >> (c0 & 16)) & 0xFFFFu;
              if (!__all_sync(0xffffffffu, w == 0xFFFFu)) {
#pragma unroll
                for (int c = 0; c < 16; ++c)
                  if (!((w >> c) & 1u)) s[c0 + c] = 0xFF800000u;
              }
            }
            exact(s, 0.0f, pw, sum, alpha, need);
            give(pw, sum, alpha, need);
          }
          publish();
        }
        if (!ok) break;
        more = advance();
      }
      // ---- whole tiles
      while (more && ok) {
        int j = e.x & kNoteTile;
        const int step = e.n < 0 ? -1 : 1;
        for (int left = e.n * step; left > 0; --left, j += step) {
          if (!take()) {
            if (!ok) break;
            continue;
          }
          if (warp_rows) {
            uint32_t s[128], pw[64];
            float sum = 0.0f, alpha = 1.0f, off = 0.0f;
            bool need = false;
            auto scores = [&] {
              load_s(s);
              if (MOD & 2) off = tilt_scores(s, pos - j * kMaskedTile);
            };
            // speculative pass, as in the dense form: the running maximum, kept when the row sums stay bounded
            bool slow = !started;
            if constexpr (MOD == 1) {
              slow |= !(p.cap_limit > 0.0f);
              if (!slow) {
                tmem_ld128_sync(tS, s);
                const float t = cap_exp_pass(s, p, cl, m_use * cl, pw, sum);
                slow = __any_sync(0xffffffffu, !(sum <= C::kSumBound && cap_fits(t)));
              }
              if (slow) scores();
            } else {
              scores();
              if (!slow) {
                exp_pass<false, 0>(s, cl, (m_use - off) * cl, pw, sum);
                slow = __any_sync(0xffffffffu, !(sum <= C::kSumBound));
                if (slow) scores();
              }
            }
            if (slow) exact(s, off, pw, sum, alpha, need);
            give(pw, sum, alpha, need);
          }
          publish();
        }
        if (!ok) break;
        more = advance();
      }
      if (!ok) break;

      // the next unit's note and row, while the last P.V runs
      e = note_at(i);
      __syncwarp();
      q = row_of(i, e.run);

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
      const size_t row_idx = static_cast<size_t>(run) * p.rows + r;
      if constexpr (SPLIT) {
        const size_t n_rows = static_cast<size_t>(p.runs) * p.rows;
        const size_t at = static_cast<size_t>(2 * share + t) * n_rows + row_idx;
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
  grid_dep_wait();
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
      // eight partials' loads in flight; what an empty share's holds is discarded by a select
      for (int k0 = 0; k0 < min(32, n - c0); k0 += 8) {
        float v[8][D / 32];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int c = min(c0 + k0 + k, n - 1);
          const float* o = p.part_o + (c * n_rows + row) * D + lane * (D / 32);
#pragma unroll
          for (int e = 0; e < D / 32; ++e) v[k][e] = o[e];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float wk = __shfl_sync(0xffffffffu, wl, k0 + k);
          L += wk;
#pragma unroll
          for (int e = 0; e < D / 32; ++e) acc[e] = wk != 0.0f ? fmaf(wk, v[k][e], acc[e]) : acc[e];
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
