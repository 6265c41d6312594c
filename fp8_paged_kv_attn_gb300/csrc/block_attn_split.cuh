// The mma.sync split kernel of kvq_block_attn (block_attn.cu says what it computes and why), and of
// kvq_block_prefix_attn for requests' own tokens.  Included after decode_attn_mma.cuh and
// tc_device.cuh.
#pragma once

#include <algorithm>
#include <climits>

#include "block_prefix.cuh"

namespace kvq {

constexpr int kBaWarps = 8;                      // consumer warps
constexpr int kBaThreads = 32 * (kBaWarps + 1);
constexpr int kBaMaxStages = 48;
constexpr int kBaSegs = 4;                       // segment descriptors in flight
constexpr int kBaSmem = 225 * 1024;              // ring + merge slots + control, per CTA

// Row tiles: 4 (one MMA column block carries the weights and their remainders),
// 8 or 16 rows a warp; larger row counts take RT tiles of 16: two, and beyond 128 rows
// all eight warps.  (Blocks of 32 rows fit requests of different rows better: 24 drafts of
// 4 - 16 rows x 6 heads, head_dim 64, 18.7 us against 23.9 with 64 and 20.2 with 128, 32 of
// 1 - 16 rows x 4 heads over long contexts 231 against 268 and 521; 64 rows x 4 heads 63.9
// against 59.2 and 59.0.)  The
// warps that the (head, row tile) pairs leave free are further teams.

struct BaShape {
  int rk, rt, hg, tw;   // rows a warp, row tiles, heads a stage, teams
  int rows;             // rows a row block holds: rk * rt
  int row_blocks;       // row blocks of a request of max_q rows
  int groups;           // head groups
  bool tc;              // the tcgen05 kernel: blocks of 32 rows of one head
  int pairs() const { return hg * rt; }
  int slots() const { return pairs() * (tw - 1); }
};

// The tcgen05 kernel reads a block of 32 rows in the time that the mma.sync kernel
// takes for 8, but starts and ends a row of work more slowly.  Measured (8 kv heads
// of 128, us, mma.sync and tcgen05): 32 requests of 1,024 - 16,384 tokens, 12 rows 115
// and 101, 16 rows 120 and 101, 32 rows 194 and 103; 128 requests of 64 - 1,024, 16 rows
// 49 and 62, 32 rows 82 and 63.  So it takes more than 16 rows always, and 9 - 16
// where requests can be long: the two meet near 1,600 tokens, taken as half of what
// the block table holds.
constexpr int64_t kTcLong = 4096;

inline BaShape ba_shape(int max_q, int G, int Hkv, int D, int64_t capacity) {
  BaShape s;
  const int64_t rows = static_cast<int64_t>(max_q) * G;
  s.tc = D == 128 && (rows > 16 || (rows > 8 && capacity >= kTcLong));
  if (s.tc) {
    s.rk = 16;
    s.rt = 2;
    s.rows = 32;
    s.row_blocks = static_cast<int>((rows + 31) / 32);
    s.hg = s.tw = 1;
    s.groups = Hkv;
    return s;
  }
  s.rk = rows <= 4 ? 4 : rows <= 8 ? 8 : 16;
  s.rt = rows <= 16 ? 1 : rows <= 128 ? 2 : kBaWarps;
  s.rows = s.rk * s.rt;
  s.row_blocks = static_cast<int>((rows + s.rows - 1) / s.rows);
  s.hg = 1;
  for (int h = 1; h <= kBaWarps / s.rt; ++h)
    if (Hkv % h == 0) s.hg = h;
  s.groups = Hkv / s.hg;
  s.tw = kBaWarps / s.pairs();
  return s;
}

// Units that a row of work counts beside its tiles: its start (q, the first
// block-table entries, the pipeline's fill) and end, in tiles' times.  Without
// them a CTA whose run holds many short rows ends long after the others.
constexpr int kRowCost = 4;

// One segment: a run of tiles of one row, of one CTA.
struct BaSeg {
  int b, grp, rb;      // request (-1: no more segments), head group, row block
  int row0, n, L;      // the request's first row, rows, length
  int t_begin, t_end;  // tokens
  int stages;
  int part;            // -1: the row is this segment alone; else the partial slot
  int parts;           // kOwn: how many parts there are then
};

// The row of work that starts in a CTA and goes on past its end, if any: the
// rows that combine has to merge (a CTA's end cuts one row at most).
struct BaCut {
  int parts;             // 0: none; its parts lie in this CTA and the next ones
  int grp, rb, row0, n;
  int pad[3];
};

struct BaCtl {
  BaSeg seg[kBaSegs];
  uint64_t full[kBaMaxStages], empty[kBaMaxStages];
  uint64_t segfull[kBaSegs], segempty[kBaSegs];
  uint64_t mfull[kBaWarps], mempty[kBaWarps];  // per (head, row tile): the teams' merge
  float2 sc[kBaMaxStages][kBaWarps];           // (K, V) scale of the stage's heads
  int bad[kBaMaxStages];
  RunScan<kBaThreads> scan;
  int fail;
};

struct BaArgs {
  const uint16_t *q;
  int64_t q_stride;
  Ragged rg;
  const int32_t *block_table;
  const uint8_t *abort_mask;
  const float2 *scales;  // [num_pages][Hkv]
  BaCut *cut;            // [CTAs]
  float *part;           // [2 CTAs][hg * rt][rk][D + kStat]
  float *kept;           // the tcgen05 kernel's flushed sums: [CTAs][kTcWarps][kTcKept]
  float *out;
  uint32_t *err_word;
  int32_t num_pages, p_shift, Hkv, Hq, G, MP, max_q;  // page size 1 << p_shift
  int32_t hg, rt, tw, rounds, groups, stages;  // rounds: of the teams' merge
  float q_scale;  // sm_scale * log2(e)
  // kOwn (kvq_block_prefix_attn): the requests and where their own tokens begin, as its plan lists
  // them, and where every row's sums go
  const PxPlan *plan;
  const PxItem *items;
  float *rows;
};

// Request b's rows, with what attention refuses; `live`: it has work.
__device__ __forceinline__ Rows ba_rows(const BaArgs &a, int b, bool &live) {
  Rows r = request_rows<true>(a.rg, b);
  if (!r.err && r.n > a.max_q) r.err = KVQ_ERRBIT_SEQLEN;
  live = r.n > 0 && !r.err && !(a.abort_mask && __ldg(a.abort_mask + b) != 0);
  return r;
}

// 16-token tiles of one row of work, and row blocks, of a live request.
__device__ __forceinline__ int ba_tiles_of(const Rows &r, int first) {
  return (r.p0 + r.n - first + kTile - 1) / kTile;
}
__device__ __forceinline__ int ba_blocks(const BaArgs &a, const Rows &r, int rows) {
  return (r.n * a.G + rows - 1) / rows;
}

// What the schedule walks over: the batch's requests, all of whose tokens are attended to, or (kOwn) the
// plan's, from the token on at which their own ones begin.
struct BaWork {
  Rows r;
  bool live;
  int b, first;  // block table, first token
};

template <bool kOwn>
__device__ __forceinline__ BaWork ba_work(const BaArgs &a, int n_grp, int i) {
  BaWork w;
  if constexpr (kOwn) {
    const PxItem it = px_load_item(a.items + n_grp + i);
    w.r = {it.row0, it.n, it.p0, 0};
    w.live = it.live;
    w.b = it.b;
    w.first = it.first;
  } else {
    w.r = ba_rows(a, i, w.live);
    w.b = i;
    w.first = 0;
  }
  return w;
}

__device__ __forceinline__ bool ba_wait(BaCtl &ctl, uint64_t *bar, uint32_t parity,
                                        uint32_t *err_word) {
  volatile int *fail = &ctl.fail;
  if (*fail) return false;
  if (mbar_wait(bar, parity)) return true;
  if (atomicExch(&ctl.fail, 1) == 0) report(err_word, KVQ_ERRBIT_TIMEOUT);
  return false;
}

// The same for a whole warp, which leaves or stays together.
__device__ __forceinline__ bool ba_wait_warp(BaCtl &ctl, uint64_t *bar, uint32_t parity,
                                             uint32_t *err_word) {
  return __all_sync(0xffffffffu, ba_wait(ctl, bar, parity, err_word));
}

// Byte offset of 16-byte chunk c of row r in a head's swizzled 16-row block.
template <int D>
__device__ __forceinline__ int swz(int r, int c) {
  return D == 128 ? r * 128 + ((c ^ (r & 7)) * 16) : r * 64 + ((c ^ ((r >> 1) & 3)) * 16);
}

// A consumer warp's state: RK rows of one kv head.
template <int D, int RK>
struct BaState {
  static constexpr int KS = D / 16;            // k-steps of q.k, 16-dim tiles of p.v
  static constexpr int NG = RK == 16 ? 2 : 1;  // 8-row groups
  uint32_t qa[NG][2][KS];                      // A fragments: rows gq (+8), words 0 and 2
  float o[KS][NG][4];
  float m[NG], l[NG], n[NG], qk[NG];
  int lim[NG];                                 // tokens that the lane's row sees; -1: a bad page among them
};

// The row of lane group gq in 8-row group g (copies of rows 0..3 in 4..7 for RK 4).
template <int RK>
__device__ __forceinline__ int lane_row(int gq, int g) {
  return RK == 4 ? (gq & 3) : gq + 8 * g;
}

// The lane's D / 4 dims of row r (of the request), scaled by 2^e so that the
// row's largest value lies in [2^14, 2^15), as f16 pairs; the scale that undoes it.
template <int D, int RK>
__device__ __forceinline__ float ba_q_row(const BaArgs &a, const BaSeg &sg, int kvh, int r, int tq,
                                          uint32_t (&lo)[D / 16], uint32_t (&hi)[D / 16]) {
  constexpr int W = D / 4;
  const int i = r / a.G;
  float x[W];
  if (i < sg.n) {
    const uint16_t *p = a.q + (static_cast<int64_t>(sg.row0) + i) * a.q_stride +
                        static_cast<int64_t>(kvh * a.G + r - i * a.G) * D + W * tq;
#pragma unroll
    for (int c = 0; c < W / 8; ++c) unpack8(__ldg(reinterpret_cast<const uint4 *>(p) + c), x + 8 * c);
  } else {
#pragma unroll
    for (int c = 0; c < W; ++c) x[c] = 0.f;
  }
  float mx = 0.f;
#pragma unroll
  for (int c = 0; c < W; ++c) mx = fmaxf(mx, fabsf(x[c]));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
  int e = mx > 0.f && mx < INFINITY ? 14 - ilogbf(mx) : 0;
  e = min(e, 126);
  const float up = pow2(e);  // e >= 14 - 127
#pragma unroll
  for (int s = 0; s < D / 16; ++s) {
    lo[s] = f32x2_to_f16x2(x[4 * s] * up, x[4 * s + 1] * up);
    hi[s] = f32x2_to_f16x2(x[4 * s + 2] * up, x[4 * s + 3] * up);
  }
  return a.q_scale * pow2(-e);
}

// A segment's start: q, limits and empty sums.
template <int D, int RK>
__device__ __forceinline__ void ba_begin(BaState<D, RK> &st, const BaArgs &a, const BaSeg &sg,
                                         int kvh, int row_base, int gq, int tq) {
  constexpr int KS = BaState<D, RK>::KS, NG = BaState<D, RK>::NG;
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const int r = row_base + lane_row<RK>(gq, g);
    const int i = r / a.G;
    st.lim[g] = i < sg.n ? sg.L - sg.n + 1 + i : sg.L;
    st.qk[g] = ba_q_row<D, RK>(a, sg, kvh, r, tq, st.qa[g][0], st.qa[g][1]);
    st.m[g] = st.n[g] = -INFINITY;
    st.l[g] = 0.f;
#pragma unroll
    for (int k = 0; k < KS; ++k) st.o[k][g][0] = st.o[k][g][1] = st.o[k][g][2] = st.o[k][g][3] = 0.f;
  }
}

// The product alone, with no sum before it.
__device__ __forceinline__ void mma_16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                                uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// p.v of one tile: words wa..wd are V rows 2t, 2t+1, 2t+8, 2t+9 at the lane's
// D / 8 dims; hi / lo the weights' f16 and remainders per row group and n-tile.
// The tensor core's additions truncate (towards zero), so that a long sum kept there
// drifts: 7e-6 of it over 8,192 tokens of positive values and 1.2e-4 over 65,536,
// measured.  So it sums a tile, and the tiles are added with rounding (5e-7 left; 1% of
// the time at one row, 3% at eight rows of a kv head.  Flushing the sums every 16 or 32
// turns, to shared or global memory, cost 3 - 5%).
template <int D, int RK>
__device__ __forceinline__ void ba_pv(float (&o)[D / 16][BaState<D, RK>::NG][4],
                                      const uint32_t (&wa)[D / 32], const uint32_t (&wb)[D / 32],
                                      const uint32_t (&wc)[D / 32], const uint32_t (&wd)[D / 32],
                                      const uint32_t (&hi)[BaState<D, RK>::NG][2],
                                      const uint32_t (&lo)[BaState<D, RK>::NG][2]) {
  constexpr int KS = D / 16, NG = BaState<D, RK>::NG;
  // the two MMAs on one accumulator lie four MMAs apart (their latency)
  constexpr int BI = 4 / NG;
#pragma unroll
  for (int i0 = 0; i0 < KS; i0 += BI) {
    uint32_t f[BI][4];
#pragma unroll
    for (int j = 0; j < BI; ++j) {
      const int i = i0 + j;
      const uint32_t sel = (i & 1) ? 0x7362u : 0x5140u;  // bytes (a.b, b.b, a.b+1, b.b+1)
      const uint32_t x = prmt(wa[i >> 1], wb[i >> 1], sel);
      const uint32_t y = prmt(wc[i >> 1], wd[i >> 1], sel);
      f[j][0] = e4m3x2_to_f16x2(x & 0xFFFFu);
      f[j][1] = e4m3x2_to_f16x2(x >> 16);
      f[j][2] = e4m3x2_to_f16x2(y & 0xFFFFu);
      f[j][3] = e4m3x2_to_f16x2(y >> 16);
    }
    float d[BI][NG][4];
#pragma unroll
    for (int j = 0; j < BI; ++j)
#pragma unroll
      for (int g = 0; g < NG; ++g)
        mma_16816_first(d[j][g], f[j][0], f[j][1], f[j][2], f[j][3], RK > 4 ? lo[g][0] : hi[g][0],
                        RK > 4 ? lo[g][1] : hi[g][1]);
    if constexpr (RK > 4) {
#pragma unroll
      for (int j = 0; j < BI; ++j)
#pragma unroll
        for (int g = 0; g < NG; ++g)
          mma_16816(d[j][g], f[j][0], f[j][1], f[j][2], f[j][3], hi[g][0], hi[g][1]);
    }
#pragma unroll
    for (int j = 0; j < BI; ++j)
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
          const float2 x = __fadd2_rn(make_float2(o[i0 + j][g][k], o[i0 + j][g][k + 1]),
                                      make_float2(d[j][g][k], d[j][g][k + 1]));
          o[i0 + j][g][k] = x.x;
          o[i0 + j][g][k + 1] = x.y;
        }
  }
}

// NaN codes anywhere in a word of four
__device__ __forceinline__ bool has_nan(uint32_t w) {
  return __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu) != 0;
}

// A tile where some row does not see every token, and V holds a NaN code: a
// weight of 0 does not stop a NaN, so every row's sum must leave the tokens out
// that it does not see.  Once for each of the tile's visibility limits, V
// rows beyond it zeroed, into sums of their own that only the rows with that
// limit take.  Rare (a NaN has been cached), so out of line.
template <int D, int RK>
struct BaMasked {
  static constexpr int KS = D / 16, NG = BaState<D, RK>::NG, W = D / 32;
  float o[KS][NG][4];
  uint32_t v[4][W], hi[NG][2], lo[NG][2];
  int lim[NG], tok0, tq;
};

template <int D, int RK>
__device__ __noinline__ void ba_pv_masked(BaMasked<D, RK> &x) {
  constexpr int KS = D / 16, NG = BaState<D, RK>::NG, W = D / 32;
  for (int seen = 1; seen <= kTile; ++seen) {
    uint32_t w[4][W];
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int c = 0; c < W; ++c)
        w[k][c] = 2 * x.tq + (k & 1) + 8 * (k >> 1) < seen ? x.v[k][c] : 0u;
    float tmp[KS][NG][4];
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int g = 0; g < NG; ++g) tmp[i][g][0] = tmp[i][g][1] = tmp[i][g][2] = tmp[i][g][3] = 0.f;
    ba_pv<D, RK>(tmp, w[0], w[1], w[2], w[3], x.hi, x.lo);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const int mine = min(x.lim[g] - x.tok0, kTile);  // the lane's row; its columns are rows 2t, 2t+1
      const int sa = __shfl_sync(0xffffffffu, mine, 8 * x.tq);
      const int sb = __shfl_sync(0xffffffffu, mine, 8 * x.tq + 4);
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        if (sa == seen) {
          x.o[i][g][0] += tmp[i][g][0];
          x.o[i][g][2] += tmp[i][g][2];
        }
        if (sb == seen) {
          x.o[i][g][1] += tmp[i][g][1];
          x.o[i][g][3] += tmp[i][g][3];
        }
      }
    }
  }
}

// V^T operand words of a tile: rows 2t, 2t+1, 2t+8, 2t+9 at dims (D / 8) gq ..
template <int D>
__device__ __forceinline__ void ba_load_v(uint32_t (&v)[4][D / 32], const uint8_t *vs, int gq, int tq) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int r = 2 * tq + (k & 1) + 8 * (k >> 1);
    if constexpr (D == 128) {
      const uint4 x = lds128(vs + swz<D>(r, gq));
      v[k][0] = x.x;
      v[k][1] = x.y;
      v[k][2] = x.z;
      v[k][3] = x.w;
    } else {
      const uint2 x = *reinterpret_cast<const uint2 *>(vs + swz<D>(r, gq >> 1) + 8 * (gq & 1));
      v[k][0] = x.x;
      v[k][1] = x.y;
    }
  }
}

// NT consecutive 16-token tiles of a segment: ks / vs the head's swizzled
// blocks, sc the blocks' scales, tok0 the first token, min_lim the fewest tokens that a
// row of the row block sees, L the length.  Two tiles share one softmax update:
// a warp is bound by the latency of its dependency chain (max, vote, exponential,
// conversion), which the second tile's work fills.
template <int D, int RK, int NT>
__device__ __forceinline__ void ba_tiles(BaState<D, RK> &st, const uint8_t *const (&ks)[NT],
                                         const uint8_t *const (&vs)[NT], const float2 (&sc)[NT],
                                         int tok0, int min_lim, int L, int gq, int tq) {
  constexpr int KS = BaState<D, RK>::KS, NG = BaState<D, RK>::NG, W = D / 32;
  // Sums a score tile: two independent chains of MMAs, which also truncate half as often
  // (error of the output 1.6 -> 1.3 times an fp32 evaluation's at worst of 8 inputs, for
  // the same time; 16 rows a warp have no registers for them).
  constexpr int CH = NT == 1 || RK < 16 ? 2 : 1;
  float s[NT][2][CH][4];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int c = 0; c < CH; ++c) s[t][j][c][0] = s[t][j][c][1] = s[t][j][c][2] = s[t][j][c][3] = 0.f;
  {
    uint32_t kw[NT][2][KS];  // rows gq and 8 + gq, the lane's D / 4 dims
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          const uint4 x = lds128(ks[t] + swz<D>(gq + 8 * j, (D / 64) * tq + c));
          kw[t][j][4 * c] = x.x;
          kw[t][j][4 * c + 1] = x.y;
          kw[t][j][4 * c + 2] = x.z;
          kw[t][j][4 * c + 3] = x.w;
        }
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          mma_16816(s[t][j][k % CH], st.qa[0][0][k], NG == 2 ? st.qa[NG - 1][0][k] : 0u,
                    st.qa[0][1][k], NG == 2 ? st.qa[NG - 1][1][k] : 0u,
                    e4m3x2_to_f16x2(kw[t][j][k] & 0xFFFFu), e4m3x2_to_f16x2(kw[t][j][k] >> 16));
  }
  const bool partial = tok0 + NT * kTile > min_lim;  // uniform over the warp
  float lv[NT], vm[NT];  // the V scales' exponents and fractions
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const float2 v = split_scale(sc[t].y);
    vm[t] = v.x;
    lv[t] = v.y;
  }
  float x[NG][NT][2][2], mx[NG], mv[NG];
  bool any = false;
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const int seen = st.lim[g] - tok0;
    mx[g] = mv[g] = -INFINITY;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float f = st.qk[g] * sc[t].x;
      float mt = -INFINITY;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float y = s[t][j][0][2 * g + e];
          if constexpr (CH == 2) y += s[t][j][CH - 1][2 * g + e];
          y *= f;
          if (partial && kTile * t + 8 * j + 2 * tq + e >= seen) y = -INFINITY;
          x[g][t][j][e] = y;
          mt = fmaxf(mt, y);
        }
      mx[g] = fmaxf(mx[g], mt);
      mv[g] = fmaxf(mv[g], mt + lv[t]);
    }
    mx[g] = fmaxf(mx[g], __shfl_xor_sync(0xffffffffu, mx[g], 1));
    mx[g] = fmaxf(mx[g], __shfl_xor_sync(0xffffffffu, mx[g], 2));
    if constexpr (NT == 1) {
      mv[g] = mx[g] + lv[0];
    } else {
      mv[g] = fmaxf(mv[g], __shfl_xor_sync(0xffffffffu, mv[g], 1));
      mv[g] = fmaxf(mv[g], __shfl_xor_sync(0xffffffffu, mv[g], 2));
    }
    any |= mx[g] > st.m[g] + kRescaleThreshold || mv[g] > st.n[g] + kRescaleThreshold;
  }
  if (__any_sync(0xffffffffu, any)) {
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      if (mx[g] > st.m[g] + kRescaleThreshold) {
        st.l[g] *= exp2f(st.m[g] - mx[g]);  // 0 when m is -inf
        st.m[g] = mx[g];
      }
      float f = 1.f;
      if (mv[g] > st.n[g] + kRescaleThreshold) {
        f = exp2f(st.n[g] - mv[g]);
        st.n[g] = mv[g];
      }
      // columns 2t and 2t + 1 of O^T are the rows of lanes 8t and 8t + 4
      const float fa = __shfl_sync(0xffffffffu, f, 8 * tq);
      const float fb = __shfl_sync(0xffffffffu, f, 8 * tq + 4);
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        st.o[i][g][0] *= fa;
        st.o[i][g][1] *= fb;
        st.o[i][g][2] *= fa;
        st.o[i][g][3] *= fb;
      }
    }
  }
  uint32_t hi[NT][NG][2], lo[NT][NG][2];
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    // a row that has seen nothing yet (m, n = -inf) has only x = -inf here:
    // its weights come out 0 with any finite reference
    const bool none = st.n[g] == -INFINITY;
    const float m = none ? 0.f : st.m[g];
    const float mn = none ? 0.f : st.m[g] - st.n[g];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      // vs 2^(m - n), with kPScale (2^7) so that the largest weights sit high in
      // f16's range; the clamp only meets rows whose weights here are below
      // 2^-112 of their largest
      const float d = vm[t] * kPScale * fast_exp2(fminf(mn + lv[t], 112.f));
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float p0 = fast_exp2(x[g][t][j][0] - m), p1 = fast_exp2(x[g][t][j][1] - m);
        st.l[g] += p0 + p1;
        const float w0 = p0 * d, w1 = p1 * d;
        const uint32_t h = f32x2_to_f16x2(w0, w1);
        const float2 hf = f16x2_to_f32x2(h);
        const uint32_t r = f32x2_to_f16x2(w0 - hf.x, w1 - hf.y);
        hi[t][g][j] = RK == 4 && gq >= 4 ? r : h;
        lo[t][g][j] = r;
      }
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    uint32_t v[4][W];
    ba_load_v<D>(v, vs[t], gq, tq);
    if (partial) {
      bool bad = false;
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int c = 0; c < W; ++c) {
          // cached bytes past the sequence may be anything
          if (tok0 + kTile * t + 2 * tq + (k & 1) + 8 * (k >> 1) >= L) v[k][c] = 0u;
          bad |= has_nan(v[k][c]);
        }
      if (__any_sync(0xffffffffu, bad)) {
        BaMasked<D, RK> x2;  // copies: the state's own registers keep no address
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
          for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int k = 0; k < 4; ++k) x2.o[i][g][k] = st.o[i][g][k];
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int c = 0; c < W; ++c) x2.v[k][c] = v[k][c];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            x2.hi[g][j] = hi[t][g][j];
            x2.lo[g][j] = lo[t][g][j];
          }
          x2.lim[g] = st.lim[g];
        }
        x2.tok0 = tok0 + kTile * t;
        x2.tq = tq;
        ba_pv_masked<D, RK>(x2);
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
          for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int k = 0; k < 4; ++k) st.o[i][g][k] = x2.o[i][g][k];
        continue;
      }
    }
    ba_pv<D, RK>(st.o, v[0], v[1], v[2], v[3], hi[t], lo[t]);
  }
}

// ---------------------------------------------------------------------------
// the split kernel
// ---------------------------------------------------------------------------

// A merge slot holds a warp's sums register by register: [KS * NG * 4 + 3 NG]
// words of 32 lanes.
template <int D, int RK>
constexpr int kBaSlotWords = (D / 16 * BaState<D, RK>::NG * 4 + 3 * BaState<D, RK>::NG) * 32;

inline size_t ba_slot_bytes(const BaShape &s, int D) {
  return (D / 16 * 4 + 3) * (s.rk == 16 ? 2 : 1) * 128;
}

// Shared memory: K ring, V ring, merge slots, control.  Teams take turns of two
// stages; the stage count is a multiple of a round of turns, so that within a
// segment every ring slot belongs to one team and its phases are waited for
// in order (a team that ran ahead of another on a shared slot could take the
// parity of the phase before last for its own).
inline int ba_stages(const BaShape &s, int D) {
  const size_t stage = 2 * static_cast<size_t>(s.hg) * kTile * D;
  const size_t room = kBaSmem - 1024 - sizeof(BaCtl) - s.slots() * ba_slot_bytes(s, D);
  const size_t fit = room / stage < kBaMaxStages ? room / stage : kBaMaxStages;
  const int n = static_cast<int>(fit);
  return s.tw > 1 ? n / (2 * s.tw) * (2 * s.tw) : n;
}

// Row r (of the request) as an output row's address.
template <int D>
__device__ __forceinline__ float *ba_out_row(const BaArgs &a, const BaSeg &sg, int kvh, int r) {
  const int i = r / a.G;
  return a.out + ((static_cast<int64_t>(sg.row0) + i) * a.Hq + kvh * a.G + r - i * a.G) * D;
}

// kOwn: for kvq_block_prefix_attn, requests' own tokens behind a prefix.  Rows of work are not
// normalised: their sums and statistics go to a.rows, or to a part's slot that a.rows names.
template <int D, int RK, bool kOwn = false>
__global__ void __launch_bounds__(kBaThreads, 1)
    block_split_kernel(const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap, BaArgs a) {
  using St = BaState<D, RK>;
  constexpr int KS = St::KS, NG = St::NG, RF = D + kStat;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);  // for the swizzle
  const uint32_t stage_bytes = static_cast<uint32_t>(a.hg) * kTile * D;
  const int NS = a.stages;
  const int ngrp = a.hg * a.rt;  // (head, row tile) pairs
  uint8_t *kbuf = smem;
  uint8_t *vbuf = smem + static_cast<size_t>(NS) * stage_bytes;
  float *slots = reinterpret_cast<float *>(smem + 2 * static_cast<size_t>(NS) * stage_bytes);
  BaCtl &ctl = *reinterpret_cast<BaCtl *>(slots + (a.tw - 1) * ngrp * kBaSlotWords<D, RK>);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = RK * a.rt;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&ctl.full[i], 1 + a.hg);
      mbar_init(&ctl.empty[i], ngrp);
    }
    for (int i = 0; i < kBaSegs; ++i) {
      mbar_init(&ctl.segfull[i], 1);
      mbar_init(&ctl.segempty[i], ngrp * a.tw);
    }
    for (int i = 0; i < ngrp; ++i) {
      mbar_init(&ctl.mfull[i], a.tw);
      mbar_init(&ctl.mempty[i], a.tw);
    }
    ctl.fail = 0;
    fence_barrier_init();
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&kmap)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&vmap)) : "memory");
  }
  __syncthreads();
  // (kOwn: the kernel ahead began, and let this one start, when the plan and all before it were
  // complete; it is waited for at the end, so that whoever waits for this one waits for both)
  if (!kOwn) grid_dependency_wait();
  const int n_grp = kOwn ? __ldcg(&a.plan->n_grp) : 0, n_req = kOwn ? __ldcg(&a.plan->n_req) : a.rg.B;
  const RunStart run = find_run<kBaThreads>(
      n_req, gridDim.x, blockIdx.x, ctl.scan, [&](int b) -> int64_t {
        const BaWork w = ba_work<kOwn>(a, n_grp, b);
        if (!kOwn && w.r.err && blockIdx.x == 0) report(a.err_word, w.r.err);
        return w.live ? static_cast<int64_t>(ba_tiles_of(w.r, w.first) + kRowCost) * a.groups * ba_blocks(a, w.r, rows)
                      : 0;
      });
  allow_dependents();
  const int64_t u0 = blockIdx.x * run.per;
  const int64_t u1 = min(u0 + run.per, run.total);

  if (warp == kBaWarps) {
    // ------------------------------------------------------------ producer
    const uint64_t pol = policy_evict_first();
    int64_t u = u0, in = run.in;
    int b = run.b;
    BaCut cut = {0, 0, 0, 0, 0, {0, 0, 0}};
    // stages and segments issued; the next stage's ring slot and the parity of
    // its empty barrier's phase (kept by steps: a division by the ring's
    // length each stage cost the warp more than the copies)
    uint32_t g = 0, nseg = 0;
    int slot = 0;
    uint32_t par = 1;
    bool ok = true;
    int win_b = -1, win = 0, cur = -1, nxt = -1;  // block-table window (two of 32 entries)
    const int32_t *bt = a.block_table;
    auto bt_load = [&](int lp) -> int { return lp < a.MP ? __ldg(bt + lp) : -1; };
    while (ok && u < u1) {
      const BaWork wk = ba_work<kOwn>(a, n_grp, b);
      const bool live = wk.live;
      const Rows rq = wk.r;
      const int tiles = live ? ba_tiles_of(rq, wk.first) : 0, units = tiles + kRowCost;
      const int64_t have = live ? static_cast<int64_t>(units) * a.groups * ba_blocks(a, rq, rows) : 0;
      if (in >= have) {
        ++b;
        in = 0;
        continue;
      }
      const int64_t rw = in / units;  // row of work: row block major
      const int s = static_cast<int>(in - rw * units);
      const int rb = static_cast<int>(rw / a.groups), grp = static_cast<int>(rw - static_cast<int64_t>(rb) * a.groups);
      const int span = static_cast<int>(min(static_cast<int64_t>(units - s), u1 - u));
      // units [0, kRowCost) of a row stand for its start; tile t is unit kRowCost + t
      const int t0 = max(0, s - kRowCost), take = s + span - kRowCost - t0;
      const int64_t ut = u - s + kRowCost;  // the row's first tile
      u += span;
      in += span;
      if (take <= 0) continue;
      const int L = rq.p0 + rq.n;
      const int t_begin = wk.first + t0 * kTile, t_end = min(wk.first + (t0 + take) * kTile, L);
      const int64_t c_lo = ut / run.per;
      const int nparts = static_cast<int>((ut + tiles - 1) / run.per - c_lo) + 1;
      const int ss = nseg % kBaSegs;
      bool w = true;
      if (lane == 0 && nseg >= kBaSegs)
        w = ba_wait(ctl, &ctl.segempty[ss], ((nseg / kBaSegs) - 1) & 1, a.err_word);
      ok = __shfl_sync(0xffffffffu, w ? 1 : 0, 0) != 0;
      if (!ok) break;
      if (lane == 0) {
        if (t0 == 0 && nparts > 1) cut = {nparts, grp, rb, rq.row, rq.n, {0, 0, 0}};
        ctl.seg[ss] = {b, grp, rb, rq.row, rq.n, L, t_begin, t_end, take,
                       nparts == 1 ? -1 : 2 * static_cast<int>(blockIdx.x) + (t0 == 0 ? 1 : 0), nparts};
        mbar_arrive(&ctl.segfull[ss]);
      }
      ++nseg;
      const int lp0 = t_begin >> a.p_shift;
      if (b != win_b || lp0 < win || lp0 >= win + 32) {
        win_b = b;
        win = lp0;
        bt = a.block_table + static_cast<int64_t>(wk.b) * a.MP;
        cur = bt_load(win + lane);
        nxt = bt_load(win + 32 + lane);
      }
      for (int st = 0, tok = t_begin; st < take; ++st, tok += kTile) {
        // on a ring's first round the wait returns at once: the phase before a
        // barrier's first counts as completed
        ok = ba_wait_warp(ctl, &ctl.empty[slot], par, a.err_word);
        if (!ok) break;
        const int lp = tok >> a.p_shift;
        if (lp >= win + 32) {  // at most one window a stage
          win += 32;
          cur = nxt;
          nxt = bt_load(win + 32 + lane);
        }
        const int page = __shfl_sync(0xffffffffu, cur, lp - win);
        const bool bad = page < 0 || page >= a.num_pages;
        if (lane == 0) {
          ctl.bad[slot] = bad;
          mbar_arrive_expect_tx(&ctl.full[slot], bad ? 0u : 2u * stage_bytes);
          if (!bad) {
            const int y = tok & ((1 << a.p_shift) - 1);
            tma_load_4d(kbuf + slot * stage_bytes, &kmap, 0, y, grp * a.hg, page, &ctl.full[slot],
                        pol);
            tma_load_4d(vbuf + slot * stage_bytes, &vmap, 0, y, grp * a.hg, page, &ctl.full[slot],
                        pol);
          } else {
            report(a.err_word, KVQ_ERRBIT_PAGE);
          }
        }
        if (lane < a.hg) {
          if (!bad) {
            cp_async8(&ctl.sc[slot][lane],
                      a.scales + static_cast<int64_t>(page) * a.Hkv + grp * a.hg + lane);
            cp_async_arrive(&ctl.full[slot]);
          } else {  // tokens that rows without a result see, and others have masked
            ctl.sc[slot][lane] = make_float2(1.f, 1.f);
            mbar_arrive(&ctl.full[slot]);
          }
        }
        ++g;
        if (++slot == NS) {
          slot = 0;
          par ^= 1;
        }
        __syncwarp();
      }
    }
    if (!kOwn && lane == 0) a.cut[blockIdx.x] = cut;
    if (ok) {  // nothing more
      const int ss = nseg % kBaSegs;
      if (lane == 0 && (nseg < kBaSegs ||
                        ba_wait(ctl, &ctl.segempty[ss], ((nseg / kBaSegs) - 1) & 1, a.err_word))) {
        ctl.seg[ss].b = -1;
        mbar_arrive(&ctl.segfull[ss]);
      }
    }
    if (*reinterpret_cast<volatile int *>(&ctl.fail)) {
      // a wait gave up: let the copies in flight land before the CTA's shared
      // memory goes to another one
      if (lane == 0)
        for (uint32_t k = g > NS ? g - NS : 0; k < g; ++k)
          mbar_wait(&ctl.full[k % NS], (k / NS) & 1);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (kOwn) grid_dependency_wait();
    return;
  }

  // -------------------------------------------------------------- consumers
  // rows of requests without work (aborted, bad lengths) are zeros
  for (int b = blockIdx.x; !kOwn && b < a.rg.B; b += gridDim.x) {
    bool live;
    const Rows r = ba_rows(a, b, live);
    if (live || r.n == 0) continue;
    float4 *o = reinterpret_cast<float4 *>(a.out + static_cast<int64_t>(r.row) * a.Hq * D);
    const int64_t n4 = static_cast<int64_t>(r.n) * a.Hq * (D / 4);
    for (int64_t k = threadIdx.x; k < n4; k += 32 * kBaWarps) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const int pair = warp % ngrp, team = warp / ngrp;  // (head, row tile), team
  if (team >= a.tw) return;
  const int head = pair / a.rt, tile = pair % a.rt;
  const int gq = lane >> 2, tq = lane & 3;
  St st;
  uint32_t g0 = 0, nseg = 0, nmerge = 0;
  while (true) {
    const int ss = nseg % kBaSegs;
    if (!ba_wait_warp(ctl, &ctl.segfull[ss], (nseg / kBaSegs) & 1, a.err_word)) return;
    const BaSeg sg = ctl.seg[ss];
    if (sg.b < 0) return;
    const int kvh = sg.grp * a.hg + head;
    const int row_base = sg.rb * rows + tile * RK;  // this warp's first row of the request
    ba_begin<D, RK>(st, a, sg, kvh, row_base, gq, tq);
    const int min_lim = min(sg.L, sg.L - sg.n + 1 + (sg.rb * rows) / a.G);
    // the ring slot and phase parity of the team's first stage
    int s0 = static_cast<int>((g0 + 2 * team) % NS);
    uint32_t p0 = ((g0 + 2 * team) / NS) & 1;
    for (int k = 2 * team; k < sg.stages; k += 2 * a.tw) {  // a turn: two stages
      const bool two = k + 1 < sg.stages;
      const int s1 = s0 + 1 == NS ? 0 : s0 + 1;
      if (!ba_wait_warp(ctl, &ctl.full[s0], p0, a.err_word)) return;
      if (two && !ba_wait_warp(ctl, &ctl.full[s1], s1 == 0 ? p0 ^ 1 : p0, a.err_word)) return;
      const int tok = sg.t_begin + k * kTile;
      const uint32_t off0 = s0 * stage_bytes + head * (kTile * D), off1 = s1 * stage_bytes + head * (kTile * D);
      // a row that sees a bad page is zeros whatever the stage holds; rows that end before it
      // have it masked, as any token that they do not see
      if (ctl.bad[s0] || (two && ctl.bad[s1])) {
        const int from = ctl.bad[s0] ? tok : tok + kTile;
#pragma unroll
        for (int g = 0; g < NG; ++g)
          if (st.lim[g] > from) st.lim[g] = -1;
      }
      if (two) {
        const uint8_t *kp[2] = {kbuf + off0, kbuf + off1}, *vp[2] = {vbuf + off0, vbuf + off1};
        const float2 sc[2] = {ctl.sc[s0][head], ctl.sc[s1][head]};
        ba_tiles<D, RK, 2>(st, kp, vp, sc, tok, min_lim, sg.L, gq, tq);
      } else {
        const uint8_t *kp[1] = {kbuf + off0}, *vp[1] = {vbuf + off0};
        const float2 sc[1] = {ctl.sc[s0][head]};
        ba_tiles<D, RK, 1>(st, kp, vp, sc, tok, min_lim, sg.L, gq, tq);
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&ctl.empty[s0]);
        if (two) mbar_arrive(&ctl.empty[s1]);
      }
      s0 += 2 * a.tw;
      if (s0 >= NS) {  // 2 tw <= NS
        s0 -= NS;
        p0 ^= 1;
      }
    }
    g0 += sg.stages;
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl.segempty[ss]);
    ++nseg;

    // ---- the segment's end: the row's denominator, marked if the row sees a bad page
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      st.l[g] += __shfl_xor_sync(0xffffffffu, st.l[g], 1);
      st.l[g] += __shfl_xor_sync(0xffffffffu, st.l[g], 2);
      if (st.lim[g] < 0) st.l[g] = -1.f;
    }
    if (a.tw > 1) {
      // The teams' sums go to team 0, halving the teams each round.  Every round
      // has slots of its own, so one barrier a round orders its writes before
      // its reads, and one after the last keeps the next segment's writes off.
      if (nmerge > 0 && !ba_wait_warp(ctl, &ctl.mempty[pair], (nmerge - 1) & 1, a.err_word)) return;
      int alive = a.tw, slot0 = 0, round = 0;
      while (alive > 1) {
        const int half = (alive + 1) / 2;
        if (team >= half && team < alive) {
          float *w = slots + static_cast<int64_t>((slot0 + team - half) * ngrp + pair) * kBaSlotWords<D, RK> + lane;
#pragma unroll
          for (int g = 0; g < NG; ++g) {
#pragma unroll
            for (int i = 0; i < KS; ++i)
#pragma unroll
              for (int k = 0; k < 4; ++k) w[32 * ((g * KS + i) * 4 + k)] = st.o[i][g][k];
            w[32 * (KS * NG * 4 + 3 * g)] = st.m[g];
            w[32 * (KS * NG * 4 + 3 * g + 1)] = st.l[g];
            w[32 * (KS * NG * 4 + 3 * g + 2)] = st.n[g];
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.mfull[pair]);
        if (!ba_wait_warp(ctl, &ctl.mfull[pair], (nmerge * a.rounds + round) & 1, a.err_word)) return;
        if (team < alive - half) {
          const float *w = slots + static_cast<int64_t>((slot0 + team) * ngrp + pair) * kBaSlotWords<D, RK> + lane;
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            const float m2 = w[32 * (KS * NG * 4 + 3 * g)], l2 = w[32 * (KS * NG * 4 + 3 * g + 1)];
            const float n2 = w[32 * (KS * NG * 4 + 3 * g + 2)];
            const bool bad = st.l[g] < 0.f || l2 < 0.f;
            // a side that saw nothing (l = 0) has no maximum and no weight
            const float M = fmaxf(st.m[g], m2), N = fmaxf(st.n[g], n2);
            const float fl = st.l[g] == 0.f ? 0.f : exp2f(st.m[g] - M), f2 = l2 == 0.f ? 0.f : exp2f(m2 - M);
            const float fo = st.l[g] == 0.f ? 0.f : exp2f(st.n[g] - N), o2 = l2 == 0.f ? 0.f : exp2f(n2 - N);
            st.l[g] = bad ? -1.f : st.l[g] * fl + l2 * f2;
            st.m[g] = M;
            st.n[g] = N;
            // columns 2t and 2t + 1 of O^T are the rows of lanes 8t and 8t + 4
            const float fa = __shfl_sync(0xffffffffu, fo, 8 * tq), fb = __shfl_sync(0xffffffffu, fo, 8 * tq + 4);
            const float ga = __shfl_sync(0xffffffffu, o2, 8 * tq), gb = __shfl_sync(0xffffffffu, o2, 8 * tq + 4);
#pragma unroll
            for (int i = 0; i < KS; ++i)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                st.o[i][g][k] = st.o[i][g][k] * ((k & 1) ? fb : fa) +
                                w[32 * ((g * KS + i) * 4 + k)] * ((k & 1) ? gb : ga);
          }
        }
        slot0 += alive - half;
        alive = half;
        ++round;
      }
      ++nmerge;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.mempty[pair]);
      if (team > 0) continue;
    }
    const int used = min(RK, sg.n * a.G - row_base);  // rows of this warp that exist
    float *to = a.part + (static_cast<int64_t>(sg.part) * ngrp + pair) * (RK * RF);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      if constexpr (RK == 4) {  // columns 4..7 hold the remainders' sums
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            st.o[i][g][k] += __shfl_down_sync(0xffffffffu, st.o[i][g][k], 2);
      }
      const float la = __shfl_sync(0xffffffffu, st.l[g], 8 * tq);
      const float lb = __shfl_sync(0xffffffffu, st.l[g], 8 * tq + 4);
      const float ma = __shfl_sync(0xffffffffu, st.m[g], 8 * tq);
      const float mb = __shfl_sync(0xffffffffu, st.m[g], 8 * tq + 4);
      const float na = __shfl_sync(0xffffffffu, st.n[g], 8 * tq);
      const float nb = __shfl_sync(0xffffffffu, st.n[g], 8 * tq + 4);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 2 * tq + e + 8 * g;
        if (r >= used || r >= RK) continue;
        const float l = e ? lb : la, m = e ? mb : ma, n = e ? nb : na;
        if constexpr (kOwn) {
          const int i = (row_base + r) / a.G;
          float *here = a.rows + ((static_cast<int64_t>(a.rg.n_tokens) + sg.row0 + i) * a.Hq + kvh * a.G + row_base + r -
                                  i * a.G) * RF;
          float *o = sg.part < 0 ? here : to + r * RF;
#pragma unroll
          for (int c = 0; c < KS; ++c)
            *reinterpret_cast<float2 *>(o + (D / 8) * gq + 2 * c) = make_float2(st.o[c][g][e], st.o[c][g][2 + e]);
          if (gq == 0) {
            *reinterpret_cast<float4 *>(o + D) = make_float4(m, l, n, kHere);
            if (sg.part >= 0 && (sg.part & 1))  // the first part: where the others are
              *reinterpret_cast<float4 *>(here + D) =
                  make_float4(__int_as_float(sg.part >> 1), __int_as_float(sg.parts), 0.f, kCut);
          }
        } else if (sg.part < 0) {
          // 2^(n - m) / (l 2^7); a bad row is zeros, selected and not scaled
          const float2 f = out_scale(n - m - 7.f, l);
          float *o = ba_out_row<D>(a, sg, kvh, row_base + r) + (D / 8) * gq;
#pragma unroll
          for (int i = 0; i < KS; ++i)
            *reinterpret_cast<float2 *>(o + 2 * i) =
                l < 0.f ? make_float2(0.f, 0.f)
                        : make_float2(st.o[i][g][e] * f.x * f.y, st.o[i][g][2 + e] * f.x * f.y);
        } else {
          float *o = to + r * RF;
#pragma unroll
          for (int i = 0; i < KS; ++i)
            *reinterpret_cast<float2 *>(o + (D / 8) * gq + 2 * i) =
                make_float2(st.o[i][g][e], st.o[i][g][2 + e]);
          if (gq == 0) *reinterpret_cast<float4 *>(o + D) = make_float4(m, l, n, 0.f);
        }
      }
    }
  }
}

inline size_t ba_part_bytes(const BaShape &s, int D, int ctas) {
  return 2ull * ctas * s.hg * s.rt * s.rk * (D + kStat) * sizeof(float);
}

}  // namespace kvq
