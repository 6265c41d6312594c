// The tcgen05 split kernel of kvq_block_attn: head_dim 128 and many rows (query
// rows times heads of a kv head; the rule is at ba_shape).  Included by block_attn.cu.
//
// mma.sync would be the bound here: a warp's 16 rows need 48 MMAs a 16-token
// tile.  On tcgen05 the 8-bit kind multiplies the cache's bytes as they are
// (both K-major K and MN-major V are the pool's own layout), so nothing of the cache
// is converted.  What has to be 8-bit too is split into pieces:
//   q   a row scaled by 2^e (largest value in [224, 448)) = q1 + q2, e4m3 and e5m2:
//       exact for values down to 2^-13.8 of the row's largest (tc_q_pieces).
//       S = q2 K + q1 K in one accumulator.
//   w   a softmax weight (times 2^6, at most 2^7) = p1 + p2/2^5 + p3/2^10 + p4/2^15, e4m3
//       (tc_pieces): off by 2^-19 of w, and by 2^-24 where f16 and e4m3 are subnormal, that
//       is by 2^-30 of the row's largest weight: tokens far below an attention sink lose
//       no more here than in the mma.sync kernel (2^-31).  The
//       pieces of 32 rows are 128 columns of one product: piece p of row r is
//       column 32 p + r, and a row's four sums are added when they leave TMEM.
// Against 64 bits the result is as near as the mma.sync kernel's (1e-6 of the output's
// norm with large scores and values).
//
//   S[128 x 128 tokens] = Q[128 x 128] K^T   q's 32 rows four times over, so that
//       each of TMEM's four lane groups has them; a warp takes 16 tokens of its tile
//       (a row a lane, no shuffles)
//   O[128 dims x 128] += V^T[128 dims x 128 tokens] P^T   so that the pieces of a
//       row are columns of the same lane, and their sum needs no shared memory
//       (with dims as columns a segment's end took 18,000 cycles, now 12,000)
// An MMA of 128 x 128 x 32 takes 64 cycles alone, 768 a tile, of the 1,424 that its
// 32 KB take from HBM; its operands are 8 KB, all that shared memory gives in that
// time, so in company it takes about twice as long.  (The cache as the operand of 128
// rows in the scores too would leave every softmax thread with all rows of one
// token: measured 262 us against 138.)
//
// Roles: warps 0-7 and 8-15 two softmax groups with their own S and O (TMEM: 4 x 128
// columns), then one warp that issues the MMAs and two that issue the copies, of
// K and of V (a 16-token page is a copy of 2 KB, and 16 a tile are too many for
// one warp at HBM's rate), each into a ring of its own, since K is free after the
// scores and V only after the values.  The groups take a head's tiles in turn and
// are merged when the segment ends; the next segment's q and scores are made
// meanwhile.  Work is scheduled, cut and combined as in the mma.sync kernel, in units
// of 128 tokens of one head; more than 32 rows are row blocks, which follow one
// another so that the second reads the cache from L2.
//
// Measured: 32 requests of 1,024 - 16,384 tokens, 8 kv heads, 1 - 8 rows of 4 heads: 107.5
// us (mma.sync 203; HBM's floor 66).  A tile takes about 2,050 cycles of a CTA: a
// group's own chain (scores, maxima, rescaling, 64 conversions a thread, products) is
// 4,000 and two are in flight; a third group would have 72 registers a thread, and shared
// memory is full.  Without rescaling, three of the four pieces and half of the products it
// was 87 us, with each of them alone 96 - 100: no single step is the bound any more.
#pragma once

namespace kvq {

constexpr int kTcTok = 128;                 // tokens a tile
constexpr int kTcK = 4, kTcV = 4;           // ring slots; V's even, so that a slot belongs to one group
                                            // within a segment
constexpr int kTcWarps = 16;                // softmax warps, eight a group; then MMAs, K copies, V copies
constexpr int kTcThreads = 32 * (kTcWarps + 3);
constexpr int kTcRows = 32;                 // rows a row block holds
constexpr int kTcTile = kTcTok * 128;       // 16 KB: one tile of K or V, q piece, or weights
constexpr int kTcRowCost = 4;               // a row's start and end, in tiles' times
constexpr int kTcFlush = 16;                // tiles whose values a group's sum in TMEM takes
constexpr int kTcKept = 17 * 32;            // floats that a warp keeps in the workspace
// Lazy rescaling: weights stay below 2^1, and their operand, 2^6 of them, below 2^7 (the third
// piece of one above 2^7 could pass e4m3's largest value).  With 2^6 and 2^1 the row's largest
// operand might be 2^1 only, and tokens 14 nats below a sink lost up to 2^-5 of their weights;
// the more frequent rescaling takes 0.5% (32 drafts of 1 - 8 rows 106.8 us, so 107.4).
constexpr float kTcThreshold = 1.f;
constexpr float kTcWScale = 64.f;
constexpr float kTcFar = 64.f;              // the denominator's reference may be further off (fp32)
constexpr uint32_t kTcColS = 0, kTcColO = 256;

struct TcSeg {
  int b, head, rb;
  int row0, n, L;
  int rows;        // rows of this block that exist (1 .. 32)
  int t_begin, tiles, part;
};

struct __align__(16) TcRow {  // of a segment that ends: the groups' factors, the row's visible tokens, its place
  float mine, other, scale;
  int lim;
  int64_t at;  // -1: no such row
  int64_t pad;
};

struct TcCtl {
  TcSeg seg[kBaSegs];
  uint64_t kfull[kTcK], kempty[kTcK], vfull[kTcV], vempty[kTcV];
  uint64_t segfull[kBaSegs], segempty[kBaSegs];
  uint64_t qfull, qfree, sfull[2], sfree[2], pfull[2], pvdone[2];
  uint64_t xch[2], epi, drain;
  float2 sc[kTcV][kTcTok / 16];
  int bad[kTcV];                   // first token of a page outside the pool, or INT_MAX
  float qk[2][32];                 // [segment & 1]: what undoes q's scale, times sm_scale log2(e)
  float2 mx[2][2][8][32];          // [group][parity][warp][row]: a tile's maxima of x and x + log2 vs
  __align__(16) float grow[kTcWarps][32];  // [warp][row]: what a rescaling multiplies by
  __align__(16) TcRow row[kTcWarps][8];                // [warp][row]
  float4 stat[2][8][32];           // [group][warp][row]: m, l, n at a segment's end
  int nan_from[2][128];            // [segment & 1], per dim: the first drafted token with a NaN code there
  RunScan<kTcThreads> scan;
  uint32_t tmem;
  int fail;
};

// A whole warp waits, bounded; the usual case is one try.
__device__ __forceinline__ bool tc_wait(TcCtl &ctl, uint64_t *bar, uint32_t parity,
                                        uint32_t *err_word) {
  bool ok = mbar_try_wait(bar, parity);
  if (__all_sync(0xffffffffu, ok)) return true;
  if (!ok && !*reinterpret_cast<volatile int *>(&ctl.fail)) {
    ok = mbar_wait(bar, parity);
    if (!ok && atomicExch(&ctl.fail, 1) == 0) report(err_word, KVQ_ERRBIT_TIMEOUT);
  }
  return __all_sync(0xffffffffu, ok);
}

// fp32 += A * e4m3, 128 x n; A is e4m3 or e5m2; transposed: it is MN-major.
__host__ __device__ constexpr uint32_t tc_idesc(uint32_t n, bool transposed, bool e5m2) {
  return (1u << 4) | ((e5m2 ? 1u : 0u) << 7) | ((transposed ? 1u : 0u) << 15) | ((n >> 3) << 17) | ((128u >> 4) << 24);
}

__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(add ? 1 : 0)
      : "memory");
}

// e4m3 codes of two f16 values.
__device__ __forceinline__ uint32_t f16x2_to_e4m3x2(__half2 x) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c) : "r"(*reinterpret_cast<uint32_t *>(&x)));
  return c;
}

// One piece of two f16 values, and 32 times what is left of them (exact: at most the
// value's lower seven bits).  A piece is rounded to its four bits, so that what it
// leaves is at most 2^-4 of the value's binade, either way: 32 apart every piece starts in
// the binade of the one before.
__device__ __forceinline__ uint32_t tc_piece16(__half2 &x) {
  const uint32_t c = f16x2_to_e4m3x2(x), p = e4m3x2_to_f16x2(static_cast<uint16_t>(c));
  x = __hfma2(*reinterpret_cast<const __half2 *>(&p), __float2half2_rn(-32.f),
              __hmul2(x, __float2half2_rn(32.f)));
  return c;
}

// Two weights' four pieces, which leave at most 2^-19 of a weight: its f16 rounding
// carries the first two, what those leave of it joins with two pieces to go, on the
// f16's last bits (2^-21).  In fp32 throughout each piece's way back costs two more
// conversions.
__device__ __forceinline__ void tc_pieces(float2 w, int shift, uint32_t &c1, uint32_t &c2, uint32_t &c3,
                                          uint32_t &c4) {
  __half2 x = __float22half2_rn(w);
  const __half2 lo = __float22half2_rn(__ffma2_rn(__half22float2(x), make_float2(-1.f, -1.f), w));
  c1 |= tc_piece16(x) << shift;
  c2 |= tc_piece16(x) << shift;
  x = __hfma2(lo, __float2half2_rn(1024.f), x);
  c3 |= tc_piece16(x) << shift;
  c4 |= f16x2_to_e4m3x2(x) << shift;
}

// q's rows into the two piece tiles, each row at 32 p + r for every p; warp
// `warp` of sixteen takes two rows.
__device__ __forceinline__ void tc_load_q(const BaArgs &a, const TcSeg &sg, uint8_t *tiles, float *qk,
                                          int warp, int lane) {
  const int r = 2 * warp + (lane >> 4), part = lane & 15;  // 8 dims a lane
  const int row = sg.rb * kTcRows + r, i = row / a.G;
  float x[8];
  if (i < sg.n) {
    unpack8(__ldg(reinterpret_cast<const uint4 *>(
                a.q + (static_cast<int64_t>(sg.row0) + i) * a.q_stride +
                static_cast<int64_t>(sg.head * a.G + row - i * a.G) * 128 + 8 * part)),
            x);
  } else {
#pragma unroll
    for (int c = 0; c < 8; ++c) x[c] = 0.f;
  }
  float mx = 0.f;
  bool odd = false;  // inf or NaN: the row's scores are NaN, as inf - inf would make them
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    mx = fmaxf(mx, finite_abs(x[c]));
    odd |= !(fabsf(x[c]) < INFINITY);
  }
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  // largest value into [224, 448): block_exponent is the smallest e with mx <= 448 2^e
  const int e = block_exponent(mx);
  const float up = pow2(-e), nan = odd ? NAN : 0.f;
  uint32_t q1[2] = {0, 0}, q2[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < 4; ++k)
    tc_q_pieces(x[2 * k] * up + nan, x[2 * k + 1] * up + nan, 16 * (k & 1), q1[k >> 1], q2[k >> 1]);
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int at = 8 * (part & 1);
    *reinterpret_cast<uint2 *>(tc_chunk(tiles, 32 * p + r, part >> 1) + at) = make_uint2(q1[0], q1[1]);
    *reinterpret_cast<uint2 *>(tc_chunk(tiles + kTcTile, 32 * p + r, part >> 1) + at) =
        make_uint2(q2[0], q2[1]);
  }
  if (part == 0) qk[r] = a.q_scale * pow2(e);
}

// Every kTcFlush tiles the sums leave TMEM, and are added with rounding to others in
// the workspace: the tensor core's additions truncate (towards zero), and a long sum there
// drifts, 1.3e-5 of it over 65,536 tokens, measured; 1e-7 are left, for 3% of the time.  This
// thread's dim of 16 rows, eight at a time (with all in registers the loop around spills, and 128
// requests of 64 - 1,024 tokens take 4% longer): kept times `keep`, the pieces times `fo`.
__device__ __forceinline__ void tc_flush(float *kept, bool first, float keep, float fo, float *rows,
                                         uint32_t addr, int half, int lane) {
#pragma unroll 1
  for (int k0 = 0; k0 < 16; k0 += 8) {
    float acc[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] = first ? 0.f : kept[32 * (k0 + k)];
    rows[lane] = keep;
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] *= rows[16 * half + k0 + k];
    __syncwarp();
    rows[lane] = fo;
    __syncwarp();
    float down = 1.f / 32768;  // the smallest pieces first
#pragma unroll 1
    for (int p = 3; p >= 0; --p, down *= 32.f) {
      float o[8];
      uint32_t *r = reinterpret_cast<uint32_t *>(o);
      asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                   : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                     "=r"(r[7])
                   : "r"(addr + 32 * p + k0));
      asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = fmaf(o[k] * down, rows[16 * half + k0 + k], acc[k]);
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 8; ++k) kept[32 * (k0 + k)] = acc[k];
  }
}

__global__ void __launch_bounds__(kTcThreads, 1)
    block_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                    BaArgs a) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  uint8_t *kt = smem;                       // K tiles
  uint8_t *vtl = kt + kTcK * kTcTile;       // V tiles
  uint8_t *qt = vtl + kTcV * kTcTile;       // q, [2 pieces]
  uint8_t *pt = qt + 2 * kTcTile;           // weights, [group]
  TcCtl &ctl = *reinterpret_cast<TcCtl *>(pt + 2 * kTcTile);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kTcK; ++i) {
      mbar_init(&ctl.kfull[i], 1);
      mbar_init(&ctl.kempty[i], 1);
    }
    for (int i = 0; i < kTcV; ++i) {
      mbar_init(&ctl.vfull[i], 1 + 8);  // and the scales of its eight blocks
      mbar_init(&ctl.vempty[i], 1);
    }
    for (int i = 0; i < kBaSegs; ++i) {
      mbar_init(&ctl.segfull[i], 1);
      mbar_init(&ctl.segempty[i], kTcWarps + 1);  // the softmax warps and the MMA warp
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(&ctl.sfull[g], 1);
      mbar_init(&ctl.sfree[g], 8);
      mbar_init(&ctl.pfull[g], 8);
      mbar_init(&ctl.pvdone[g], 1);
      mbar_init(&ctl.xch[g], 8);
    }
    mbar_init(&ctl.qfull, kTcWarps);
    mbar_init(&ctl.qfree, 1);
    mbar_init(&ctl.epi, kTcWarps);
    mbar_init(&ctl.drain, 1);
    ctl.fail = 0;
    fence_barrier_init();
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&kmap)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&vmap)) : "memory");
  }
  if (warp == kTcWarps) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_addr(&ctl.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = ctl.tmem;
  grid_dependency_wait();
  const RunStart run = find_run<kTcThreads>(
      a.rg.B, gridDim.x, blockIdx.x, ctl.scan, [&](int b) -> int64_t {
        bool live;
        const Rows r = ba_rows(a, b, live);
        if (r.err && blockIdx.x == 0) report(a.err_word, r.err);
        return live ? static_cast<int64_t>((r.p0 + r.n + kTcTok - 1) / kTcTok + kTcRowCost) * a.groups *
                          ba_blocks(a, r, kTcRows)
                    : 0;
      });
  allow_dependents();
  const int64_t u0 = blockIdx.x * run.per;
  const int64_t u1 = min(u0 + run.per, run.total);

  if (warp > kTcWarps) {
    // ----------------------------------------------- producers: K, then V
    const int is_v = warp - kTcWarps - 1;
    const CUtensorMap *map = is_v ? &vmap : &kmap;
    uint64_t *full = is_v ? ctl.vfull : ctl.kfull, *empty = is_v ? ctl.vempty : ctl.kempty;
    uint8_t *tiles_at = is_v ? vtl : kt;
    const uint32_t stages = is_v ? kTcV : kTcK;
    const uint64_t once = policy_evict_first();
    uint64_t again;  // the cache is read by several row blocks
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(again));
    int64_t u = u0, in = run.in;
    int b = run.b;
    BaCut cut = {0, 0, 0, 0, 0, {0, 0, 0}};
    uint32_t g = 0, nseg = 0, par = 1, slot = 0;
    bool ok = true;
    int win_b = -1, win = 0, cur = -1, nxt = -1;
    const int32_t *bt = a.block_table;
    auto bt_load = [&](int lp) -> int { return lp < a.MP ? __ldg(bt + lp) : -1; };
    while (ok && u < u1) {
      bool live;
      const Rows rq = ba_rows(a, b, live);
      const int tiles = live ? (rq.p0 + rq.n + kTcTok - 1) / kTcTok : 0, units = tiles + kTcRowCost;
      const int nb = live ? ba_blocks(a, rq, kTcRows) : 0;
      const int64_t have = static_cast<int64_t>(units) * a.groups * nb;
      if (in >= have) {
        ++b;
        in = 0;
        continue;
      }
      const int64_t rw = in / units;
      const int s = static_cast<int>(in - rw * units);
      const int head = static_cast<int>(rw / nb), rb = static_cast<int>(rw - static_cast<int64_t>(head) * nb);
      const uint64_t pol = nb > 1 ? again : once;
      const int span = static_cast<int>(min(static_cast<int64_t>(units - s), u1 - u));
      const int t0 = max(0, s - kTcRowCost), take = s + span - kTcRowCost - t0;
      const int64_t ut = u - s + kTcRowCost;
      u += span;
      in += span;
      if (take <= 0) continue;
      const int L = rq.p0 + rq.n;
      const int64_t c_lo = ut / run.per;
      const int nparts = static_cast<int>((ut + tiles - 1) / run.per - c_lo) + 1;
      const int ss = nseg % kBaSegs;
      if (!is_v && nseg >= kBaSegs)
        ok = tc_wait(ctl, &ctl.segempty[ss], ((nseg / kBaSegs) - 1) & 1, a.err_word);
      if (!ok) break;
      if (!is_v && lane == 0) {
        if (t0 == 0 && nparts > 1) cut = {nparts, head, rb, rq.row, rq.n, {0, 0, 0}};
        ctl.seg[ss] = {b, head, rb, rq.row, rq.n, L, min(rq.n * a.G - rb * kTcRows, kTcRows),
                       t0 * kTcTok, take,
                       nparts == 1 ? -1 : 2 * static_cast<int>(blockIdx.x) + (t0 == 0 ? 1 : 0)};
        mbar_arrive(&ctl.segfull[ss]);
      }
      ++nseg;
      const int lp0 = (t0 * kTcTok) >> a.p_shift;
      if (b != win_b || lp0 < win || lp0 >= win + 32) {
        win_b = b;
        win = lp0;
        bt = a.block_table + static_cast<int64_t>(b) * a.MP;
        cur = bt_load(win + lane);
        nxt = bt_load(win + 32 + lane);
      }
      for (int st = 0, tok = t0 * kTcTok; st < take; ++st, tok += kTcTok) {
        ok = tc_wait(ctl, &empty[slot], par, a.err_word);
        if (!ok) break;
        if ((tok >> a.p_shift) >= win + 32) {
          win += 32;
          cur = nxt;
          nxt = bt_load(win + 32 + lane);
        }
        // lane j < 8: tokens tok + 16 j ..; their page lies within two windows
        const int mine = tok + 16 * (lane & 7);
        const int idx = (mine >> a.p_shift) - win;
        const int from_cur = __shfl_sync(0xffffffffu, cur, idx & 31);
        const int from_nxt = __shfl_sync(0xffffffffu, nxt, idx & 31);
        const int page = idx < 32 ? from_cur : from_nxt;
        const bool needed = lane < 8 && mine < L;
        const bool good = needed && page >= 0 && page < a.num_pages;
        const uint32_t goods = __ballot_sync(0xffffffffu, good);
        const uint32_t needs = __ballot_sync(0xffffffffu, needed);
        if (lane == 0) {
          if (is_v) ctl.bad[slot] = needs == goods ? INT_MAX : tok + 16 * (__ffs(needs ^ goods) - 1);
          if (needs != goods) report(a.err_word, KVQ_ERRBIT_PAGE);
          mbar_arrive_expect_tx(&full[slot], static_cast<uint32_t>(__popc(goods)) * 2048u);
        }
        __syncwarp();
        int pages[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) pages[j] = __shfl_sync(0xffffffffu, page, j);
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (goods >> j & 1)
              tma_load_4d(tiles_at + slot * kTcTile + 2048 * j, map, 0,
                          (tok + 16 * j) & ((1 << a.p_shift) - 1), head, pages[j], &full[slot], pol);
        }
        __syncwarp();
        if (is_v && lane < 8) {
          if (good) {
            cp_async8(&ctl.sc[slot][lane], a.scales + static_cast<int64_t>(page) * a.Hkv + head);
            cp_async_arrive(&full[slot]);
          } else {
            ctl.sc[slot][lane] = make_float2(1.f, 1.f);  // masked tokens
            mbar_arrive(&full[slot]);
          }
        }
        ++g;
        if (++slot == stages) {
          slot = 0;
          par ^= 1;
        }
        __syncwarp();
      }
    }
    if (!is_v && lane == 0) a.cut[blockIdx.x] = cut;
    if (ok && !is_v) {  // nothing more
      const int ss = nseg % kBaSegs;
      if (nseg >= kBaSegs) ok = tc_wait(ctl, &ctl.segempty[ss], ((nseg / kBaSegs) - 1) & 1, a.err_word);
      if (ok && lane == 0) {
        ctl.seg[ss].b = -1;
        mbar_arrive(&ctl.segfull[ss]);
      }
    }
    if (*reinterpret_cast<volatile int *>(&ctl.fail) && lane == 0)
      for (uint32_t k = g > stages ? g - stages : 0; k < g; ++k)
        mbar_wait(&full[k % stages], (k / stages) & 1);
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == kTcWarps) {
    // ------------------------------------------------------------ MMA issue
    uint32_t nseg = 0, g0 = 0;
    uint32_t ns[2] = {0, 0}, np[2] = {0, 0};  // S and P tiles so far
    uint32_t kg = 0;                          // K tiles so far
    bool ok = true;
    const uint32_t k_a = smem_addr(kt), v_a = smem_addr(vtl), q_a = smem_addr(qt), p_a = smem_addr(pt);
    // a tile's scores, once its group has taken its last ones out of TMEM
    auto issue_s = [&](int g, bool last) -> bool {
      const int slot = kg % kTcK;
      if (!tc_wait(ctl, &ctl.kfull[slot], (kg / kTcK) & 1, a.err_word) ||
          !tc_wait(ctl, &ctl.sfree[g], (ns[g]++ & 1) ^ 1, a.err_word))
        return false;
      ++kg;
      tc_after();
      if (elect_one()) {
        const uint64_t kd = tc_desc(k_a + slot * kTcTile), qd = tc_desc(q_a);
#pragma unroll
        for (int piece = 1; piece >= 0; --piece)  // the smaller first: each sum is truncated
#pragma unroll
          for (int k = 0; k < 4; ++k)  // 32 dims each: 32 bytes within the swizzled rows
            tc_mma(tmem + kTcColS + 128 * g, qd + piece * (kTcTile >> 4) + 2 * k, kd + 2 * k,
                   tc_idesc(128, false, piece == 1), piece == 0 || k > 0);
        tc_commit(&ctl.sfull[g]);
        tc_commit(&ctl.kempty[slot]);
        if (last) tc_commit(&ctl.qfree);
      }
      __syncwarp();
      return true;
    };
    auto issue_pv = [&](int g, int slot, bool add) {
      if (elect_one()) {
        const uint64_t vd = tc_desc(v_a + slot * kTcTile), pd = tc_desc(p_a + g * kTcTile);
#pragma unroll
        for (int k = 0; k < 4; ++k)  // 32 tokens each: 32 bytes of P's rows, 32 rows of V
          tc_mma(tmem + kTcColO + 128 * g, vd + k * (32 * 128 >> 4), pd + 2 * k, tc_idesc(128, true, false),
                 add || k > 0);
        tc_commit(&ctl.pvdone[g]);
        tc_commit(&ctl.vempty[slot]);
      }
      __syncwarp();
    };
    while (ok) {
      const int ss = nseg % kBaSegs;
      ok = tc_wait(ctl, &ctl.segfull[ss], (nseg / kBaSegs) & 1, a.err_word);
      if (!ok) break;
      const TcSeg sg = ctl.seg[ss];
      if (sg.b < 0) break;
      ok = tc_wait(ctl, &ctl.qfull, nseg & 1, a.err_word);
      // A tile's scores are issued when its group has taken those of two tiles before
      // out of TMEM, and are there when it has done that tile's weights.  The groups
      // are half a tile's time apart, so that the order of their waits is this one's.
      for (int t = -2; ok && t <= sg.tiles; ++t) {
        if (t + 2 < sg.tiles) ok = issue_s(t & 1, t + 3 == sg.tiles);
        const int u = t - 1;
        if (!ok || u < 0 || u >= sg.tiles) continue;
        // (the group's warps have waited for the tile of V)
        const int g = u & 1;
        ok = tc_wait(ctl, &ctl.pfull[g], np[g]++ & 1, a.err_word);
        if (!ok) break;
        tc_after();
        issue_pv(g, (g0 + u) % kTcV, (u >> 1) % kTcFlush != 0);
      }
      g0 += sg.tiles;
      ++nseg;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.segempty[ss]);
    }
    if (*reinterpret_cast<volatile int *>(&ctl.fail)) {
      // the products in flight end before the CTA's memory goes to another one
      if (elect_one()) tc_commit(&ctl.drain);
      mbar_wait(&ctl.drain, 0);
    }
  } else {
    // ------------------------------------------------------------- softmax
    // rows of requests without work are zeros
    for (int b = blockIdx.x; b < a.rg.B; b += gridDim.x) {
      bool live;
      const Rows r = ba_rows(a, b, live);
      if (live || r.n == 0) continue;
      float4 *o = reinterpret_cast<float4 *>(a.out + static_cast<int64_t>(r.row) * a.Hq * 128);
      const int64_t n4 = static_cast<int64_t>(r.n) * a.Hq * 32;
      for (int64_t k = threadIdx.x; k < n4; k += 32 * kTcWarps) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    // group, TMEM lanes, and half of the lanes' 32 tokens
    const int grp = warp >> 3, quad = warp & 3, half = (warp >> 2) & 1, gw = 2 * quad + half;
    const uint32_t lanes = static_cast<uint32_t>(32 * quad) << 16;
    const uint32_t s_addr = tmem + lanes + kTcColS + 128 * grp + 16 * gw;
    const uint32_t o_addr = tmem + lanes + kTcColO + 128 * grp;
    uint8_t *ptile = pt + grp * kTcTile;
    uint32_t nseg = 0, g0 = 0, nt = 0, nx = 0, ne = 0;
    auto group_sync = [&]() -> bool {  // the group's eight warps
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.xch[grp]);
      return tc_wait(ctl, &ctl.xch[grp], nx++ & 1, a.err_word);
    };
    auto both_sync = [&]() -> bool {  // both groups
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.epi);
      return tc_wait(ctl, &ctl.epi, ne++ & 1, a.err_word);
    };
    // Segment k's q, while segment k - 1 still sums its values: its scores are
    // there when that one has been written.  A wait for the segment's descriptor holds
    // nothing up that it needs: the copies post it when those before it are issued.
    auto load_q = [&](uint32_t k) -> bool {
      const int s = k % kBaSegs;
      if (!tc_wait(ctl, &ctl.segfull[s], (k / kBaSegs) & 1, a.err_word)) return false;
      const TcSeg next = ctl.seg[s];
      if (next.b < 0) return true;
      if (k > 0 && !tc_wait(ctl, &ctl.qfree, (k - 1) & 1, a.err_word)) return false;
      if (threadIdx.x < 128) ctl.nan_from[k & 1][threadIdx.x] = INT_MAX;  // last read in segment k - 2
      tc_load_q(a, next, qt, ctl.qk[k & 1], warp, lane);
      proxy_fence();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.qfull);
      return true;
    };
    bool ok = load_q(0);
    while (ok) {
      const int ss = nseg % kBaSegs;
      const TcSeg sg = ctl.seg[ss];
      if (sg.b < 0) break;
      const int row = sg.rb * kTcRows + lane;  // of the request
      const int my_i = row / a.G;
      const int lim = my_i < sg.n ? sg.L - sg.n + 1 + my_i : sg.L;
      const int min_lim = min(sg.L, sg.L - sg.n + 1 + (sg.rb * kTcRows) / a.G);
      ok = tc_wait(ctl, &ctl.qfull, nseg & 1, a.err_word);
      if (!ok) break;
      const float qk = ctl.qk[nseg & 1][lane];
      int *nan_from = ctl.nan_from[nseg & 1];
      float m = -INFINITY, n = -INFINITY, l = 0.f;
      bool any_tile = false;
      int bad_from = INT_MAX;  // rows that see this token are zeros; others have it masked
      for (int t = grp; t < sg.tiles; t += 2) {
        const uint32_t gg = g0 + t;
        const int slot = gg % kTcV;
        const int tok0 = sg.t_begin + t * kTcTok, tw = tok0 + 16 * gw;  // this warp's tokens: one block
        ok = tc_wait(ctl, &ctl.sfull[grp], nt & 1, a.err_word) &&
             tc_wait(ctl, &ctl.vfull[slot], (gg / kTcV) & 1, a.err_word);
        if (!ok) break;
        bad_from = min(bad_from, ctl.bad[slot]);
        tc_after();
        float x[16];
        tc_ld16(x, s_addr);
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.sfree[grp]);
        const bool partial = tok0 + kTcTok > min_lim;
        const float2 sc = ctl.sc[slot][gw];
        const float2 v_scale = split_scale(sc.y);
        const float vm = v_scale.x, lv = v_scale.y, f = qk * sc.x;
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          float y = x[c] * f;
          if (partial && tw + c >= lim) y = -INFINITY;
          x[c] = y;
          mx = fmaxf(mx, y);
        }
        float mv = mx + lv;
        float2(*xm)[32] = ctl.mx[grp][nt & 1];
        xm[gw][lane] = make_float2(mx, mv);
        ok = group_sync();
        if (!ok) break;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          const float2 o = xm[w][lane];
          mx = fmaxf(mx, o.x);
          mv = fmaxf(mv, o.y);
        }
        // the row's references: the same in all of the group's warps
        if (mx > m + kTcFar) {
          l *= exp2f(m - mx);
          m = mx;
        }
        float fo = 1.f;
        if (mv > n + kTcThreshold) {
          fo = exp2f(n - mv);
          n = mv;
        }
        // the group's product before this one has been read and summed
        if (any_tile) {
          ok = tc_wait(ctl, &ctl.pvdone[grp], (nt & 1) ^ 1, a.err_word);
          if (!ok) break;
          const bool flush = (t >> 1) % kTcFlush == 0;
          if (flush || __any_sync(0xffffffffu, fo != 1.f)) {
            float *grow = ctl.grow[warp];
            tc_after();
            if (flush) {
              float *kept = a.kept + static_cast<int64_t>(blockIdx.x * kTcWarps + warp) * kTcKept + lane;
              const bool first = (t >> 1) == kTcFlush;
              const float kept_n = first ? n : kept[16 * 32];  // the kept sums' reference
              kept[16 * 32] = n;
              tc_flush(kept, first, kept_n == n ? 1.f : exp2f(kept_n - n), fo, grow, o_addr + 16 * half, half, lane);
            } else {
              grow[lane] = fo;
              __syncwarp();
            }
#pragma unroll 1
            for (int c = 64 * half; !flush && c < 64 * half + 64; c += 16) {  // 16 rows of a piece
              float o[16];
              tc_ld16(o, o_addr + c);
#pragma unroll
              for (int k = 0; k < 16; k += 4) {
                const float4 g = *reinterpret_cast<const float4 *>(grow + (c & 16) + k);
                o[k] *= g.x;
                o[k + 1] *= g.y;
                o[k + 2] *= g.z;
                o[k + 3] *= g.w;
              }
              tc_st16(o_addr + c, o);
            }
            __syncwarp();
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
          }
        }
        any_tile = true;
        const bool none = n == -INFINITY;  // nothing seen yet: every x is -inf
        const float mm = none ? 0.f : m, mn = none ? 0.f : m - n;
        // vs 2^(m - n), times 2^6 (kTcThreshold keeps the operand below 2^7)
        const float d = vm * kTcWScale * fast_exp2(fminf(mn + lv, 112.f));
        float2 l2 = make_float2(0.f, 0.f);
        uint32_t w1[4], w2[4], w3[4], w4[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t c1 = 0, c2 = 0, c3 = 0, c4 = 0;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int c = 4 * k + 2 * j;
            const float2 y = __fadd2_rn(make_float2(x[c], x[c + 1]), make_float2(-mm, -mm));
            const float2 e = make_float2(fast_exp2(y.x), fast_exp2(y.y));
            l2 = __fadd2_rn(l2, e);
            tc_pieces(__fmul2_rn(e, make_float2(d, d)), 16 * j, c1, c2, c3, c4);
          }
          w1[k] = c1;
          w2[k] = c2;
          w3[k] = c3;
          w4[k] = c4;
        }
        l += l2.x + l2.y;
        *reinterpret_cast<uint4 *>(tc_chunk(ptile, lane, gw)) = make_uint4(w1[0], w1[1], w1[2], w1[3]);
        *reinterpret_cast<uint4 *>(tc_chunk(ptile, 32 + lane, gw)) = make_uint4(w2[0], w2[1], w2[2], w2[3]);
        *reinterpret_cast<uint4 *>(tc_chunk(ptile, 64 + lane, gw)) = make_uint4(w3[0], w3[1], w3[2], w3[3]);
        *reinterpret_cast<uint4 *>(tc_chunk(ptile, 96 + lane, gw)) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
        if (partial) {
          // V rows past the end (whatever the slot or the cache holds) become
          // zeros, and NaN codes of drafted tokens (and of a bad page's stale rows) too: a
          // weight of 0 does not stop a NaN.  Rows that see such a token get their NaN when they are written.
          const int tr = 32 * quad + lane, tok = tok0 + tr;
          uint8_t *vt = vtl + slot * kTcTile;
          if (tok >= sg.L) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              *reinterpret_cast<uint4 *>(tc_chunk(vt, tr, 4 * half + c)) = make_uint4(0, 0, 0, 0);
          } else if (tok >= min_lim) {
            uint32_t nan = 0;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint4 v = *reinterpret_cast<const uint4 *>(tc_chunk(vt, tr, 4 * half + c));
              nan |= nan_codes(v.x) | nan_codes(v.y) | nan_codes(v.z) | nan_codes(v.w);
            }
            if (nan) {
              for (int k = 64 * half; k < 64 * half + 64; ++k) {
                uint8_t *p = tc_chunk(vt, tr, k >> 4) + (k & 15);
                if ((*p & 0x7F) != 0x7F) continue;
                *p = 0;
                atomicMin(&nan_from[k], tok);
              }
            }
          }
        }
        ++nt;
        proxy_fence();
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.pfull[grp]);
      }
      if (!ok) break;
      g0 += sg.tiles;

      // ---- the segment's end
      ok = load_q(nseg + 1);
      if (!ok) break;
      if (any_tile) {
        ok = tc_wait(ctl, &ctl.pvdone[grp], (nt & 1) ^ 1, a.err_word);
        if (!ok) break;
        tc_after();
      }
      // this thread's dim (32 quad + lane) of 16 rows: the pieces' sum, smallest first
      float sum[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) sum[k] = 0.f;
      if (any_tile) {
#pragma unroll
        for (int p = 3; p >= 0; --p) {
          float o[16];
          tc_ld16(o, o_addr + 32 * p + 16 * half);
          const float down = p == 0 ? 1.f : p == 1 ? 1.f / 32 : p == 2 ? 1.f / 1024 : 1.f / 32768;
#pragma unroll
          for (int k = 0; k < 16; ++k) sum[k] = fmaf(o[k], down, sum[k]);
        }
      }
      if (sg.tiles > 2 * kTcFlush + grp) {  // and what was flushed
        const float *kept = a.kept + static_cast<int64_t>(blockIdx.x * kTcWarps + warp) * kTcKept + lane;
        float *grow = ctl.grow[warp];
        const float kept_n = kept[16 * 32];
        grow[lane] = kept_n == n ? 1.f : exp2f(kept_n - n);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 16; ++k) sum[k] = fmaf(kept[32 * k], grow[16 * half + k], sum[k]);
      }
      // group 0 writes the first eight of them and group 1 the others; each hands the
      // other its sums of those, [half][row][dim], in its own (free) weight tile
      const int dim = 32 * quad + lane;
      float *give = reinterpret_cast<float *>(ptile) + 1024 * half + dim;
      const float *take = reinterpret_cast<const float *>(pt + (grp ^ 1) * kTcTile) + 1024 * half + dim;
      if (grp == 0) {
#pragma unroll
        for (int k = 0; k < 8; ++k) give[128 * k] = sum[8 + k];
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          give[128 * k] = sum[k];
          sum[k] = sum[8 + k];
        }
      }
      ctl.stat[grp][gw][lane] = make_float4(m, lim > bad_from ? -1.f : l, n, 0.f);
      ok = both_sync();
      if (!ok) break;
      float M = -INFINITY, N = -INFINITY, L1 = 0.f, gm[2], gn[2], gl[2], f[2];
      bool bad = false;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        gl[k] = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          const float4 v = ctl.stat[k][w][lane];
          bad |= v.y < 0.f;
          gl[k] += v.y;
          gm[k] = v.x;
          gn[k] = v.z;
        }
        if (gl[k] != 0.f) {  // (also NaN); a group that saw nothing has no weight
          M = fmaxf(M, gm[k]);
          N = fmaxf(N, gn[k]);
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        f[k] = gl[k] != 0.f ? exp2f(gn[k] - N) : 0.f;
        if (gl[k] != 0.f) L1 += gl[k] * exp2f(gm[k] - M);
      }
      const bool used = lane < sg.rows;
      // a partial's row: sums, then m, l, n (n counts the 2^7 of the other kernel, here 2^6)
      const int64_t at = sg.part < 0 ? ((static_cast<int64_t>(sg.row0) + my_i) * a.Hq + sg.head * a.G + row -
                                        my_i * a.G) * 128
                                     : (static_cast<int64_t>(sg.part) * kTcRows + lane) * (128 + kStat);
      float *out = sg.part < 0 ? a.out : a.part;
      {
        // out = 2^(N - M - 6) sum / l; zeros where the row sees a bad page.  Half of a power far from
        // 1 goes to the groups' factors (out_scale says why; one more factor a value took 3%
        // of the time of 128 requests of 64 - 1,024 tokens)
        const float t = N - M - 6.f;
        const float h = sg.part >= 0 || fabsf(t) <= 60.f ? 0.f : rintf(fminf(fmaxf(0.5f * t, -100.f), 100.f));
        const float scale = sg.part < 0 ? exp2f(t - h) / L1 : 1.f, up = pow2(static_cast<int>(h));
        const bool zero = bad && sg.part < 0;
        TcRow w;
        w.mine = zero ? 0.f : f[grp] * up;
        w.other = zero ? 0.f : f[grp ^ 1] * up;
        w.scale = zero ? 0.f : scale;
        w.lim = zero ? INT_MIN : lim;
        w.at = used ? at : -1;
        const int k = lane - 16 * half - 8 * grp;
        if (k >= 0 && k < 8) ctl.row[warp][k] = w;
      }
      __syncwarp();
      const int nan_at = nan_from[dim];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const TcRow w = ctl.row[warp][k];
        const float other = take[128 * k];
        float acc = 0.f;
        if (w.mine != 0.f) acc = w.mine * sum[k];
        if (w.other != 0.f) acc = fmaf(w.other, other, acc);
        acc = nan_at < w.lim ? NAN : acc * w.scale;
        if (w.at >= 0) out[w.at + dim] = acc;
      }
      ok = both_sync();  // the tiles and nan_from are read
      if (!ok) break;
      if (used && sg.part >= 0 && warp == 0)
        *reinterpret_cast<float4 *>(out + at + 128) = make_float4(M, bad ? -1.f : L1, N + 1.f, 0.f);
      ++nseg;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.segempty[ss]);
    }
    tc_before();
  }
  __syncthreads();  // every role comes here, also when a wait gave up
  if (warp == kTcWarps) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

inline size_t tc_smem_bytes() {
  return static_cast<size_t>(kTcK + kTcV + 4) * kTcTile + sizeof(TcCtl) + 1024;
}

}  // namespace kvq
