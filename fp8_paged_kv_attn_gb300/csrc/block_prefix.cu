// kvq_block_prefix_attn: causal attention over the block-scaled cache for a batch
// whose requests form groups with a shared prefix of whole pages.
//
// Softmax over a row's tokens in any number of parts: with m, a reference of the scores x (base 2), and
// n, one of x + log2 v for the V scales v, a part is
//   l = sum 2^(x - m),   O = sum (2^(x - m) v 2^(m - n) 2^7) c   (c a token's V code),
// and parts are joined as  out = 2^(N - M - 7) sum_p 2^(n_p - N) O_p / sum_p 2^(m_p - M) l_p.
// The two references keep the operand of the second product in f16's range however far apart the V
// scales are; both follow their maxima lazily.  A prefix is a part of every row of its group, read once for
// 128 rows of it (times heads a kv head); a request's own tokens are another.
//
// Four launches: the plan and q's pieces; prefixes (prefix_kernel, tcgen05); own tokens (the mma.sync kernel
// of kvq_block_attn, where a request has few rows); the merge.  Measured on 256 requests of 64 heads over 8
// behind 32,768 tokens: 10, 273, 28 and 20 us one by one and cold, 315 in all (kvq_block_attn, which reads
// the prefix for every request: 2,556).
//
// What bounds prefix_kernel: a tile (128 rows, 128 tokens, head_dim 128) is 1,080 cycles of the tensor core (8 of
// its steps for the scores, q being two 8-bit pieces, 8 in f16 for the values) and some 1,150 of shared
// memory (V goes through it a second time, as f16), and takes 2,380: tensor pipe 43%, issue slots 50%.  The softmax
// groups need 3,500 - 4,000 cycles a tile each, two in turn, and the MMA warp's own instructions
// and waits beside the softmax's take 1,300 a tile.  Weights are f16 (2^-11), not kvq_block_attn's four
// 8-bit pieces (2^-19), since the output is bf16 (2^-8): a quarter of the products.
#include <algorithm>
#include <atomic>
#include <climits>

#include "block_common.cuh"
#include "decode_common.cuh"
#include "decode_attn_mma.cuh"
#include "tc_device.cuh"
#include "block_attn_split.cuh"

namespace kvq {

struct PfArgs {
  const uint16_t *q;
  int64_t q_stride;
  uint8_t *qp;    // [n_tokens][Hq][2][D]: q's two pieces
  float *qk;      // [n_tokens][Hq]: what undoes their scale, times |sm_scale| log2(e)
  PxPlan *plan;
  PxItem *items;         // [2 n_tokens]: groups' prefixes, then requests
  int64_t *units;        // [2 n_tokens + 1]: units before each item
  Ragged rg;
  const int32_t *block_table, *group_start, *prefix_pages;
  const uint8_t *abort_mask;
  const float2 *scales;  // [num_pages][Hkv]
  float *rows;  // [2][n_tokens][Hq][D + kStat]: a row's prefix, and its own tokens
  float *cut;   // [2 CTAs][kPxRows][D + kStat]: parts of rows of work that CTAs share
  uint16_t *out;
  uint32_t *err_word;
  int32_t num_pages, p_shift, Hkv, Hq, G, MP, max_q, n_groups;
  int32_t own_split;  // own tokens are attended to by the mma.sync kernel; its shape:
  int32_t hg, rt, rk;
  const float *own_cut;
  float q_scale;  // sm_scale * log2(e)
};

// A request's rows and the tokens in front of its own: those of its group's prefix.
struct PfReq {
  Rows r;
  int pre;     // tokens of the prefix
  int group;   // or -1
  bool live;
};

// The group that holds request b, or -1; group_start is in order (checked apart).
__device__ __forceinline__ int pf_group(const PfArgs &a, int b) {
  if (a.n_groups == 0 || b < __ldg(a.group_start) || b >= __ldg(a.group_start + a.n_groups)) return -1;
  int lo = 0, hi = a.n_groups - 1;
  while (lo < hi) {  // the last that starts at b or before
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(a.group_start + mid) <= b)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// The rows [x, y) of a group's requests.
__device__ __forceinline__ int2 pf_group_rows(const PfArgs &a, int g) {
  const int s = __ldg(a.group_start + g), e = __ldg(a.group_start + g + 1);
  const int x = a.rg.tok_start ? __ldg(a.rg.tok_start + s) : s;
  const int y = a.rg.tok_start ? __ldg(a.rg.tok_start + e) : e;
  return make_int2(max(x, 0), min(y, a.rg.n_tokens));
}

__device__ __forceinline__ PfReq pf_request(const PfArgs &a, int b) {
  PfReq o;
  o.r = request_rows<true>(a.rg, b);
  o.group = pf_group(a, b);
  const int pages = o.group < 0 ? 0 : __ldg(a.prefix_pages + o.group);
  const bool bad = pages < 0 || pages > a.MP;
  o.pre = bad ? 0 : pages << a.p_shift;
  if (!o.r.err && o.r.n > 0 && (o.r.n > a.max_q || bad || o.r.p0 < o.pre)) o.r.err = KVQ_ERRBIT_SEQLEN;
  if (!o.r.err && o.pre > 0) {  // the prefix is read for the rows between the group's ends
    const int2 rows = pf_group_rows(a, o.group);
    if (o.r.n > 0 && (o.r.row < rows.x || o.r.row + o.r.n > rows.y)) o.r.err = KVQ_ERRBIT_REQ;
  }
  o.live = o.r.n > 0 && !o.r.err && !(a.abort_mask && __ldg(a.abort_mask + b) != 0);
  return o;
}

// Whether group_start is in order and within the batch.
__device__ __forceinline__ bool pf_group_ok(const PfArgs &a, int g) {
  const int s = __ldg(a.group_start + g), e = __ldg(a.group_start + g + 1);
  return s >= 0 && s <= e && e <= a.rg.B;
}

// ---------------------------------------------------------------------------
// work: items, rows of work, segments
// ---------------------------------------------------------------------------

constexpr int kPxTok = 128;         // tokens a tile
constexpr int kPxRows = 128;        // rows a block
// Tiles of a row of work that the tensor core sums before the sums are taken out and added with rounding.  Its
// additions truncate, up to 2^-27 of a sum of one sign for each token: 2^-12 for these 32,768, and half a bf16
// step for 262,144 (summed without a limit, a million tokens' means that stand 2^-11 above a rounding's
// border came out a bf16 step too small).
constexpr int kPxSumTiles = 256;
constexpr int kPxRowCost = 2;       // a row of work's start and end, in tiles' times (1 - 6: within 3%)
constexpr int kPxSegs = 8;          // segment descriptors in flight
constexpr int kPxStats = 4;         // segments whose statistics are in flight
constexpr int kPxScales = 8;        // tiles whose scales are in flight
constexpr int kPxK = 4, kPxV = 4;   // tiles of K and of V in flight
// warps: softmax (two groups of four), sides (q in, V's conversion, sums out); then MMAs, copies of K,
// of V, scales
constexpr int kPxSoft = 8, kPxSide = 4;
constexpr int kPxMma = kPxSoft + kPxSide, kPxThreads = 32 * (kPxMma + 4);
constexpr float kPxFar = 64.f;      // how far the denominator's reference may be off (fp32)

// Where the tokens end that block rb of an item sees.
__device__ __forceinline__ int px_end(const PfArgs &a, const PxItem &it, int rb) {
  return it.own ? it.p0 + 1 + (min((rb + 1) * kPxRows, it.rows) - 1) / a.G : it.end;
}
__device__ __forceinline__ int px_tiles(const PfArgs &a, const PxItem &it, int rb) {
  return (px_end(a, it, rb) - it.first + kPxTok - 1) / kPxTok;
}

// Units of one kv head of an item.
__device__ __forceinline__ int64_t px_units(const PfArgs &a, const PxItem &it) {
  if (!it.live) return 0;
  if (!it.own || it.nb == 1) return static_cast<int64_t>(it.nb) * (px_tiles(a, it, 0) + kPxRowCost);
  int64_t u = 0;
  for (int rb = 0; rb < it.nb; ++rb) u += px_tiles(a, it, rb) + kPxRowCost;
  return u;
}

// 64-bit division of numbers that are usually small.
__device__ __forceinline__ int64_t px_div(int64_t x, int64_t y) {
  if (((x | y) >> 31) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
  return x / y;
}

struct PxSeg {
  int b, head, rb;         // b -1: no more segments
  int row0, rows;          // the item's first token row; rows of this block that exist
  int tok, tiles, t_end;   // first token, tiles, where the block's tokens end
  int lim0;                // tokens that the item's first token row sees, each next one more; 0: all see all
  int part, parts;         // the slot of a row of work that CTAs share, and how many share it
  int own, pre;
  int again, more;         // the row of work has earlier, further segments in this CTA (kPxSumTiles)
};

// A producer's way through its CTA's run [u0, u1); every lane of the warp keeps the same.  Where
// it stands: tile or start unit `at` of the row of work (head, rb), which has `tiles`.
struct PxWalk {
  int64_t u, u0, u1, per;
  int i, n, head, rb, tiles, at;
  PxItem it;
};

// in: the unit of item w.i that the run begins with.
__device__ __forceinline__ void px_start(const PfArgs &a, PxWalk &w, int64_t in) {
  w.it = px_load_item(a.items + w.i);
  const int64_t units = px_units(a, w.it);
  w.head = static_cast<int>(px_div(in, units));  // row of work: head major
  int64_t s = in - w.head * units;
  w.rb = 0;
  w.tiles = px_tiles(a, w.it, 0);
  if (!w.it.own) {
    w.rb = static_cast<int>(px_div(s, w.tiles + kPxRowCost));
    s -= static_cast<int64_t>(w.rb) * (w.tiles + kPxRowCost);
  } else {
    while (s >= w.tiles + kPxRowCost) {
      s -= w.tiles + kPxRowCost;
      w.tiles = px_tiles(a, w.it, ++w.rb);
    }
  }
  w.at = static_cast<int>(s);
}

// The next segment; false: the run has ended.  Out of line: two roles call it.
__device__ __noinline__ bool px_next(const PfArgs &a, PxWalk &w, PxSeg &sg) {
  while (w.u < w.u1) {
    if (w.head == a.Hkv) {
      do {
        if (++w.i >= w.n) return false;
        w.it = px_load_item(a.items + w.i);
      } while (!w.it.live || (w.it.own && a.own_split));
      w.head = w.rb = w.at = 0;
      w.tiles = px_tiles(a, w.it, 0);
    }
    // units [0, kPxRowCost) of a row of work stand for its start; tile t is unit kPxRowCost + t
    int span = static_cast<int>(min(static_cast<int64_t>(w.tiles + kPxRowCost - w.at), w.u1 - w.u));
    const int t0 = max(0, w.at - kPxRowCost);
    int take = w.at + span - kPxRowCost - t0;
    const int64_t ut = w.u - w.at + kPxRowCost;  // its first tile
    sg.again = t0 > 0 && w.u > w.u0;
    sg.more = take > kPxSumTiles;
    if (sg.more) {
      span -= take - kPxSumTiles;
      take = kPxSumTiles;
    }
    sg.parts = 1;
    if (ut < w.u0 || ut + w.tiles > w.u0 + w.per)
      sg.parts = static_cast<int>(px_div(ut + w.tiles - 1, w.per) - px_div(ut, w.per)) + 1;
    sg.part = sg.parts == 1 ? -1 : 2 * static_cast<int>(blockIdx.x) + (ut >= w.u0 ? 1 : 0);
    sg.b = w.it.b;
    sg.head = w.head;
    sg.rb = w.rb;
    sg.row0 = w.it.row0;
    sg.rows = min(w.it.rows - w.rb * kPxRows, kPxRows);
    sg.tok = w.it.first + t0 * kPxTok;
    sg.tiles = take;
    sg.t_end = px_end(a, w.it, w.rb);
    sg.lim0 = w.it.own ? w.it.p0 + 1 : 0;
    sg.own = w.it.own;
    sg.pre = w.it.pre;
    w.u += span;
    w.at += span;
    if (w.at == w.tiles + kPxRowCost) {
      w.at = 0;
      if (++w.rb == w.it.nb) {
        w.rb = 0;
        ++w.head;
      }
      if (w.it.nb > 1) w.tiles = px_tiles(a, w.it, w.rb);
    }
    if (take > 0) return true;
  }
  return false;
}

// ---------------------------------------------------------------------------
// shared memory and tcgen05
// ---------------------------------------------------------------------------

// Barriers, those that expect as many arrivals together: 1, 4, 12, 14.
enum : int {
  kKFull = 0,
  kKEmpty = kKFull + kPxK,
  kVFull = kKEmpty + kPxK,
  kScFull = kVFull + kPxV,
  kScEmpty = kScFull + kPxScales,
  kSegFull = kScEmpty + kPxScales,
  kQFree = kSegFull + kPxSegs,
  kSFull = kQFree + 2,
  kHEmpty = kSFull + 2,
  kODone = kHEmpty + 2,
  kDrain,
  kRef,  // [group][quarter of the rows]
  kVEmpty = kRef + 8,  // four warps each from here
  kQFull = kVEmpty + kPxV,
  kQReady = kQFull + 2,
  kHFull = kQReady + kPxStats,
  kOFree = kHFull + 2,
  kPHalf,  // a group's weights for the first 64 tokens of a tile
  // All of a tile's weights.  Four in turn: the scores two tiles on come once a tile's first half is there, so
  // that a warp that is ahead (one without rows has nothing else to wait for) ends the group's next tile while
  // another is still at this one.  On one barrier a group its second arrival stood for the other's, and scores
  // were taken for weights.  The scores four tiles on come behind all arrivals for this tile.
  kPFull = kPHalf + 2,
  kStatFull = kPFull + 4,  // softmax and sides
  kSegEmpty = kStatFull + kPxStats,  // everybody but the copies
  kBars = kSegEmpty + kPxSegs
};

__device__ __forceinline__ int px_arrivals(int bar) {
  return bar < kVEmpty ? 1 : bar < kStatFull ? 4 : bar < kSegEmpty ? kPxSoft + kPxSide : kPxMma + 2;
}

struct PxCtl {
  float4 sc[kPxScales][kPxTok / 16];  // of a tile's blocks: K scale; V scale's fraction times 2^7, exponent
  float4 end[kPxStats][2][kPxRows];   // [segment][group]: m that its l stands on, l, n, -
  float2 now[2][kPxRows];             // [group]: (m, n), a row's references
  float qk[kPxStats][kPxRows];
  unsigned long long nan_from[kPxStats][128];  // per dim: px_nan of a token with a NaN code that some row
                                               // does not see, the first of the last segment that had one
  uint64_t bar[kBars];
  int64_t run_in;                     // where the CTA's run begins: unit of item run_i
  int run_i;
  int nan_seg[kPxStats];              // 1 + the last segment that had one
  int come[kPxStats][2];              // [segment][group]: tiles of the segment up to the group's last
  int bad[kPxScales];                 // first token of a page outside the pool, or INT_MAX
  PxSeg seg[kPxSegs];
  uint32_t tmem;
  int fail;
};

// A later segment's is smaller than an earlier one's, so that nothing needs to be cleared.
__device__ __forceinline__ unsigned long long px_nan(uint32_t seg, int tok) {
  return (static_cast<unsigned long long>(~seg) << 32) | static_cast<uint32_t>(tok);
}

// TMEM columns: scores, a ring of five halves of a tile (64 tokens), from 0 on; q; sums.
constexpr uint32_t kPxQ = 320, kPxO = 384;
template <int D>
constexpr int kPxQs = 128 / D;  // segments' q
__device__ __forceinline__ uint32_t px_scol(uint32_t g, int half) { return 64 * ((2 * g + half) % 5); }


template <int D>
struct PxSmem {
  static constexpr int kTile = kPxTok * D;      // a tile of K or V
  static constexpr int kHalf = 2 * kTile;       // V in f16
  static constexpr int k = 0, v = kPxK * kTile, h = v + kPxV * kTile, ctl = h + 2 * kHalf;
  static constexpr size_t bytes = ctl + sizeof(PxCtl) + 1024;
  static_assert(bytes <= 227 * 1024 && ctl % 16 == 0, "shared memory of a CTA");
};

// Barriers by their shared-memory address.
// A try sleeps until the phase ends, for up to a millisecond (left to its own, it comes back after a short
// time, and the waiting warps' polls were a fifth of all instructions).
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity), "r"(1000000)
      : "memory");
  return done != 0;
}

__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void bar_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// A whole warp waits, bounded.  The wait itself is out of line: inlined at each place, with the schedule's
// walk, the kernel was 173 KB of code for five roles at once, and instruction fetches were its bound.
__device__ __noinline__ bool px_wait_long(int *fail, uint32_t bar, uint32_t parity, uint32_t *err_word) {
  bool ok = false;
  if (!*reinterpret_cast<volatile int *>(fail)) {
    const long long t0 = clock64();
    for (uint32_t i = 0; i < kWaitPolls; ++i) {
      ok = bar_try(bar, parity);
      if (ok || clock64() - t0 > kWaitCycles) break;
    }
    if (!ok && atomicExch(fail, 1) == 0) report(err_word, KVQ_ERRBIT_TIMEOUT);
  }
  return __all_sync(0xffffffffu, ok);
}

// Whether a phase is over, without waiting for it.
__device__ __forceinline__ uint32_t bar_test(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done;
}

// Rows of D bytes: for 64 a 64-byte swizzle, 8-row groups 512 bytes apart.
template <int D>
__device__ __forceinline__ uint64_t px_kdesc(uint32_t addr) {
  if (D == 128) return tc_desc(addr);
  return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) | (1ull << 16) | (32ull << 32) | (1ull << 46) | (4ull << 61);
}

// V in f16, tokens by dims, dims contiguous: 64 dims a row of 128 bytes, 128-byte swizzle;
// 8 tokens 1,024 bytes apart, the other 64 dims 16 KB.
__device__ __forceinline__ uint64_t px_vdesc(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) | (1024ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

// fp32 += A (TMEM, 128 rows) * B (shared memory, n columns)
__device__ __forceinline__ void px_mma8(uint32_t d, uint32_t a, uint64_t b, uint32_t n, bool e5m2, bool add) {
  const uint32_t idesc = (1u << 4) | ((e5m2 ? 1u : 0u) << 7) | ((n >> 3) << 17) | ((128u >> 4) << 24);
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(add ? 1 : 0)
      : "memory");
}

// the same, f16 by f16, B with its columns contiguous (bit 16)
__device__ __forceinline__ void px_mma16(uint32_t d, uint32_t a, uint64_t b, uint32_t n, bool add) {
  const uint32_t idesc = (1u << 4) | (1u << 16) | ((n >> 3) << 17) | ((128u >> 4) << 24);
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(add ? 1 : 0)
      : "memory");
}

// 32 consecutive columns of this warp's lanes, loaded and waited for in one statement, so that no use
// moves between.
__device__ __forceinline__ void tc_ld32(float (&v)[32], uint32_t addr) {
  uint32_t *r = reinterpret_cast<uint32_t *>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}

__device__ __forceinline__ void tc_st32(uint32_t addr, const float (&v)[32]) {
  const uint32_t *r = reinterpret_cast<const uint32_t *>(v);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(addr)
      : "memory");
}

__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}

__device__ __forceinline__ void tc_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ---------------------------------------------------------------------------
// q's pieces
// ---------------------------------------------------------------------------

constexpr int kPxQThreads = 1024;

// Exclusive scan of v over the CTA; *total = the sum.
__device__ __forceinline__ int64_t px_scan(int64_t v, int64_t *warps, int64_t *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  __syncthreads();  // the scratch may be read
  if (lane == 31) warps[warp] = incl;
  __syncthreads();
  int64_t w = warps[lane], wi = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, wi, o);
    if (lane >= o) wi += u;
  }
  *total = __shfl_sync(0xffffffffu, wi, 31);
  return __shfl_sync(0xffffffffu, wi - w, warp) + incl - v;
}

// One CTA: the items with work, or with rows to be zeroed, and the units before each.  (Worked out by
// every CTA of the next kernel for itself, as kvq_block_attn does, it took them 6.4 us: groups make a
// request three dependent reads, and the code is long.)  A group's first request that takes part is looked
// for by one thread, 0.3 us a request: 1,024 slots of which the last 64 take part make a call of 354 us.
__device__ __forceinline__ void px_plan(const PfArgs &a, int ctas) {
  __shared__ int64_t warps[32];
  bool order = true;
  for (int g = threadIdx.x; g < a.n_groups; g += kPxQThreads) order &= pf_group_ok(a, g);
  order = __syncthreads_and(order);
  if (!order && threadIdx.x == 0) report(a.err_word, KVQ_ERRBIT_REQ);
  const int groups = order ? a.n_groups : 0, all = groups + a.rg.B;
  const int64_t room = 2 * static_cast<int64_t>(a.rg.n_tokens);
  int64_t units = 0, count = 0;
  int n_grp = 0;
  // groups' items, then requests', in one list (in rounds of their own they cost a chain of loads each:
  // 40 requests of five groups took 1.6 us more)
  for (int i0 = 0; i0 < all; i0 += kPxQThreads) {
    const int i = i0 + threadIdx.x;
    const bool grp = i < groups;
    PxItem o = {};
    bool has = false;
    if (grp) {
      const int s = __ldg(a.group_start + i), e = __ldg(a.group_start + i + 1);
      const int pages = __ldg(a.prefix_pages + i);
      if (s < e && pages > 0 && pages <= a.MP) {
        const int2 r = pf_group_rows(a, i);
        o.row0 = r.x;
        o.n = r.y - r.x;
        o.end = pages << a.p_shift;
        for (o.b = s; o.n > 0 && o.b < e; ++o.b)
          if (pf_request(a, o.b).live) {
            o.live = has = true;
            break;
          }
      }
    } else if (i < all) {
      o.b = i - groups;
      PfReq q;
      if (order) {
        q = pf_request(a, o.b);
      } else {
        q.r = request_rows<true>(a.rg, o.b);
        q.pre = 0;
        q.group = -1;
        q.live = false;
      }
      if (q.r.err) report(a.err_word, q.r.err);
      has = q.r.n > 0;
      o.row0 = q.r.row;
      o.n = q.r.n;
      o.p0 = q.r.p0;
      o.first = q.pre;
      o.end = q.r.p0 + q.r.n;
      o.own = 1;
      o.pre = q.pre > 0;
      o.live = q.live;
      o.row_pre = q.live && q.pre > 0 ? pf_group_rows(a, q.group).x : 0;
    }
    o.rows = o.n * a.G;
    o.nb = (o.rows + kPxRows - 1) / kPxRows;
    const int64_t u = has && (grp || !a.own_split) ? px_units(a, o) * a.Hkv : 0;
    int64_t n_all, u_all;
    const int64_t at = count + px_scan(has, warps, &n_all);
    const int64_t before = units + px_scan(u, warps, &u_all);
    if (has && at < room) a.items[at] = o;
    if (has && at <= room) a.units[at] = before;
    if (has && at >= room) report(a.err_word, KVQ_ERRBIT_REQ);  // requests that own the same rows
    count += n_all;
    units += u_all;
    if (i0 < groups) n_grp += __syncthreads_count(has && grp);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    const int64_t n = min(count, room), total = count > room ? a.units[room] : units;
    a.units[n] = total;
    a.plan->total = total;
    a.plan->per = max(static_cast<int64_t>(1), px_div(total + ctas - 1, ctas));
    a.plan->n_grp = min(n_grp, static_cast<int>(n));
    a.plan->n_req = max(static_cast<int>(n) - n_grp, 0);
  }
}

// Block 0 makes the plan.  The others: four dims a lane; each row scaled by 2^e, its largest value into
// [224, 448], and split into an e4m3 and an e5m2 piece (tc_q_pieces).  Done once a call, since every
// CTA that works on a part of a row's tokens needs them.
template <int D>
__global__ void __launch_bounds__(kPxQThreads) prefix_plan_kernel(PfArgs a, int ctas) {
  grid_dependency_wait();
  allow_dependents();
  if (blockIdx.x == 0) {
    px_plan(a, ctas);
    return;
  }
  const int64_t idx = (static_cast<int64_t>(blockIdx.x - 1) * kPxQThreads + threadIdx.x) / (D / 4);  // (token, head)
  const int part = threadIdx.x % (D / 4);
  const bool has = idx < static_cast<int64_t>(a.rg.n_tokens) * a.Hq;
  float x[4] = {0.f, 0.f, 0.f, 0.f};
  if (has) {
    const int64_t t = idx / a.Hq, h = idx - t * a.Hq;
    const uint2 w = __ldg(reinterpret_cast<const uint2 *>(a.q + t * a.q_stride + h * D + 4 * part));
    bf16x2_to_f32(w.x, x);
    bf16x2_to_f32(w.y, x + 2);
  }
  float mx = 0.f;
  bool odd = false;  // inf or NaN: the row's scores are NaN, as inf - inf would make them
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    mx = fmaxf(mx, finite_abs(x[k]));
    odd |= !(fabsf(x[k]) < INFINITY);
  }
#pragma unroll
  for (int o = 1; o < D / 4; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if (!has) return;
  const int e = block_exponent(mx);
  // a negative sm_scale's sign goes to q, so that a larger score is a larger product
  const float up = copysignf(pow2(-e), a.q_scale), nan = odd ? NAN : 0.f;
  uint32_t c1 = 0, c2 = 0;
  tc_q_pieces(x[0] * up + nan, x[1] * up + nan, 0, c1, c2);
  tc_q_pieces(x[2] * up + nan, x[3] * up + nan, 16, c1, c2);
  uint32_t *to = reinterpret_cast<uint32_t *>(a.qp + idx * (2 * D)) + part;
  to[0] = c1;
  to[D / 4] = c2;
  if (part == 0) a.qk[idx] = fabsf(a.q_scale) * pow2(e);
}

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------

// A segment's q into TMEM, a row a lane: D / 4 columns of each piece.
template <int D>
__device__ __forceinline__ void px_load_q(const PfArgs &a, const PxSeg &sg, uint32_t cols, float *qk, int r) {
  const int row = sg.rb * kPxRows + r, i = row / a.G;
  const int64_t at = (static_cast<int64_t>(sg.row0) + i) * a.Hq + sg.head * a.G + row - i * a.G;
  const bool has = r < sg.rows;
  const uint4 *p = reinterpret_cast<const uint4 *>(a.qp + (has ? at : 0) * (2 * D));
#pragma unroll
  for (int c = 0; c < 2 * D / 64; ++c) {
    float w[16];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint4 x = has ? __ldcg(p + 4 * c + j) : make_uint4(0, 0, 0, 0);
      w[4 * j] = __uint_as_float(x.x);
      w[4 * j + 1] = __uint_as_float(x.y);
      w[4 * j + 2] = __uint_as_float(x.z);
      w[4 * j + 3] = __uint_as_float(x.w);
    }
    tc_st16(cols + 16 * c, w);
  }
  qk[r] = has ? __ldcg(a.qk + at) : 0.f;
}

// Chunk j (16 codes) of a row of a tile as the copy left it.
template <int D>
__device__ __forceinline__ const uint8_t *px_codes(const uint8_t *v, int row, int j) {
  return D == 128 ? v + row * 128 + ((j ^ (row & 7)) * 16) : v + row * 64 + ((j ^ ((row >> 1) & 3)) * 16);
}

// The same in f16: 64 dims a row of 128 bytes.
template <int D>
__device__ __forceinline__ void px_store_half(uint8_t *h, int row, int j, uint4 w) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
  uint32_t o[8];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    o[2 * q] = e4m3x2_to_f16x2(static_cast<uint16_t>(x[q] & 0xFFFFu));
    o[2 * q + 1] = e4m3x2_to_f16x2(static_cast<uint16_t>(x[q] >> 16));
  }
  const int c = (2 * j) & 7;
  uint8_t *to = h + (D == 128 && j >= 4 ? 16384 : 0) + row * 128;
  *reinterpret_cast<uint4 *>(to + ((c ^ (row & 7)) * 16)) = make_uint4(o[0], o[1], o[2], o[3]);
  *reinterpret_cast<uint4 *>(to + (((c + 1) ^ (row & 7)) * 16)) = make_uint4(o[4], o[5], o[6], o[7]);
}

// A chunk of 32 tokens of a row's scores: the maxima of x and of x + log2 vs.
__device__ __forceinline__ void px_max(const float (&x)[32], const float4 *sc, float qk, float &mx, float &mv) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float4 b = sc[h];
    const float *y = x + 16 * h;
    const float u0 = max3(y[0], y[1], y[2]), u1 = max3(y[3], y[4], y[5]), u2 = max3(y[6], y[7], y[8]);
    const float u3 = max3(y[9], y[10], y[11]), u4 = max3(y[12], y[13], y[14]);
    const float z = max3(max3(u0, u1, u2), fmaxf(u3, y[15]), u4) * (qk * b.x);  // (0 times -inf: no maximum)
    mx = fmaxf(mx, z);
    mv = fmaxf(mv, z + b.z);
  }
}

// Its weights: e = 2^(x - m) for the sum l, and e vs 2^(m - n) 2^7 in f16.
template <bool kMasked>
__device__ __forceinline__ void px_weights(const float (&x)[32], const float4 *sc, float qk, float m, float mn,
                                           float2 (&l)[2], float (&p)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float4 b = sc[h];
    const float f = qk * b.x, d = b.y * fast_exp2(fminf(mn + b.z, 112.f));
#pragma unroll
    for (int j = 0; j < 16; j += 2) {
      float2 y = make_float2(x[16 * h + j], x[16 * h + j + 1]);
      y = __ffma2_rn(y, make_float2(f, f), make_float2(-m, -m));
      if (kMasked) {  // (0 times -inf is no score)
        if (x[16 * h + j] == -INFINITY) y.x = -INFINITY;
        if (x[16 * h + j + 1] == -INFINITY) y.y = -INFINITY;
      }
      const float2 e = make_float2(fast_exp2(y.x), fast_exp2(y.y));
      l[h] = __fadd2_rn(l[h], e);
      const float2 w = __fmul2_rn(e, make_float2(d, d));
      p[8 * h + j / 2] = __uint_as_float(f32x2_to_f16x2(w.x, w.y));
    }
  }
}

__device__ __forceinline__ void px_mask(float (&x)[32], int see) {
#pragma unroll
  for (int j = 0; j < 32; ++j)
    if (j >= see) x[j] = -INFINITY;
}

// A further segment of a row of work (kPxSumTiles): its sums O and statistics (m, l, n) are added to what lies
// in `to`, which this lane wrote, or with `out` the joined row is written.  The joined statistics.  Out of line,
// since segments that long are few: within the sides' loop it took 256 requests behind 32k from 314 to 329 us.
template <int D>
__device__ __noinline__ float4 px_join(uint32_t o_addr, float *to, float4 s, bool has, uint16_t *out) {
  float4 was = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
  if (has) was = *reinterpret_cast<const float4 *>(to + D);
  const float M = fmaxf(was.x, s.x), N = fmaxf(was.z, s.z);
  const bool bad = was.y < 0.f || s.y < 0.f;
  // who saw nothing (l = 0) has no maximum and no weight
  const float x = was.y == 0.f ? 0.f : exp2f(was.z - N), y = s.y == 0.f ? 0.f : exp2f(s.z - N);
  const float l = bad ? -1.f
                      : (was.y == 0.f ? 0.f : was.y * exp2f(was.x - M)) + (s.y == 0.f ? 0.f : s.y * exp2f(s.x - M));
  const float2 f = bad ? make_float2(0.f, 0.f) : out_scale(N - M - 7.f, l);
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    float o[32];
    tc_ld32(o, o_addr + c);
    if (!has) continue;
    uint4 w[4];
    uint32_t *u = reinterpret_cast<uint32_t *>(w);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float4 v = *reinterpret_cast<const float4 *>(to + c + 4 * j);
      v = make_float4(v.x * x + o[4 * j] * y, v.y * x + o[4 * j + 1] * y, v.z * x + o[4 * j + 2] * y,
                      v.w * x + o[4 * j + 3] * y);
      if (!out) *reinterpret_cast<float4 *>(to + c + 4 * j) = v;
      u[2 * j] = bad ? 0u : pack_bf16x2(v.x * f.x * f.y, v.y * f.x * f.y);
      u[2 * j + 1] = bad ? 0u : pack_bf16x2(v.z * f.x * f.y, v.w * f.x * f.y);
    }
    if (out)
#pragma unroll
      for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4 *>(out + c + 8 * j) = w[j];
  }
  if (has) *reinterpret_cast<float4 *>(to + D) = make_float4(M, l, N, out ? kDone : kHere);
  return make_float4(M, l, N, 0.f);
}

// One CTA an SM, each with its run of tiles; a tile passes, in turn,
//   copies (a warp each for K and V, rings of four tiles; a warp for scales, eight tiles ahead),
//   the MMA warp: S = q K^T into TMEM,
//   a group of four softmax warps, a row a thread: maximum, references, weights into S's own columns in
//     f16; tiles alternate between two groups, which hand the references on before they make the weights,
//   the MMA warp: O += P V,
// and beside them four side warps turn V's codes into f16, bring q in and take finished sums out.  A row a
// thread: with two (16 softmax warps of 80 registers, which exchange their maxima) 256 requests behind 32k take 326
// us, and 316 with one.
template <int D>
__global__ void __launch_bounds__(kPxThreads, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, PfArgs a) {
  using S = PxSmem<D>;
  constexpr int RF = D + kStat;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  PxCtl &ctl = *reinterpret_cast<PxCtl *>(smem + S::ctl);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bars = smem_addr(ctl.bar);
  auto bar = [&](int i) -> uint32_t { return bars + 8u * i; };
  auto wait = [&](int i, uint32_t parity) -> bool {
    if (__all_sync(0xffffffffu, bar_try(bars + 8u * i, parity))) return true;
    return px_wait_long(&ctl.fail, bars + 8u * i, parity, a.err_word);
  };
  auto test = [&](int i, uint32_t parity) { return bar_test(bars + 8u * i, parity); };  // (a lane's)
  if (threadIdx.x < kBars) {
    const int i = threadIdx.x;
    mbar_init(&ctl.bar[i], px_arrivals(i));
    fence_barrier_init();
  }
  if (threadIdx.x < kPxStats) ctl.nan_seg[threadIdx.x] = 0;
  if (threadIdx.x == 0) {
    ctl.fail = 0;
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&kmap)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&vmap)) : "memory");
  }
  for (int i = threadIdx.x; i < kPxStats * 128; i += kPxThreads) ctl.nan_from[0][i] = ~0ull;
  if (warp == kPxMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&ctl.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  grid_dependency_wait();  // the plan and q's pieces
  allow_dependents();
  const int64_t per = __ldcg(&a.plan->per), total = __ldcg(&a.plan->total);
  const int n_items = __ldcg(&a.plan->n_grp) + __ldcg(&a.plan->n_req);
  const int64_t u0 = blockIdx.x * per, u1 = min(u0 + per, total);
  if (u0 < u1)
    for (int i = threadIdx.x; i < n_items; i += kPxThreads) {
      const int64_t lo = __ldcg(a.units + i), hi = __ldcg(a.units + i + 1);
      if (lo <= u0 && u0 < hi) {
        ctl.run_i = i;
        ctl.run_in = u0 - lo;
      }
    }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = ctl.tmem;

  if (warp == kPxMma + 3) {
    // --------------------------------------------- scales, four tiles at a time
    uint32_t g = 0;
    bool ok = true;
    for (uint32_t k = 0; ok; ++k) {
      const int ss = k % kPxSegs;
      ok = wait(kSegFull + ss, (k / kPxSegs) & 1);
      if (!ok) break;
      const PxSeg sg = ctl.seg[ss];
      if (sg.b < 0) break;
      const int32_t *bt = a.block_table + static_cast<int64_t>(sg.b) * a.MP;
      for (int t0 = 0; ok && t0 < sg.tiles; t0 += 4) {
        const int mine = t0 + (lane >> 3), tok = sg.tok + mine * kPxTok + 16 * (lane & 7);
        const bool needed = mine < sg.tiles && tok < sg.t_end;
        const int page = needed ? __ldg(bt + (tok >> a.p_shift)) : -1;
        const bool good = page >= 0 && page < a.num_pages;
        // tokens without a page are masked
        const float2 x = good ? __ldg(a.scales + static_cast<int64_t>(page) * a.Hkv + sg.head) : make_float2(1.f, 1.f);
        const float2 vs = split_scale(x.y);
        const uint32_t bads = __ballot_sync(0xffffffffu, needed && !good);
#pragma unroll 1
        for (int j = 0; ok && j < 4 && t0 + j < sg.tiles; ++j, ++g) {
          const int cs = g % kPxScales;
          ok = wait(kScEmpty + cs, ((g / kPxScales) & 1) ^ 1);
          if (!ok) break;
          // the weights' operand: kPScale (2^7), so that the largest sit high in f16's range
          if (lane >> 3 == j) ctl.sc[cs][lane & 7] = make_float4(x.x, vs.x * kPScale, vs.y, 0.f);
          if (lane == 0) {
            const uint32_t bad = bads >> (8 * j) & 0xFFu;
            ctl.bad[cs] = bad ? sg.tok + (t0 + j) * kPxTok + 16 * (__ffs(bad) - 1) : INT_MAX;
          }
          __syncwarp();
          if (lane == 0) bar_arrive(bar(kScFull + cs));
        }
      }
      __syncwarp();
      if (ok && lane == 0) bar_arrive(bar(kSegEmpty + ss));
    }
  } else if (warp > kPxMma) {
    // ------------------------------------------------------- producers: K, then V
    const int is_v = warp - kPxMma - 1;
    const CUtensorMap *map = is_v ? &vmap : &kmap;
    const int full = is_v ? kVFull : kKFull, empty = is_v ? kVEmpty : kKEmpty;
    uint8_t *tiles_at = smem + (is_v ? S::v : S::k);
    const uint32_t stages = is_v ? kPxV : kPxK;
    uint64_t again;  // a prefix is read by several row blocks and CTAs
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(again));
    const uint64_t once = policy_evict_first();
    const int pages_tile = kPxTok >> a.p_shift;  // a tile begins with a page
    const uint32_t page_bytes = static_cast<uint32_t>(D) << a.p_shift;
    uint32_t g = 0, nseg = 0, par = 1, slot = 0;
    bool ok = true;
    PxWalk walk = {u0, u0, u1, per, ctl.run_i, n_items, 0, 0, 0, 0, {}};
    if (u0 < u1) px_start(a, walk, ctl.run_in);
    PxSeg sg;
    while (ok && px_next(a, walk, sg)) {
      const int ss = nseg % kPxSegs;
      if (!is_v) {
        if (nseg >= kPxSegs) ok = wait(kSegEmpty + ss, ((nseg / kPxSegs) - 1) & 1);
        if (!ok) break;
        if (lane == 0) {
          ctl.seg[ss] = sg;
          bar_arrive(bar(kSegFull + ss));
        }
      }
      ++nseg;
      const int32_t *bt = a.block_table + static_cast<int64_t>(sg.b) * a.MP;
      for (int t = 0; t < sg.tiles; ++t) {
        const int tok = sg.tok + t * kPxTok;
        // lane j: page j of the tile
        const int lp = (tok >> a.p_shift) + lane;
        const bool needed = lane < pages_tile && static_cast<int64_t>(lp) << a.p_shift < sg.t_end;
        const int page = needed ? __ldg(bt + lp) : 0;
        const bool good = needed && page >= 0 && page < a.num_pages;
        const uint32_t goods = __ballot_sync(0xffffffffu, good), needs = __ballot_sync(0xffffffffu, needed);
        ok = wait(empty + slot, par);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&ctl.bar[full + slot], static_cast<uint32_t>(__popc(goods)) * page_bytes);
        __syncwarp();
        int pages[kPxTok / 16];
#pragma unroll
        for (int j = 0; j < kPxTok / 16; ++j) pages[j] = __shfl_sync(0xffffffffu, page, j);
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < kPxTok / 16; ++j)
            if (goods >> j & 1)
              tma_load_4d(tiles_at + slot * S::kTile + j * page_bytes, map, 0, 0, sg.head, pages[j], &ctl.bar[full + slot],
                          sg.own ? once : again);
        }
        __syncwarp();
        if (!is_v && lane == 0 && needs != goods) report(a.err_word, KVQ_ERRBIT_PAGE);
        ++g;
        if (++slot == stages) {
          slot = 0;
          par ^= 1;
        }
        __syncwarp();
      }
    }
    if (ok && !is_v) {  // nothing more
      const int ss = nseg % kPxSegs;
      if (nseg >= kPxSegs) ok = wait(kSegEmpty + ss, ((nseg / kPxSegs) - 1) & 1);
      if (ok && lane == 0) {
        ctl.seg[ss].b = -1;
        bar_arrive(bar(kSegFull + ss));
      }
    }
    if (*reinterpret_cast<volatile int *>(&ctl.fail) && lane == 0)
      for (uint32_t k = g > stages ? g - stages : 0; k < g; ++k) mbar_wait(&ctl.bar[full + k % stages], (k / stages) & 1);
  } else if (warp == kPxMma) {
    // ------------------------------------------------------------- MMA issue
    // Scores run two tiles ahead of values, into the next segment too.  S(t + 2) takes the columns of the
    // second half of S(t - 1) and of the first of S(t), whose weights the products issued before it read
    // there: it is made while the softmax ends the weights of t.
    const uint32_t k_a = smem_addr(smem + S::k), h_a = smem_addr(smem + S::h);
    uint32_t ks = 0, ps = 0;  // segments of the scores' and of the values' cursor
    int kt = 0, pt = 0;       // tiles in them
    uint32_t kg = 0, pg = 0;  // tiles so far
    int k_tiles = 0, k_len = 0, p_tiles = 0, p_len = 0;  // their segments' tiles and tokens
    bool ok = true, k_in = false, p_in = false, k_end = false;
    auto tokens = [](int len, int t) {  // of a tile, in whole chunks of 32
      return min(kPxTok, (len - t * kPxTok + 31) & ~31);
    };
    // the scores' next segment; not if it is not there, unless `must`
    auto next = [&](bool must) {
      const int ss = ks % kPxSegs, qs = ks % kPxQs<D>;
      const uint32_t sp = (ks / kPxSegs) & 1, qp = (ks / kPxQs<D>) & 1;
      if (!must && !__all_sync(0xffffffffu, test(kSegFull + ss, sp))) return false;
      if (!(ok = wait(kSegFull + ss, sp))) return false;
      const PxSeg &sg = ctl.seg[ss];
      k_tiles = sg.tiles;
      k_len = sg.t_end - sg.tok;
      if (sg.b < 0) {
        k_end = true;
        return false;
      }
      if (!must && !__all_sync(0xffffffffu, test(kQFull + qs, qp))) return false;
      if (!(ok = wait(kQFull + qs, qp))) return false;
      kt = 0;
      return k_in = true;
    };
    // Each turn: the first half of a tile's values, then the scores two tiles on, if they can be, then the other
    // half; scores alone where they are not that far ahead.
    while (ok) {
      const bool more = !k_end && (k_in || next(kg == pg));  // the next scores' segment is here
      if (!ok || (!more && kg == pg)) break;
      const bool pv = kg - pg == 2 || !more;
      const int buf = pg & 1, slot = kg % kPxK;
      const uint32_t par = (pg >> 1) & 1, kpar = (kg / kPxK) & 1;
      if (pv && !p_in) {
        const PxSeg &sg = ctl.seg[ps % kPxSegs];  // (its scores have been issued)
        p_tiles = sg.tiles;
        p_len = sg.t_end - sg.tok;
        p_in = true;
        pt = 0;
        ok = ps == 0 || wait(kOFree, (ps - 1) & 1);
        if (!ok) break;
      }
      {  // a round trip is some 150 cycles beside the tiles' traffic: the tests go out together
        const int kb = more ? kKFull + slot : kHFull + buf, vb = pv ? kHFull + buf : kb;
        const uint32_t kp = more ? kpar : par, vp = pv ? par : kp;
        const int hb = pv ? kPHalf + buf : kb;
        const uint32_t hp = pv ? par : kp;
        const uint32_t x = test(kb, kp), y = test(vb, vp), z = test(hb, hp);
        ok = __all_sync(0xffffffffu, x & y & z) || (wait(kb, kp) && wait(vb, vp) && wait(hb, hp));
      }
      if (!ok) break;
      tc_after();
      // 16 tokens a step: 8 columns of P, 16 rows of V
      const int steps = tokens(p_len, pt) / 16;
      const uint64_t vd = px_vdesc(h_a + buf * S::kHalf);
      auto values = [&](int half) {
        const uint32_t p = tmem + px_scol(pg, half);
        const uint64_t rows = vd + half * (64 * 128 >> 4);
        const int n = min(steps - 4 * half, 4);
        if (elect_one())
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (k < n)
              px_mma16(tmem + kPxO, p + 32 * (k >> 1) + 8 * (k & 1), rows + k * (16 * 128 >> 4), D, pt + half + k > 0);
        __syncwarp();
      };
      if (pv) values(0);
      if (more) {
        const int n = tokens(k_len, kt), qs = ks % kPxQs<D>;
        const uint32_t q = tmem + kPxQ + qs * (D / 2);
        uint32_t to = px_scol(kg, 0);
        // at the ring's end in two (half a tile's product takes 0.65 of a whole one's: one tile in five)
        const int wide = to == 256 ? 64 : kPxTok;
#pragma unroll 1
        for (int at = 0; at < n; at += wide, to = 0) {
          const uint64_t kd = px_kdesc<D>(k_a + slot * S::kTile) + (at * D >> 4);
          const int cols = min(n - at, wide);
          if (elect_one())
#pragma unroll
            for (int piece = 1; piece >= 0; --piece)  // the smaller first: each sum is truncated
#pragma unroll
              for (int k = 0; k < D / 32; ++k)
                px_mma8(tmem + to, q + piece * (D / 4) + 8 * k, kd + 2 * k, cols, piece == 1, piece == 0 || k > 0);
          __syncwarp();
        }
        const bool last = kt + 1 == k_tiles;
        if (elect_one()) {
          bar_commit(bar(kSFull + (kg & 1)));
          bar_commit(bar(kKEmpty + slot));
        }
        __syncwarp();
        // (a condition within the elected lane's block lost the commit: it stands around the election)
        if (last && elect_one()) bar_commit(bar(kQFree + qs));
        __syncwarp();
        ++kg;
        ++kt;
        if (last) {
          k_in = false;
          ++ks;
        }
      }
      if (!pv) continue;
      ok = wait(kPFull + (pg & 3), (pg >> 2) & 1);
      if (!ok) break;
      tc_after();
      values(1);
      const bool last = pt + 1 == p_tiles;
      if (elect_one()) bar_commit(bar(kHEmpty + buf));
      __syncwarp();
      if (last && elect_one()) bar_commit(bar(kODone));
      if (lane == 0) bar_arrive(bar(kScEmpty + pg % kPxScales));
      __syncwarp();
      ++pg;
      ++pt;
      if (last) {
        if (lane == 0) bar_arrive(bar(kSegEmpty + ps % kPxSegs));
        p_in = false;
        ++ps;
      }
    }
    if (*reinterpret_cast<volatile int *>(&ctl.fail)) {
      // the products in flight end before the CTA's memory goes to another one
      if (elect_one()) bar_commit(bar(kDrain));
      mbar_wait(&ctl.bar[kDrain], 0);
    }
  } else if (warp >= kPxSoft) {
    // ---------- sides: q in; V from e4m3 to f16; sums out, to the output or to where the merge finds them
    const int quad = warp & 3, r = 32 * quad + lane;
    const uint32_t lanes = static_cast<uint32_t>(32 * quad) << 16;
    // This lane's chunk of 16 codes, and rows, kR apart.  With head_dim 128 the lanes of the upper 64 dims
    // take the neighbouring row, so that the eight lanes of a store's phase meet eight groups of banks.
    constexpr int kC = D / 16, kR = 32 / kC;
    const int chunk = lane % kC, row0 = (32 * quad + lane / kC) ^ (D == 128 ? chunk >> 2 : 0);
    auto px_put = [&](uint32_t k) -> bool {  // segment k's sums
      const int ss = k % kPxSegs, ks = k % kPxStats;
      const PxSeg &sg = ctl.seg[ss];
      if (!wait(kStatFull + ks, (k / kPxStats) & 1) || !wait(kODone, k & 1)) return false;
      tc_after();
      if (32 * quad < sg.rows) {
        const int row = sg.rb * kPxRows + r, i = row / a.G;
        const int fin = ctl.come[ks][1] > ctl.come[ks][0];  // who had the last tile
        const float4 e0 = ctl.end[ks][fin][r], e1 = ctl.end[ks][fin ^ 1][r];
        const float M = e0.x, N = e0.z;
        bool bad = e0.y < 0.f || e1.y < 0.f;
        float l = e0.y;
        if (e1.y != 0.f) l += e1.y * exp2f(e1.x - M);
        const bool whole = sg.part < 0 && sg.own && !sg.pre && !sg.more;  // nothing to be merged with
        const int64_t at = (static_cast<int64_t>(sg.row0) + i) * a.Hq + sg.head * a.G + row - i * a.G;
        float *here = a.rows + (static_cast<int64_t>(sg.own) * a.rg.n_tokens * a.Hq + at) * RF;
        float *to = sg.part < 0 ? here : a.cut + (static_cast<int64_t>(sg.part) * kPxRows + r) * RF;
        const bool has = r < sg.rows;
        if (bad) l = -1.f;
        if (sg.again) {
          const float4 all = px_join<D>(tmem + lanes + kPxO, to, make_float4(M, l, N, 0.f), has, whole ? a.out + at * D : nullptr);
          bad = all.y < 0.f;
        }
        if (has && !sg.again) {
          *reinterpret_cast<float4 *>(to + D) = make_float4(M, l, N, whole ? kDone : kHere);
          if (sg.part >= 0 && (sg.part & 1))  // the first part: where the others are
            *reinterpret_cast<float4 *>(here + D) =
                make_float4(__int_as_float(sg.part >> 1), __int_as_float(sg.parts), 0.f, kCut);
        }
        float2 f = make_float2(1.f, 1.f);
        if (whole) f = bad ? make_float2(0.f, 0.f) : out_scale(N - M - 7.f, l);
        const bool nan = ctl.nan_seg[ks] == static_cast<int>(k) + 1;
        const int lim = sg.lim0 ? sg.lim0 + i : INT_MAX;
#pragma unroll 1
        for (int c = sg.again ? D : 0; c < D; c += 32) {
          float o[32];
          tc_ld32(o, tmem + lanes + kPxO + c);
          if (!has) continue;
          if (whole) {
            uint4 w[4];
            uint32_t *u = reinterpret_cast<uint32_t *>(w);
#pragma unroll
            for (int j = 0; j < 16; ++j)
              u[j] = bad ? 0u : pack_bf16x2(o[2 * j] * f.x * f.y, o[2 * j + 1] * f.x * f.y);
#pragma unroll
            for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4 *>(a.out + at * D + c + 8 * j) = w[j];
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              *reinterpret_cast<float4 *>(to + c + 4 * j) =
                  make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
          }
        }
        if (nan && has && !(whole && bad))
#pragma unroll 1
          for (int c = 0; c < D; ++c)
            if (ctl.nan_from[ks][c] < px_nan(k, lim)) {
              if (whole)
                a.out[at * D + c] = 0x7FFF;
              else
                to[c] = NAN;
            }
      }
      tc_before();
      __syncwarp();
      if (lane == 0) {
        bar_arrive(bar(kOFree));
        bar_arrive(bar(kSegEmpty + ss));
      }
      return true;
    };
    uint32_t g = 0;
    bool ok = true;
    for (uint32_t k = 0; ok; ++k) {  // segment k's q and first tile of V, the sums of the one before, the rest
      const int ss = k % kPxSegs;
      ok = wait(kSegFull + ss, (k / kPxSegs) & 1);
      if (!ok) break;
      const PxSeg &next = ctl.seg[ss];
      const bool ended = next.b < 0;
      const int tiles = ended ? 0 : next.tiles, t_end = next.t_end, tok0 = next.tok;
      const int min_lim = next.lim0 ? min(t_end, next.lim0 + next.rb * kPxRows / a.G) : t_end;
      if (!ended) {
        constexpr uint32_t kQs = kPxQs<D>;
        ok = k < kQs || wait(kQFree + k % kQs, (k / kQs - 1) & 1);
        if (!ok) break;
        tc_after();
        if (32 * quad < next.rows) {
          px_load_q<D>(a, next, tmem + lanes + kPxQ + k % kQs * (D / 2), ctl.qk[k % kPxStats], r);
          tc_st_wait();
        }
        tc_before();
        __syncwarp();
        if (lane == 0) {
          bar_arrive(bar(kQFull + k % kQs));
          bar_arrive(bar(kQReady + k % kPxStats));
        }
      }
      for (int t = 0; t < max(tiles, 1); ++t) {
        if (t < tiles) {
          const int slot = g % kPxV, buf = g & 1, tok = tok0 + t * kPxTok + 32 * quad;
          ok = wait(kVFull + slot, (g / kPxV) & 1) && wait(kHEmpty + buf, ((g >> 1) & 1) ^ 1);
          if (!ok) break;
          const uint8_t *v = smem + S::v + slot * S::kTile;
          uint8_t *h = smem + S::h + buf * S::kHalf;
          if (tok + 32 <= min_lim) {
            // rows eight apart have the same swizzle: the addresses are two and constants
            const uint8_t *va = px_codes<D>(v, row0, chunk), *vb = px_codes<D>(v, row0 + 4, chunk);
            uint8_t *ha = h, *hb = h;
#pragma unroll 1
            for (int q = 0; q < 4; q += 2) {
              constexpr int kS = 8 * D;
              if constexpr (D == 128) {
                const uint4 w0 = *reinterpret_cast<const uint4 *>(va), w1 = *reinterpret_cast<const uint4 *>(vb);
                const uint4 w2 = *reinterpret_cast<const uint4 *>(va + kS), w3 = *reinterpret_cast<const uint4 *>(vb + kS);
                px_store_half<D>(ha, row0, chunk, w0);
                px_store_half<D>(hb, row0 + 4, chunk, w1);
                px_store_half<D>(ha + 1024, row0, chunk, w2);
                px_store_half<D>(hb + 1024, row0 + 4, chunk, w3);
                vb += 2 * kS;
                hb += 2048;
              } else {
                const uint4 w0 = *reinterpret_cast<const uint4 *>(va), w2 = *reinterpret_cast<const uint4 *>(va + kS);
                px_store_half<D>(ha, row0, chunk, w0);
                px_store_half<D>(ha + 1024, row0, chunk, w2);
              }
              va += 2 * kS;
              ha += 2048;
            }
          } else if (tok < t_end) {
#pragma unroll 1
            for (int it = 0; it < kC; ++it) {
              const int row = row0 + kR * it, tk = tok + row - 32 * quad;
              uint4 w = *reinterpret_cast<const uint4 *>(px_codes<D>(v, row, chunk));
              uint32_t *x = reinterpret_cast<uint32_t *>(&w);
              if (tk >= t_end) {
                w = make_uint4(0, 0, 0, 0);  // cached bytes behind may be anything
              } else if (tk >= min_lim) {
                // a weight of 0 does not stop a NaN: it is put where its rows are written
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  uint32_t nan = nan_codes(x[q]);
                  x[q] &= ~((nan >> 7) * 0xFFu);
                  while (nan) {
                    const int byte = (__ffs(nan) - 1) >> 3;
                    nan &= nan - 1;
                    atomicMin(&ctl.nan_from[k % kPxStats][16 * chunk + 4 * q + byte], px_nan(k, tk));
                    ctl.nan_seg[k % kPxStats] = static_cast<int>(k) + 1;
                  }
                }
              }
              px_store_half<D>(h, row, chunk, w);
            }
          }
          proxy_fence();
          __syncwarp();
          if (lane == 0) {
            bar_arrive(bar(kVEmpty + slot));
            bar_arrive(bar(kHFull + buf));
          }
          ++g;
        }
        if (t == 0 && k > 0) {
          ok = px_put(k - 1);
          if (!ok) break;
        }
      }
      if (!ok || ended) break;
      __syncwarp();
      if (lane == 0) bar_arrive(bar(kStatFull + k % kPxStats));
    }
  } else {
    // ------------------------------------------------------- softmax, a row a lane
    const int grp = warp >> 2, quad = warp & 3, r = 32 * quad + lane;
    const uint32_t lanes = static_cast<uint32_t>(32 * quad) << 16;
    const uint32_t o_addr = tmem + lanes + kPxO;
    const int ref_mine = kRef + 4 * grp + quad, ref_other = kRef + 4 * (grp ^ 1) + quad;
    uint32_t g = 0;  // tiles of the CTA so far
    bool ok = true;
    for (uint32_t k = 0; ok; ++k) {
      const int ss = k % kPxSegs, ks = k % kPxStats;
      ok = wait(kSegFull + ss, (k / kPxSegs) & 1);
      if (!ok) break;
      const PxSeg &sg = ctl.seg[ss];
      if (sg.b < 0) break;
      const int tiles = sg.tiles, t_end = sg.t_end, tok0 = sg.tok;
      const bool act = 32 * quad < sg.rows;
      const int lim = sg.lim0 ? min(t_end, sg.lim0 + (sg.rb * kPxRows + r) / a.G) : t_end;
      const int min_lim = sg.lim0 ? min(t_end, sg.lim0 + sg.rb * kPxRows / a.G) : t_end;
      float m = -INFINITY, n = -INFINITY, l = 0.f, lm = -INFINITY, qk = 0.f;
      int bad_from = INT_MAX, come = 0;
      const int first = (g & 1) != static_cast<uint32_t>(grp);  // the group's first tile
      if (first < tiles) {
        ok = wait(kQReady + ks, (k / kPxStats) & 1);
        if (!ok) break;
        qk = ctl.qk[ks][r];  // (of a row that exists)
      }
      for (int t = first; t < tiles; t += 2) {
        const uint32_t gt = g + t;
        const int cs = gt % kPxScales, tok = tok0 + t * kPxTok;
        ok = wait(kScFull + cs, (gt / kPxScales) & 1) && wait(kSFull + grp, (gt >> 1) & 1);
        if (!ok) break;
        tc_after();
        come = t + 1;
        const float4 *sc = ctl.sc[cs];
        const uint32_t s0 = tmem + lanes + px_scol(gt, 0), s1 = tmem + lanes + px_scol(gt, 1) - 64;
        float mx = -INFINITY, mv = -INFINITY, x[32];
        const bool full = tok + kPxTok <= min_lim;  // everybody sees all of it
        const int chunks = full ? 4 : (min(kPxTok, t_end - tok) + 31) >> 5;  // of 32 tokens
        if (act) {
          bad_from = min(bad_from, ctl.bad[cs]);
          // (rolled loops: with the chunks laid out one after another the roles' code did not fit the
          // instruction caches, and its fetching took twice the time of the work)
          if (full) {
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              tc_ld32(x, (c < 2 ? s0 : s1) + 32 * c);
              px_max(x, sc + 2 * c, qk, mx, mv);
            }
          } else {
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
              tc_ld32(x, (c < 2 ? s0 : s1) + 32 * c);
              px_mask(x, lim - tok - 32 * c);
              px_max(x, sc + 2 * c, qk, mx, mv);
            }
          }
        }
        // the references, which the groups hand one another
        if (gt > 0) {
          ok = wait(ref_other, ((gt - 1) >> 1) & 1);
          if (!ok) break;
        }
        float fo = 1.f;
        if (act) {
          if (t > 0) {
            const float2 now = ctl.now[grp ^ 1][r];
            m = now.x;
            n = now.y;
          }
          if (m == -INFINITY || mx > m + kPxFar) m = mx;
          if (n == -INFINITY) {
            n = mv;
          } else if (mv > n + kRescaleThreshold) {
            fo = fast_exp2(n - mv);
            n = mv;
          }
          ctl.now[grp][r] = make_float2(m, n);
        }
        __syncwarp();
        if (lane == 0) bar_arrive(bar(ref_mine));
        if (act) {
          if (lm != m) {
            l = l == 0.f ? 0.f : l * fast_exp2(lm - m);
            lm = m;
          }
          const bool none = n == -INFINITY;  // nothing seen yet: every x is -inf
          const float mm = none ? 0.f : m, mn = none ? 0.f : m - n;
          float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          float p[16];
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {  // 64 tokens
            if (full) {
#pragma unroll 1
              for (int c = 2 * h; c < 2 * h + 2; ++c) {
                tc_ld32(x, (c < 2 ? s0 : s1) + 32 * c);
                px_weights<false>(x, sc + 2 * c, qk, mm, mn, l2, p);
                tc_st16((h ? s1 : s0) + 32 * c, p);  // in the chunk's own columns
              }
            } else {
#pragma unroll 1
              for (int c = 2 * h; c < min(2 * h + 2, chunks); ++c) {
                tc_ld32(x, (c < 2 ? s0 : s1) + 32 * c);
                px_mask(x, lim - tok - 32 * c);
                px_weights<true>(x, sc + 2 * c, qk, mm, mn, l2, p);
                tc_st16((h ? s1 : s0) + 32 * c, p);
              }
            }
            if (h == 0 && t > 0 && __any_sync(0xffffffffu, fo != 1.f)) {  // before any of the tile's products
              ok = wait(kHEmpty + (grp ^ 1), ((gt - 1) >> 1) & 1);
              if (!ok) break;
              tc_after();
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                float o[32];
                tc_ld32(o, o_addr + c);
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] *= fo;
                tc_st32(o_addr + c, o);
              }
            }
            tc_st_wait();
            tc_before();
            __syncwarp();
            if (lane == 0) bar_arrive(bar(h ? kPFull + (gt & 3) : kPHalf + grp));
          }
          if (!ok) break;
          l += (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y);
        } else {
          tc_before();
          __syncwarp();
          if (lane == 0) {
            bar_arrive(bar(kPHalf + grp));
            bar_arrive(bar(kPFull + (gt & 3)));
          }
        }
      }
      if (!ok) break;
      g += tiles;
      ctl.end[ks][grp][r] = make_float4(lm, lim > bad_from ? -1.f : l, n, 0.f);
      if (quad == 0 && lane == 0) ctl.come[ks][grp] = come;
      __syncwarp();
      if (lane == 0) {
        bar_arrive(bar(kStatFull + ks));
        bar_arrive(bar(kSegEmpty + ss));
      }
    }
    tc_before();
  }
  __syncthreads();  // every role comes here, also when a wait gave up
  if (warp == kPxMma) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

// ---------------------------------------------------------------------------
// merge: a row's prefix and own tokens, each here or in the parts of several CTAs
// ---------------------------------------------------------------------------

constexpr int kPxMergeWarps = 8;

// One request of the plan, a warp a row and head, the lanes its dims; four parts' loads in flight.
//   out = 2^(N - M) sum_p 2^(n_p - N) o_p / sum_p 2^(m_p - M) l_p
// (a part 2^126 below the largest adds nothing: weights are held to 2^-31 of that)
template <int D>
__global__ void __launch_bounds__(32 * kPxMergeWarps) prefix_merge_kernel(PfArgs a) {
  constexpr int RF = D + kStat, V = D / 32, kBatch = 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // (the kernel ahead began, and let this one start, when the plan was complete)
  const int n_grp = __ldcg(&a.plan->n_grp), n_req = __ldcg(&a.plan->n_req);
  const PxItem it = px_load_item(a.items + n_grp + min(static_cast<int>(blockIdx.x), max(n_req - 1, 0)));
  grid_dependency_wait();
  allow_dependents();
  if (static_cast<int>(blockIdx.x) >= n_req) return;
  for (int64_t u = blockIdx.y * kPxMergeWarps + warp; u < static_cast<int64_t>(it.n) * a.Hq;
       u += gridDim.y * kPxMergeWarps) {
    const int i = static_cast<int>(px_div(u, a.Hq)), h = static_cast<int>(u - static_cast<int64_t>(i) * a.Hq);
    const int64_t at = (static_cast<int64_t>(it.row0) + i) * a.Hq + h;
    uint16_t *o = a.out + at * D + V * lane;
    const float *rows = a.rows + at * RF, *own_rows = rows + static_cast<int64_t>(a.rg.n_tokens) * a.Hq * RF;
    float M = -INFINITY, N = -INFINITY, l = 0.f, acc[V];
    bool bad = !it.live;
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = 0.f;
    // where the sums lie: the prefix's, then those of its own tokens
    float4 where[2];
    where[0] = where[1] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (it.live) {
      if (it.pre) where[0] = __ldcg(reinterpret_cast<const float4 *>(rows + D));
      where[1] = __ldcg(reinterpret_cast<const float4 *>(own_rows + D));
      if (where[1].w == kDone) continue;
    }
    // The parts of both in one list.  Part p lies in the p-th CTA from here on: the first in slot 1, others in
    // slot 0.
    const float *base[2] = {rows, own_rows};
    int parts[2];
    int64_t slot[2];  // from one CTA's slot to the next; 0: not cut
#pragma unroll
    for (int own = 0; own < 2; ++own) {
      const float4 e = where[own];
      parts[own] = e.w == 0.f ? 0 : 1;
      slot[own] = 0;
      if (e.w != kCut) continue;
      parts[own] = __float_as_int(e.y);
      const int row = (it.row0 + i - (own ? it.row0 : it.row_pre)) * a.G + h % a.G;
      int64_t at_row = row % kPxRows, rows_slot = kPxRows;
      if (own && a.own_split) {
        const int in = row % (a.rt * a.rk), kvh = h / a.G;
        rows_slot = a.hg * a.rt * a.rk;
        at_row = (kvh % a.hg * a.rt + in / a.rk) * a.rk + in % a.rk;
      }
      slot[own] = rows_slot * RF;
      base[own] = (own && a.own_split ? a.own_cut : a.cut) + (2 * __float_as_int(e.x) * rows_slot + at_row) * RF;
    }
    const int all = parts[0] + parts[1];
    for (int p0 = 0; p0 < all; p0 += kBatch) {
      float4 s[kBatch];
      float v[kBatch][V];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        s[j] = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
        if (p0 + j < all) {
          const bool own = p0 + j >= parts[0];
          const int p = p0 + j - (own ? parts[0] : 0);
          const float *q = (own ? base[1] : base[0]) + (2 * p + (p == 0)) * (own ? slot[1] : slot[0]);
          s[j] = __ldcg(reinterpret_cast<const float4 *>(q + D));
          if constexpr (V == 4) {
            const float4 x = __ldcg(reinterpret_cast<const float4 *>(q) + lane);
            v[j][0] = x.x;
            v[j][1] = x.y;
            v[j][2] = x.z;
            v[j][3] = x.w;
          } else {
            const float2 x = __ldcg(reinterpret_cast<const float2 *>(q) + lane);
            v[j][0] = x.x;
            v[j][1] = x.y;
          }
        }
      }
      float Mb = M, Nb = N;
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        Mb = fmaxf(Mb, s[j].x);
        Nb = fmaxf(Nb, s[j].z);
        bad |= s[j].y < 0.f;
      }
      const float fl = M == -INFINITY ? 0.f : fast_exp2(M - Mb), fo = N == -INFINITY ? 0.f : fast_exp2(N - Nb);
      l *= fl;
#pragma unroll
      for (int k = 0; k < V; ++k) acc[k] *= fo;
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (s[j].y == 0.f) continue;  // saw nothing
        l = fmaf(fast_exp2(s[j].x - Mb), s[j].y, l);
        const float f = fast_exp2(s[j].z - Nb);
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] = fmaf(f, v[j][k], acc[k]);
      }
      M = Mb;
      N = Nb;
    }
    const float2 f = bad ? make_float2(0.f, 0.f) : out_scale(N - M - 7.f, l);
#pragma unroll
    for (int k = 0; k < V; k += 2)
      *reinterpret_cast<uint32_t *>(o + k) =
          bad ? 0u : pack_bf16x2(acc[k] * f.x * f.y, acc[k + 1] * f.x * f.y);
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

namespace {

size_t px_up256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }
size_t px_rows_bytes(int64_t n_tokens, int Hq, int D) {
  return px_up256(2ull * n_tokens * Hq * (D + kStat) * sizeof(float));
}
size_t px_cut_bytes(int ctas, int D) { return px_up256(2ull * ctas * kPxRows * (D + kStat) * sizeof(float)); }

size_t px_q_bytes(int64_t n_tokens, int Hq, int D) { return px_up256(2ull * n_tokens * Hq * D); }
size_t px_qk_bytes(int64_t n_tokens, int Hq) { return px_up256(4ull * n_tokens * Hq); }
size_t px_plan_bytes(int64_t n_tokens) {
  return 256 + px_up256(2 * n_tokens * sizeof(PxItem)) + px_up256((2 * n_tokens + 1) * sizeof(int64_t));
}
size_t px_own_cut_bytes(int Hq, int Hkv, int D, int ctas);
size_t px_bytes(int64_t n_tokens, int Hq, int Hkv, int D, int ctas) {
  return px_own_cut_bytes(Hq, Hkv, D, ctas) + px_plan_bytes(n_tokens) + px_rows_bytes(n_tokens, Hq, D) + px_cut_bytes(ctas, D) +
         px_q_bytes(n_tokens, Hq, D) + px_qk_bytes(n_tokens, Hq);
}

using PxFn = void (*)(CUtensorMap, CUtensorMap, PfArgs);

// Opt the kernel into its shared memory, once per device.
template <typename Fn>
bool px_opt_in(Fn fn, int variant, size_t smem) {
  constexpr int kMaxDev = 64;
  static std::atomic<bool> done[kMaxDev][6];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return false;
  if (done[dev][variant].load(std::memory_order_acquire)) return true;
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
    return false;
  done[dev][variant].store(true, std::memory_order_release);
  return true;
}

// [page][head][slot][dim] as a 4-D map; a box is `slots` slots of `heads` heads.
bool px_map(CUtensorMap *map, const void *pool, const kvq_block_cache &c, int slots, int heads) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t D = c.head_dim, P = c.page_size, H = c.num_kv_heads, NP = c.num_pages;
  const cuuint64_t dims[4] = {D, P, H, NP};
  const cuuint64_t strides[3] = {D, P * D, H * P * D};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(D), static_cast<cuuint32_t>(slots),
                             static_cast<cuuint32_t>(heads), 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(pool), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Own tokens: the mma.sync kernel where a request has few rows.
using BaFn = void (*)(CUtensorMap, CUtensorMap, BaArgs);

template <int D>
BaFn px_own_kernel(int rk) {
  return rk == 4 ? block_split_kernel<D, 4, true>
                 : rk == 8 ? block_split_kernel<D, 8, true> : block_split_kernel<D, 16, true>;
}

// Rows (times heads a kv head) of a request that it takes, the most that its warps hold at once.  Both sides, us, it
// and prefix_kernel: 256 requests of 1 - 700 own tokens, 4 rows 37 and 139, 8 rows 47 and 139, 16 rows 78 and 150;
// 64 of 8,193, 8 rows 185 and 287, 16 rows 308 and 291.
constexpr int kPxOwnRows = 16;

// The slots of its parts, for every number of rows that a call may allow.
size_t px_own_cut_bytes(int Hq, int Hkv, int D, int ctas) {
  size_t most = 0;
  for (int rows : {4, 8, 16})
    if (rows >= Hq / Hkv) most = std::max(most, ba_part_bytes(ba_shape(rows, 1, Hkv, D, 0), D, ctas));
  return px_up256(most);
}

}  // namespace

}  // namespace kvq

using namespace kvq;

extern "C" size_t kvq_block_prefix_attn_workspace_size(int32_t n_tokens, int32_t Hq,
                                                       int32_t num_kv_heads, int32_t head_dim) {
  if (n_tokens < 0 || Hq <= 0 || num_kv_heads <= 0 || Hq % num_kv_heads) return 0;
  if (head_dim != 64 && head_dim != 128) return 0;
  int sms = 0;
  if (device_sm_count(&sms) != KVQ_OK) return 0;
  return px_bytes(n_tokens, Hq, num_kv_heads, head_dim, sms);
}

extern "C" kvq_status kvq_block_prefix_attn(
    const kvq_block_cache *cache, const void *q, int64_t q_stride, int32_t Hq,
    const int32_t *tok_start, int32_t n_tokens, int32_t max_q, const int32_t *seq_lens,
    const int32_t *block_table, int32_t B, int32_t MP, const int32_t *group_start,
    const int32_t *prefix_pages, int32_t n_groups, const uint8_t *abort_mask, float sm_scale,
    void *out, void *workspace, size_t workspace_bytes, uint32_t *err_word, kvq_stream_t stream) {
  kvq_status st = validate_block_cache(cache);
  if (st != KVQ_OK) return st;
  const int D = cache->head_dim, Hkv = cache->num_kv_heads;
  st = validate_ragged(tok_start, n_tokens, block_table, B, MP, cache->page_size);
  if (st != KVQ_OK) return st;
  if (Hq <= 0 || Hq % Hkv || max_q <= 0 || n_groups < 0 || !std::isfinite(sm_scale)) return KVQ_ERR_INVALID_ARG;
  const int G = Hq / Hkv;
  if (static_cast<int64_t>(n_tokens) * G > INT32_MAX / 2) return KVQ_ERR_INVALID_ARG;
  if (static_cast<int64_t>(n_groups) + B > 1 << 30) return KVQ_ERR_INVALID_ARG;  // px_plan walks both as one list
  const int64_t capacity = static_cast<int64_t>(MP) * cache->page_size;
  if (capacity > INT32_MAX - 255) return KVQ_ERR_INVALID_ARG;
  if (n_tokens == 0 || B == 0) return KVQ_OK;
  if (!seq_lens || !out || !workspace || !aligned16(out) || !rows_ok(q, q_stride, Hq, D)) return KVQ_ERR_INVALID_ARG;
  if (n_groups > 0 && (!group_start || !prefix_pages)) return KVQ_ERR_INVALID_ARG;
  int sms = 0;
  if (device_sm_count(&sms) != KVQ_OK) return KVQ_ERR_CUDA;
  if (!aligned256(workspace) || workspace_bytes < px_bytes(n_tokens, Hq, Hkv, D, sms)) return KVQ_ERR_WORKSPACE;
  PfArgs a;
  a.q = static_cast<const uint16_t *>(q);
  a.q_stride = q_stride;
  a.rg = {tok_start, seq_lens, B, n_tokens, capacity};
  a.block_table = block_table;
  a.group_start = group_start;
  a.prefix_pages = prefix_pages;
  a.abort_mask = abort_mask;
  uint8_t *at = static_cast<uint8_t *>(workspace);
  a.plan = reinterpret_cast<PxPlan *>(at);
  a.items = reinterpret_cast<PxItem *>(at + 256);
  a.units = reinterpret_cast<int64_t *>(at + 256 + px_up256(2ull * n_tokens * sizeof(PxItem)));
  at += px_plan_bytes(n_tokens);
  a.rows = reinterpret_cast<float *>(at);
  at += px_rows_bytes(n_tokens, Hq, D);
  a.cut = reinterpret_cast<float *>(at);
  at += px_cut_bytes(sms, D);
  a.qp = at;
  at += px_q_bytes(n_tokens, Hq, D);
  a.qk = reinterpret_cast<float *>(at);
  at += px_qk_bytes(n_tokens, Hq);
  const BaShape shape = ba_shape(std::min(max_q, kPxOwnRows), G, Hkv, D, 0);
  a.own_split = static_cast<int64_t>(max_q) * G <= kPxOwnRows;
  a.hg = shape.hg;
  a.rt = shape.rt;
  a.rk = shape.rk;
  a.own_cut = reinterpret_cast<float *>(at);
  a.scales = reinterpret_cast<const float2 *>(cache->scales);
  a.out = static_cast<uint16_t *>(out);
  a.err_word = err_word;
  a.num_pages = cache->num_pages;
  a.p_shift = cache->page_size == 16 ? 4 : cache->page_size == 32 ? 5 : 6;
  a.Hkv = Hkv;
  a.Hq = Hq;
  a.G = G;
  a.MP = MP;
  a.max_q = max_q;
  a.n_groups = n_groups;
  a.q_scale = sm_scale * kLog2e;
  const PxFn fn = D == 128 ? prefix_kernel<128> : prefix_kernel<64>;
  const size_t smem = D == 128 ? PxSmem<128>::bytes : PxSmem<64>::bytes;
  if (!px_opt_in(fn, D == 128, smem)) return KVQ_ERR_CUDA;
  CUtensorMap kmap, vmap;
  if (!px_map(&kmap, cache->k_pool, *cache, cache->page_size, 1) ||
      !px_map(&vmap, cache->v_pool, *cache, cache->page_size, 1))
    return KVQ_ERR_CUDA;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const int64_t q_ctas = (static_cast<int64_t>(n_tokens) * Hq * (D / 4) + kPxQThreads - 1) / kPxQThreads;
  if (launch_dependent(D == 128 ? prefix_plan_kernel<128> : prefix_plan_kernel<64>, static_cast<unsigned>(1 + q_ctas),
                       kPxQThreads, 0, cs, a, sms) != cudaSuccess)
    return KVQ_ERR_CUDA;
  if (launch_dependent(fn, sms, kPxThreads, smem, cs, kmap, vmap, a) != cudaSuccess) return KVQ_ERR_CUDA;
  if (a.own_split) {
    BaArgs o = {};
    o.q = a.q;
    o.q_stride = q_stride;
    o.rg = a.rg;
    o.block_table = block_table;
    o.scales = a.scales;
    o.part = reinterpret_cast<float *>(at);
    o.err_word = err_word;
    o.num_pages = a.num_pages;
    o.p_shift = a.p_shift;
    o.Hkv = Hkv;
    o.Hq = Hq;
    o.G = G;
    o.MP = MP;
    o.max_q = max_q;
    o.hg = shape.hg;
    o.rt = shape.rt;
    o.tw = shape.tw;
    for (int t = shape.tw; t > 1; t = (t + 1) / 2) ++o.rounds;
    o.groups = shape.groups;
    o.stages = ba_stages(shape, D);
    o.q_scale = a.q_scale;
    o.plan = a.plan;
    o.items = a.items;
    o.rows = a.rows;
    const BaFn own = D == 128 ? px_own_kernel<128>(shape.rk) : px_own_kernel<64>(shape.rk);
    const int variant = shape.rk == 4 ? 0 : shape.rk == 8 ? 1 : 2;
    if (!(D == 128 ? px_opt_in<BaFn>(own, 3 + variant, kBaSmem) : px_opt_in<BaFn>(own, variant, kBaSmem)))
      return KVQ_ERR_CUDA;
    if (!px_map(&kmap, cache->k_pool, *cache, kTile, shape.hg) || !px_map(&vmap, cache->v_pool, *cache, kTile, shape.hg))
      return KVQ_ERR_CUDA;
    if (launch_dependent(own, sms, kBaThreads, kBaSmem, cs, kmap, vmap, o) != cudaSuccess) return KVQ_ERR_CUDA;
  }
  // a warp a row and head, up to 64 CTAs a request
  const int64_t most = (static_cast<int64_t>(std::min(max_q, n_tokens)) * Hq + kPxMergeWarps - 1) / kPxMergeWarps;
  const dim3 grid(static_cast<unsigned>(std::min(B, n_tokens)), static_cast<unsigned>(std::min<int64_t>(64, most)));
  if (launch_dependent(D == 128 ? prefix_merge_kernel<128> : prefix_merge_kernel<64>, grid, 32 * kPxMergeWarps, 0, cs,
                       a) != cudaSuccess)
    return KVQ_ERR_CUDA;
  return KVQ_OK;
}
