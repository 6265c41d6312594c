// kvq_block_append, kvq_rope_block_append, kvq_block_read: writing the
// block-scaled cache (rotation, scale, quantisation in one pass) and reading
// it back.
//
// Mathematics: include/kvq.h.  Work item: one (request, page) that the step
// touches, with all kv heads; every CTA scans the requests once and takes an
// equal run of items (find_run), so that one prompt among decode tokens
// does not leave the other SMs idle.
//
// Append has three kernels, all with the maximum that sets a block's scale and
// the conversion in one visit:
//   short  decode and draft steps, with parts of prompts among them or not: latency
//          counts.  K, V and q of a page go to CTAs of their own, a warp takes one
//          head's rows, four (head_dim 128) at a time; further rows are read twice,
//          the second time from L1.  64 rows of 64 requests, K and V of 8 heads, q of
//          32, rotated: 2.75 us; 256 drafts of 1 - 8 rows 9.1.
//   ring   prompts with enough kv heads: bandwidth counts (2 D (2 + 1) bytes a
//          token and kv head, 4 D a query head).  A producer warp stages the
//          rows of a page and a group of heads with one TMA copy each into a
//          shared-memory ring; a consumer warp takes 16 rows of one head.  64
//          prompts of 8,192 tokens: 497 - 507 us, 94 - 96% of the measured copy rate.
//   wide   prompts with few kv heads: the same without the ring, a warp's 16
//          rows loaded by itself.
// Reading back has one kernel: 48 ragged prefixes 215 us, 97%.
// In 32- and 64-token pages the warps of a block exchange their maxima through
// shared memory.  The page's angles are computed once into shared memory and
// used by all heads.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "block_common.cuh"

namespace kvq {

constexpr int kBcThreads = 256;
constexpr int kBcWarps = kBcThreads / 32;
constexpr int kRowsPerWarp = 16;

struct BlockPool {
  uint8_t *k, *v;
  float *scales;
  int32_t num_pages, P, H;
  int32_t ps;  // P = 1 << ps: a division by P in the chain of a decode step's loads costs 0.1 us
};

struct BlockAppendArgs {
  BlockPool c;
  Ragged rg;
  const int32_t *block_table;
  uint32_t *err_word;
  const uint16_t *k_new, *v_new, *q;
  uint16_t *q_out;
  int64_t k_stride, v_stride, q_stride, q_out_stride;
  int32_t MP, Hq;
  RopeArgs rope;
};

// Pages that a request's rows touch.
__device__ __forceinline__ int pages_touched(const Rows &r, int ps) {
  return r.n == 0 || r.err ? 0 : ((r.p0 + r.n - 1) >> ps) - (r.p0 >> ps) + 1;
}

// Old codes of a block whose scale grew: rows [0, n_old) from `block` on.
template <int D>
__device__ __forceinline__ void requantise_rows(uint8_t *block, int n_old, float ratio, int lane) {
  constexpr int kLanes = D / 16;  // lanes a row, 16 codes each
  for (int r = lane / kLanes; r < n_old; r += 32 / kLanes) {
    uint4 *p = reinterpret_cast<uint4 *>(block + r * D) + lane % kLanes;
    const uint4 w = *p;
    uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float x[4];
      e4m3x4_to_f32(u[j], x);
      u[j] = static_cast<uint32_t>(f32x2_to_e4m3x2(x[0] * ratio, x[1] * ratio)) |
             (static_cast<uint32_t>(f32x2_to_e4m3x2(x[2] * ratio, x[3] * ratio)) << 16);
    }
    *p = make_uint4(u[0], u[1], u[2], u[3]);
  }
}

// The next page of a CTA's run.
struct PageWalk {
  int64_t left, in;
  int b;
};

struct PageItem {
  int page;          // -1: outside the pool
  int first;         // position of the first row
  int slot0, nrow;   // slots [slot0, slot0 + nrow) of the page
  int64_t row0;
};

template <bool kLens>
__device__ __forceinline__ bool next_page(const Ragged &rg, const int32_t *block_table, int MP,
                                          int ps, int num_pages, PageWalk &w, PageItem &it) {
  if (w.left <= 0) return false;
  Rows rq = request_rows<kLens>(rg, w.b);
  while (w.in >= pages_touched(rq, ps)) {
    ++w.b;
    w.in = 0;
    rq = request_rows<kLens>(rg, w.b);
  }
  const int lp = (rq.p0 >> ps) + static_cast<int>(w.in);
  ++w.in;
  --w.left;
  const int page = __ldg(block_table + static_cast<int64_t>(w.b) * MP + lp);
  it.page = page >= 0 && page < num_pages ? page : -1;
  it.first = max(rq.p0, lp << ps);
  it.slot0 = it.first - (lp << ps);
  it.nrow = min(rq.p0 + rq.n, (lp + 1) << ps) - it.first;
  it.row0 = static_cast<int64_t>(rq.row) + (it.first - rq.p0);
  return true;
}

// The CTA's run of pages (every thread calls it).
template <int NT, bool kLens>
__device__ __forceinline__ PageWalk page_run(const Ragged &rg, int ps, uint32_t *err_word,
                                             RunScan<NT> &scan) {
  const RunStart run = find_run<NT>(rg.B, gridDim.x, blockIdx.x, scan, [&](int b) -> int64_t {
    const Rows r = request_rows<kLens>(rg, b);
    if (r.err && blockIdx.x == 0) report(err_word, r.err);
    return pages_touched(r, ps);
  });
  return {min(run.per, run.total - blockIdx.x * run.per), run.in, run.b};
}

// Angles of rows 0 .. nrow - 1, at positions first + row, into tab: threads
// tid, tid + nt, ... of those that call.
__device__ __forceinline__ void fill_angles(float4 *tab, const uint64_t *freq, int first, int nrow,
                                            int rd, bool half, float mscale, int tid, int nt) {
  const int nq = rd / 4;
  for (int j = tid; j < nrow * nq; j += nt) {
    const int r = j / nq, q = j - r * nq;
    const float2 x = rotation(first + r, freq[2 * q], mscale);
    const float2 y = rotation(first + r, freq[2 * q + 1], mscale);
    tab[r * nq + angle_slot(q, rd, half)] = make_float4(x.x, x.y, y.x, y.y);
  }
}

// 8 values -> their codes.
__device__ __forceinline__ uint2 codes8(const float *v, float inv) {
  const float2 s = make_float2(inv, inv);
  uint32_t o[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float2 x = __fmul2_rn(make_float2(v[4 * j], v[4 * j + 1]), s);
    const float2 y = __fmul2_rn(make_float2(v[4 * j + 2], v[4 * j + 3]), s);
    o[j] = static_cast<uint32_t>(f32x2_to_e4m3x2(x.x, x.y)) |
           (static_cast<uint32_t>(f32x2_to_e4m3x2(y.x, y.y)) << 16);
  }
  return make_uint2(o[0], o[1]);
}

// 16 values (an item) -> codes at the two chunks of a row.
__device__ __forceinline__ void store_codes(uint8_t *row, ItemChunks ch, const float (&y)[16],
                                            float inv) {
  *reinterpret_cast<uint2 *>(row + ch.c0 * 8) = codes8(y, inv);
  *reinterpret_cast<uint2 *>(row + ch.c1 * 8) = codes8(y + 8, inv);
}

// A rotated item -> bf16 at the two chunks; a chunk past rotary_dim as it came.
__device__ __forceinline__ void store_rotated(uint16_t *row, ItemChunks ch, const float (&y)[16],
                                              uint4 w0, uint4 w1, int i, int D, int rd, bool half) {
  const int lim = half ? (i < rd / 16 ? D / 8 : 0) : rd / 8;
  *reinterpret_cast<uint4 *>(row + ch.c0 * 8) = ch.c0 < lim ? pack8(y) : w0;
  *reinterpret_cast<uint4 *>(row + ch.c1 * 8) = ch.c1 < lim ? pack8(y + 8) : w1;
}

// Largest magnitudes, as the bits of a float (their order is the magnitudes'),
// inf and NaN included: kept as they come, since one instruction a value is
// what there is time for.  Only when the maximum turns out not finite is it
// taken again over the finite values (kFinite).
template <bool kFinite>
__device__ __forceinline__ uint32_t item_max(const float (&y)[16]) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const uint32_t u = __float_as_uint(y[j]) & 0x7FFFFFFFu;
    m = max(m, kFinite && u >= 0x7F800000u ? 0u : u);
  }
  return m;
}

template <bool kFinite>
__device__ __forceinline__ uint32_t words_max(uint4 a, uint4 b) {  // 16 bf16
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    uint32_t u = w[j] & 0x7FFF7FFFu;
    if (kFinite) u &= ~__vcmpgeu2(u, 0x7F807F80u);
    m = __vmaxu2(m, u);
  }
  return max(m & 0xFFFF0000u, m << 16);
}

// The block's amax from a function that gives a lane's maximum, whole warp.
template <typename F>
__device__ __forceinline__ float warp_amax(F lane_max) {
  uint32_t m = __reduce_max_sync(0xffffffffu, lane_max(std::false_type()));
  if (m >= 0x7F800000u) m = __reduce_max_sync(0xffffffffu, lane_max(std::true_type()));
  return __uint_as_float(m);
}

// ---- short steps

// A share of a page: K (0), V (1), or qheads heads of q (2 ..).
struct ShortShare {
  bool is_v, is_q;
  int h0, heads;
  const uint16_t *src;
  int64_t stride;
};

__device__ __forceinline__ ShortShare short_share(const BlockAppendArgs &a, int share, int qheads, int D) {
  ShortShare s;
  s.is_v = share == 1;
  s.is_q = share > 1;
  s.h0 = s.is_q ? (share - 2) * qheads : 0;
  s.heads = s.is_q ? min(qheads, a.Hq - s.h0) : a.c.H;
  s.src = s.is_q ? a.q + static_cast<int64_t>(s.h0) * D : s.is_v ? a.v_new : a.k_new;
  s.stride = s.is_q ? a.q_stride : s.is_v ? a.v_stride : a.k_stride;
  return s;
}

// A thread's place in a warp's rows.
struct ShortLane {
  int warp, lane, i, r0, rd;
  bool half;
  ItemChunks ch;
};

template <int D, bool kRope>
__device__ __forceinline__ ShortLane short_lane(const BlockAppendArgs &a) {
  constexpr int kItems = D / 16;  // lanes a row (two 8-dim chunks each)
  ShortLane t;
  t.warp = threadIdx.x >> 5;
  t.lane = threadIdx.x & 31;
  t.i = t.lane % kItems;
  t.r0 = t.lane / kItems;
  t.half = !kRope || a.rope.layout == KVQ_ROPE_HALF;
  t.rd = kRope ? a.rope.rd : D;
  t.ch = item_chunks(t.i, D, t.rd, t.half);
  return t;
}

// A CTA's share of request b's page pg (counted from the first that the step touches).
// tab: kRope: [P][rd / 4] angles of the page's rows; freq: the pairs' turns a token, set but
// not yet synchronised.
template <int D, bool kRope>
__device__ __forceinline__ void append_page(const BlockAppendArgs &a, const ShortShare &sh, const ShortLane &t,
                                            const Rows &rq, int b, int pg, float4 *tab, const uint64_t *freq) {
  constexpr int kItems = D / 16;
  constexpr int kRpp = 32 / kItems;   // rows a warp pass
  // passes whose rows are asked for together in the first reading (2 requests of 44 rows 5.45
  // us, one by one 7.1); rotation has no registers for it
  constexpr int kAhead = kRope ? 1 : 4;
  const int P = a.c.P, H = a.c.H, heads = sh.heads;
  const int warp = t.warp, lane = t.lane, i = t.i, r0 = t.r0, rd = t.rd;
  const bool half = t.half;
  const ItemChunks ch = t.ch;
  const int lp = (rq.p0 >> a.c.ps) + pg;
  const int page = __ldg(a.block_table + static_cast<int64_t>(b) * a.MP + lp);
  const int first = max(rq.p0, lp << a.c.ps), slot0 = first - (lp << a.c.ps);
  const int nrow = min(rq.p0 + rq.n, (lp + 1) << a.c.ps) - first;
  const int64_t row0 = static_cast<int64_t>(rq.row) + (first - rq.p0);
  auto load = [&](int r, int h, uint4 (&w)[2]) {
    w[0] = w[1] = make_uint4(0, 0, 0, 0);
    if (r < nrow && h < heads) {
      const uint16_t *s = sh.src + (row0 + r) * sh.stride + static_cast<int64_t>(h) * D;
      w[0] = *reinterpret_cast<const uint4 *>(s + ch.c0 * 8);
      w[1] = *reinterpret_cast<const uint4 *>(s + ch.c1 * 8);
    }
  };
  // this warp's first rows, before anything that waits: head `warp` (K, V),
  // or the (token, head) rows from `e` on (q)
  int e = warp * kRpp + r0;
  uint4 w[2];
  load(sh.is_q ? e / heads : r0, sh.is_q ? e % heads : warp, w);
  if (kRope && !sh.is_v) {  // uniform over the CTA
    __syncthreads();  // the previous page's angles are no longer read, and freq is set
    fill_angles(tab, freq, first, nrow, rd, half, a.rope.mscale, threadIdx.x, kBcThreads);
    __syncthreads();
  }
  if (page < 0 || page >= a.c.num_pages) {
    if (threadIdx.x == 0) report(a.err_word, KVQ_ERRBIT_PAGE);
    return;
  }
  auto values = [&](const uint4 (&w)[2], int r, float (&y)[16]) {
    unpack8(w[0], y);
    unpack8(w[1], y + 8);
    if constexpr (kRope)
      if (!sh.is_v && r < nrow) rotate_item(y, tab + r * (rd / 4), i, rd, half, ch);
  };
  if (sh.is_q) {
    const int total = nrow * heads;
    while (e - r0 < total) {
      const int r = e / heads, h = e - r * heads;
      const int e2 = e + kBcWarps * kRpp;
      uint4 w2[2];
      load(e2 / heads, e2 % heads, w2);  // the next rows, in flight meanwhile
      float y[16];
      values(w, r, y);
      if (r < nrow)
        store_rotated(a.q_out + (row0 + r) * a.q_out_stride + static_cast<int64_t>(sh.h0 + h) * D,
                      ch, y, w[0], w[1], i, D, rd, half);
      w[0] = w2[0];
      w[1] = w2[1];
      e = e2;
    }
    return;
  }
  for (int h = warp; h < H; h += kBcWarps) {
    if (h != warp) load(r0, h, w);
    const int64_t blk = static_cast<int64_t>(page) * H + h;
    float *scale = a.c.scales + 2 * blk + sh.is_v;
    const float s_old = slot0 > 0 ? *scale : 0.f;
    float y[16];
    values(w, r0, y);
    const float amax = warp_amax([&](auto finite) {
      uint32_t m = item_max<decltype(finite)::value>(y);
#pragma unroll kAhead
      for (int r = kRpp + r0; r - r0 < nrow; r += kRpp) {
        uint4 v[2];
        float z[16];
        load(r, h, v);
        values(v, r, z);
        m = max(m, item_max<decltype(finite)::value>(z));
      }
      return m;
    });
    const float s_new = fmaxf(pow2(block_exponent(amax)), s_old);
    const float inv = 1.0f / s_new;  // exact for a power of two
    uint8_t *block = (sh.is_v ? a.c.v : a.c.k) + blk * P * D;
    if (s_new > s_old && slot0 > 0) requantise_rows<D>(block, slot0, s_old / s_new, lane);
    if (lane == 0) *scale = s_new;
    for (int r = r0; r - r0 < nrow; r += kRpp) {
      if (r != r0) {
        load(r, h, w);
        values(w, r, y);
      }
      if (r < nrow) store_codes(block + (slot0 + r) * D, ch, y, inv);
    }
  }
}

// A CTA beyond the requests' own (idle_b < 0), or request idle_b's first, which has no pages: scans
// the requests and takes an equal run of the pages that are beyond the requests' own CTAs'.
// Out of line, so that its state costs those no registers (256 drafts 9.1 us, inlined 9.6; the
// part of 2,048 rows below 27 and 25).
template <int D, bool kRope>
__device__ __noinline__ void append_shared(const BlockAppendArgs &a, int shares, int qheads, int own,
                                           int idle_b, float4 *tab, uint64_t *freq) {
  __shared__ RunScan<kBcThreads> scan;
  __shared__ int idle[2];  // requests without pages: before this CTA's, and all
  const int first_shared = a.rg.B * shares;  // CTA
  int ctas = (static_cast<int>(gridDim.x) - first_shared) * gridDim.y;
  int cta = (static_cast<int>(blockIdx.x) - first_shared) * gridDim.y + blockIdx.y;
  if (idle_b >= 0) {
    if (threadIdx.x < 2) idle[threadIdx.x] = 0;
    bool any = false;
    int before = 0, all = 0;
    for (int k = threadIdx.x; k < a.rg.B; k += kBcThreads) {
      const int n = pages_touched(request_rows<true>(a.rg, k), a.c.ps);
      any |= n > own;
      all += n == 0;
      before += n == 0 && k < idle_b;
    }
    if (!__syncthreads_or(any)) return;
    atomicAdd(&idle[0], before);
    atomicAdd(&idle[1], all);
    __syncthreads();
    ctas = idle[1];
    cta = idle[0];
  }
  if constexpr (kRope)
    if (threadIdx.x < a.rope.rd / 2) freq[threadIdx.x] = turns_per_token(a.rope.inv_freq[threadIdx.x]);
  auto items = [&](const Rows &rq) -> int64_t {  // (page, share) pairs
    return static_cast<int64_t>(max(pages_touched(rq, a.c.ps) - own, 0)) * shares;
  };
  const RunStart r = find_run<kBcThreads>(a.rg.B, ctas, cta, scan,
                                          [&](int k) { return items(request_rows<true>(a.rg, k)); });
  int b = r.b;
  int64_t in = r.in;
  const ShortLane t = short_lane<D, kRope>(a);
  for (int64_t left = min(r.per, r.total - cta * r.per); left > 0; --left, ++in) {
    Rows rq = request_rows<true>(a.rg, b);
    while (in >= items(rq)) {
      in = 0;
      rq = request_rows<true>(a.rg, ++b);
    }
    const int page = static_cast<int>(in / shares);
    const ShortShare sh = short_share(a, static_cast<int>(in - static_cast<int64_t>(page) * shares), qheads, D);
    append_page<D, kRope>(a, sh, t, rq, b, own + page, tab, freq);
  }
}

// blockIdx.x below B * shares: request and share of its pages; blockIdx.y: its page, counting
// from the first that the step touches, and every gridDim.y-th one after it, up to `own` pages in
// all.  No scan over the requests: the time of a decode step is a chain of loads (starts and
// length; table entry beside the rows; old scale), and this is the shortest one.
// The pages beyond (a prompt's part among decode rows) are the other CTAs' (255 requests of one
// row and one of 2,048: 608 us without them, now 27).  A step of no more rows than requests has
// none; where one request has many rows all the same, others have no rows, and those requests'
// CTAs take their place (1,024 slots, one with a part of 1,000 rows and the others idle: 482 us
// without, now 21; 256 slots with 64 rows of decode 4.2 and 4.25).
// Three CTAs an SM with rotation, for its registers, and four without (rotated, 64 rows of 64
// requests 2.75 us against 3.05, 1,024 rows 16.7 against 16.3; as they come, 1,024 rows 9.4 and 7.8).
template <int D, bool kRope>
__global__ void __launch_bounds__(kBcThreads, kRope ? 3 : 4)
    block_append_short(const __grid_constant__ BlockAppendArgs a, int shares, int qheads, int own) {
  extern __shared__ float4 tab[];
  __shared__ uint64_t s_freq[kRope ? D / 2 : 1];
  const int rd = kRope ? a.rope.rd : D;
  const int first_shared = a.rg.B * shares;  // CTA
  const int b = blockIdx.x / shares, share = blockIdx.x - b * shares;
  const ShortShare sh = short_share(a, share, qheads, D);
  const ShortLane t = short_lane<D, kRope>(a);
  grid_dependency_wait();
  allow_dependents();
  if (static_cast<int>(blockIdx.x) >= first_shared) {
    append_shared<D, kRope>(a, shares, qheads, own, -1, tab, s_freq);
    return;
  }
  double freq = 0.0;
  if constexpr (kRope)
    if (share != 1 && threadIdx.x < rd / 2) freq = a.rope.inv_freq[threadIdx.x];  // rd / 2 <= blockDim
  const Rows rq = request_rows<true>(a.rg, b);
  if (rq.err && blockIdx.y == 0 && share == 0 && threadIdx.x == 0) report(a.err_word, rq.err);
  const int touched = pages_touched(rq, a.c.ps), pages = min(touched, own);
  if (static_cast<int>(blockIdx.y) >= pages) {
    if (touched == 0 && share == 0 && blockIdx.y == 0 && own < INT32_MAX &&
        static_cast<int>(gridDim.x) == first_shared)
      append_shared<D, kRope>(a, shares, qheads, own, b, tab, s_freq);
    return;
  }
  if constexpr (kRope)
    if (share != 1 && threadIdx.x < rd / 2) s_freq[threadIdx.x] = turns_per_token(freq);
  for (int pg = blockIdx.y; pg < pages; pg += gridDim.y)
    append_page<D, kRope>(a, sh, t, rq, b, pg, tab, s_freq);
}

// ---- prompts, a warp's rows loaded by itself

template <int D, bool kRope>
__global__ void __launch_bounds__(kBcThreads, kRope ? 2 : 3) block_append_wide(BlockAppendArgs a) {
  constexpr int kItems = D / 16;
  constexpr int kRpp = 32 / kItems;
  constexpr int kPasses = kRowsPerWarp / kRpp;
  extern __shared__ float4 tab[];
  __shared__ RunScan<kBcThreads> scan;
  __shared__ uint64_t s_freq[kRope ? D / 2 : 1];
  __shared__ float s_amax[2][kBcWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int P = a.c.P, H = a.c.H;
  const int i = lane % kItems, r0 = lane / kItems;
  const bool half = !kRope || a.rope.layout == KVQ_ROPE_HALF;
  const int rd = kRope ? a.rope.rd : D;
  const ItemChunks ch = item_chunks(i, D, rd, half);
  grid_dependency_wait();
  allow_dependents();
  if constexpr (kRope)
    if (threadIdx.x < rd / 2) s_freq[threadIdx.x] = turns_per_token(a.rope.inv_freq[threadIdx.x]);
  PageWalk walk = page_run<kBcThreads, true>(a.rg, a.c.ps, a.err_word, scan);
  PageItem it;
  uint32_t round = 0;
  while (next_page<true>(a.rg, a.block_table, a.MP, a.c.ps, a.c.num_pages, walk, it)) {  // uniform
    if (it.page < 0) {
      if (threadIdx.x == 0) report(a.err_word, KVQ_ERRBIT_PAGE);
      continue;
    }
    if constexpr (kRope) {
      __syncthreads();  // the previous item's angles are no longer read (and s_freq is set)
      fill_angles(tab, s_freq, it.first, it.nrow, rd, half, a.rope.mscale, threadIdx.x, kBcThreads);
      __syncthreads();
    }
    // warps a block: one takes up to 16 rows, more rows take one for each 16 slots
    const int team = it.nrow <= kRowsPerWarp ? 1 : P / kRowsPerWarp;
    const int sub = team == 1 ? 0 : warp % team;
    const int wbase = team == 1 ? it.slot0 : kRowsPerWarp * sub;
    const int lo = max(it.slot0, wbase), hi = min(it.slot0 + it.nrow, wbase + kRowsPerWarp);
    for (int u0 = 0; u0 < 2 * H; u0 += kBcWarps / team) {
      const int u = u0 + warp / team;  // (head, K or V)
      const bool live = u < 2 * H;
      const int h = u >> 1, is_v = u & 1;
      uint4 w[kPasses][2];
      if (live) {
        const uint16_t *src = (is_v ? a.v_new : a.k_new) + static_cast<int64_t>(h) * D;
        const int64_t stride = is_v ? a.v_stride : a.k_stride;
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
          const int slot = wbase + p * kRpp + r0;
          w[p][0] = w[p][1] = make_uint4(0, 0, 0, 0);
          if (slot >= lo && slot < hi) {
            const uint16_t *s = src + (it.row0 + slot - it.slot0) * stride;
            w[p][0] = __ldg(reinterpret_cast<const uint4 *>(s + ch.c0 * 8));
            w[p][1] = __ldg(reinterpret_cast<const uint4 *>(s + ch.c1 * 8));
          }
        }
      }
      const int64_t blk = static_cast<int64_t>(it.page) * H + h;
      const float s_old = live && it.slot0 > 0 ? a.c.scales[2 * blk + is_v] : 0.f;
      auto item = [&](int p, float (&y)[16]) {
        const int slot = wbase + p * kRpp + r0;
        unpack8(w[p][0], y);
        unpack8(w[p][1], y + 8);
        if constexpr (kRope)
          if (!is_v && slot >= lo && slot < hi)
            rotate_item(y, tab + (slot - it.slot0) * (rd / 4), i, rd, half, ch);
      };
      float amax = 0.f;
      if (live)
        amax = warp_amax([&](auto finite) {
          uint32_t m = 0;
#pragma unroll
          for (int p = 0; p < kPasses; ++p) {
            if (kRope && !is_v) {
              float y[16];
              item(p, y);
              m = max(m, item_max<decltype(finite)::value>(y));
            } else {
              m = max(m, words_max<decltype(finite)::value>(w[p][0], w[p][1]));
            }
          }
          return m;
        });
      if (team > 1) {  // uniform over the CTA
        // two buffers, taken in turn by the rounds that have this barrier and by no others:
        // a warp that writes one again has passed the barrier behind its last reads
        float *m = s_amax[round & 1];
        ++round;
        if (lane == 0) m[warp] = amax;
        __syncthreads();
        const int t0 = warp - sub;
        amax = fmaxf(m[t0], m[t0 + 1]);
        if (team == 4) amax = fmaxf(amax, fmaxf(m[t0 + 2], m[t0 + 3]));
      }
      if (!live) continue;
      const float s_new = fmaxf(pow2(block_exponent(amax)), s_old);
      const float inv = 1.0f / s_new;
      uint8_t *block = (is_v ? a.c.v : a.c.k) + blk * P * D;
      if (s_new > s_old && it.slot0 > 0) {  // this warp's old rows: its 16's, or all of them
        const int from = team == 1 ? 0 : wbase;
        requantise_rows<D>(block + from * D, min(it.slot0 - from, team == 1 ? P : kRowsPerWarp),
                           s_old / s_new, lane);
      }
      if (lane == 0 && sub == 0) a.c.scales[2 * blk + is_v] = s_new;
#pragma unroll
      for (int p = 0; p < kPasses; ++p) {
        const int slot = wbase + p * kRpp + r0;
        float y[16];
        item(p, y);
        if (slot >= lo && slot < hi) store_codes(block + slot * D, ch, y, inv);
      }
    }
    if constexpr (kRope) {
      const int total = it.nrow * a.Hq;
      for (int base = warp * kRpp; base < total; base += kBcWarps * kRpp) {
        const int e = base + r0, r = e / a.Hq;
        if (e >= total) continue;
        const int64_t col = static_cast<int64_t>(e - r * a.Hq) * D;
        const uint16_t *s = a.q + (it.row0 + r) * a.q_stride + col;
        const uint4 w0 = *reinterpret_cast<const uint4 *>(s + ch.c0 * 8);
        const uint4 w1 = *reinterpret_cast<const uint4 *>(s + ch.c1 * 8);
        float y[16];
        unpack8(w0, y);
        unpack8(w1, y + 8);
        rotate_item(y, tab + r * (rd / 4), i, rd, half, ch);
        store_rotated(a.q_out + (it.row0 + r) * a.q_out_stride + col, ch, y, w0, w1, i, D, rd, half);
      }
    }
  }
}

// ---- prompts, staged by TMA

constexpr int kRingMaxStages = 6;

// Ring stage: `rows` rows of heads h0 .. h0 + hg - 1 of K (0), V (1) or q (2).
struct RingStage {
  PageItem it;
  int what, h0;
};

struct RingCtl {
  RingStage st[kRingMaxStages];
  uint64_t full[kRingMaxStages], empty[kRingMaxStages];
  uint64_t sync;  // the consumer warps among themselves
  RunScan<kBcThreads + 32> scan;
  float amax[2][kBcWarps];
  int fail;
};

// A stage is what eight warps take at once: 16 rows of a head each.
template <int D>
struct RingCfg {
  static constexpr int STAGE = kBcWarps * kRowsPerWarp * D * 2;
};

// Stages that fit half an SM's shared memory beside the angles.
inline int ring_stages(int D, size_t angle_bytes) {
  const size_t stage = static_cast<size_t>(kBcWarps) * kRowsPerWarp * D * 2;
  const size_t n = (110 * 1024 - angle_bytes) / stage;
  return static_cast<int>(n < kRingMaxStages ? n : kRingMaxStages);
}

__device__ __forceinline__ bool ring_wait(RingCtl &ctl, uint64_t *bar, uint32_t parity,
                                          uint32_t *err_word) {
  bool ok = false;
  if (!*reinterpret_cast<volatile int *>(&ctl.fail)) {
    ok = mbar_wait(bar, parity);
    if (!ok && atomicExch(&ctl.fail, 1) == 0) report(err_word, KVQ_ERRBIT_TIMEOUT);
  }
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, int x, int y, int z,
                                            uint64_t *bar, uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar)), "l"(pol)
      : "memory");
}

// A barrier of the consumer warps, bounded like every wait.
__device__ __forceinline__ bool consumers_sync(RingCtl &ctl, uint32_t &phase, int lane,
                                               uint32_t *err_word) {
  __syncwarp();
  if (lane == 0) mbar_arrive(&ctl.sync);
  const bool ok = ring_wait(ctl, &ctl.sync, phase, err_word);
  phase ^= 1;
  return ok;
}

// hg heads of P rows make a stage (hg P = 128).  Dynamic shared memory: the
// ring of NS stages, then the angles.
template <int D, bool kRope>
__global__ void __launch_bounds__(kBcThreads + 32, 2)
    block_append_ring(const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap,
                      const __grid_constant__ CUtensorMap qmap, BlockAppendArgs a, int NS) {
  using C = RingCfg<D>;
  constexpr int kItems = D / 16, kRpp = 32 / kItems, kPasses = kRowsPerWarp / kRpp;
  extern __shared__ __align__(128) uint8_t ring[];
  float4 *tab = reinterpret_cast<float4 *>(ring + NS * C::STAGE);
  __shared__ RingCtl ctl;
  __shared__ uint64_t s_freq[kRope ? D / 2 : 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int P = a.c.P, H = a.c.H;
  const int team = P / kRowsPerWarp, hg = kBcWarps / team;
  const int rd = kRope ? a.rope.rd : D;
  if (threadIdx.x == 0) {
    for (int k = 0; k < NS; ++k) {
      mbar_init(&ctl.full[k], 1);
      mbar_init(&ctl.empty[k], kBcWarps);
    }
    mbar_init(&ctl.sync, kBcWarps);
    ctl.fail = 0;
    fence_barrier_init();
  }
  __syncthreads();
  grid_dependency_wait();
  allow_dependents();
  if constexpr (kRope)
    if (threadIdx.x < rd / 2) s_freq[threadIdx.x] = turns_per_token(a.rope.inv_freq[threadIdx.x]);
  PageWalk walk = page_run<kBcThreads + 32, true>(a.rg, a.c.ps, a.err_word, ctl.scan);  // syncs

  if (warp == kBcWarps) {
    // ------------------------------------------------------------ producer
    const uint64_t pol = policy_evict_first();
    uint32_t g = 0, par = 1;
    int slot = 0;
    bool ok = true;
    PageItem it;
    while (ok && next_page<true>(a.rg, a.block_table, a.MP, a.c.ps, a.c.num_pages, walk, it)) {
      if (it.page < 0) {
        if (lane == 0) report(a.err_word, KVQ_ERRBIT_PAGE);
        continue;
      }
      for (int what = 0; ok && what < (kRope && a.Hq > 0 ? 3 : 2); ++what) {
        const int heads = what == 2 ? a.Hq : H;
        for (int h0 = 0; h0 < heads; h0 += hg) {
          ok = ring_wait(ctl, &ctl.empty[slot], par, a.err_word);
          if (!ok) break;
          if (lane == 0) {
            ctl.st[slot] = {it, what, h0};
            mbar_arrive_expect_tx(&ctl.full[slot], C::STAGE);
            tma_load_3d(ring + slot * C::STAGE, what == 0 ? &kmap : what == 1 ? &vmap : &qmap, 0,
                        h0, static_cast<int>(it.row0), &ctl.full[slot], pol);
          }
          ++g;
          if (++slot == NS) {
            slot = 0;
            par ^= 1;
          }
          __syncwarp();
        }
      }
    }
    if (ok) ok = ring_wait(ctl, &ctl.empty[slot], par, a.err_word);
    if (lane == 0) {
      if (ok) {  // nothing more
        ctl.st[slot].what = -1;
        mbar_arrive(&ctl.full[slot]);
      } else {
        // a wait gave up: the copies in flight land before the CTA's shared
        // memory goes to another one
        for (uint32_t k = g > NS ? g - NS : 0; k < g; ++k)
          mbar_wait(&ctl.full[k % NS], (k / NS) & 1);
      }
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  const int i = lane % kItems, r0 = lane / kItems;
  const bool half = !kRope || a.rope.layout == KVQ_ROPE_HALF;
  const ItemChunks ch = item_chunks(i, D, rd, half);
  const int sub = warp % team, hw = warp / team;  // rows 16 sub .. of head hw of the stage
  const int rbase = kRowsPerWarp * sub + r0;
  uint32_t par = 0, phase = 0, round = 0;
  int slot = 0;
  while (true) {
    if (!ring_wait(ctl, &ctl.full[slot], par, a.err_word)) return;
    const RingStage st = ctl.st[slot];
    if (st.what < 0) return;
    const PageItem &it = st.it;
    if (kRope && st.what == 0 && st.h0 == 0) {  // a page begins
      if (!consumers_sync(ctl, phase, lane, a.err_word)) return;  // the last one's angles are read
      fill_angles(tab, s_freq, it.first, it.nrow, rd, half, a.rope.mscale, threadIdx.x, kBcThreads);
      if (!consumers_sync(ctl, phase, lane, a.err_word)) return;
    }
    const int h = st.h0 + hw;
    const bool live = h < (st.what == 2 ? a.Hq : H);
    uint4 w[kPasses][2];
    const uint8_t *src = ring + slot * C::STAGE;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const uint8_t *s = src + ((rbase + p * kRpp) * hg + hw) * (2 * D);
      w[p][0] = *reinterpret_cast<const uint4 *>(s + ch.c0 * 16);
      w[p][1] = *reinterpret_cast<const uint4 *>(s + ch.c1 * 16);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&ctl.empty[slot]);
    if (++slot == NS) {
      slot = 0;
      par ^= 1;
    }
    auto item = [&](int p, float (&y)[16]) {
      const int r = rbase + p * kRpp;
      unpack8(w[p][0], y);
      unpack8(w[p][1], y + 8);
      if constexpr (kRope)
        if (st.what != 1 && r < it.nrow) rotate_item(y, tab + r * (rd / 4), i, rd, half, ch);
    };
    if (kRope && st.what == 2) {
      if (!live) continue;
#pragma unroll
      for (int p = 0; p < kPasses; ++p) {
        const int r = rbase + p * kRpp;
        float y[16];
        item(p, y);
        if (r < it.nrow)
          store_rotated(a.q_out + (it.row0 + r) * a.q_out_stride + static_cast<int64_t>(h) * D, ch,
                        y, w[p][0], w[p][1], i, D, rd, half);
      }
      continue;
    }
    const bool is_v = st.what == 1;
    const int64_t blk = static_cast<int64_t>(it.page) * H + h;
    const float s_old = live && it.slot0 > 0 ? a.c.scales[2 * blk + is_v] : 0.f;
    float amax = warp_amax([&](auto finite) {
      uint32_t m = 0;
#pragma unroll
      for (int p = 0; p < kPasses; ++p) {
        if (rbase + p * kRpp >= it.nrow) continue;  // rows of others
        if (kRope && !is_v) {
          float y[16];
          item(p, y);
          m = max(m, item_max<decltype(finite)::value>(y));
        } else {
          m = max(m, words_max<decltype(finite)::value>(w[p][0], w[p][1]));
        }
      }
      return m;
    });
    if (team > 1) {  // uniform over the grid
      float *m = ctl.amax[round & 1];
      ++round;
      if (lane == 0) m[warp] = amax;
      if (!consumers_sync(ctl, phase, lane, a.err_word)) return;
      const int t0 = warp - sub;
      amax = fmaxf(m[t0], m[t0 + 1]);
      if (team == 4) amax = fmaxf(amax, fmaxf(m[t0 + 2], m[t0 + 3]));
    }
    if (!live) continue;
    const float s_new = fmaxf(pow2(block_exponent(amax)), s_old);
    const float inv = 1.0f / s_new;
    uint8_t *block = (is_v ? a.c.v : a.c.k) + blk * P * D;
    if (sub == 0) {
      if (s_new > s_old && it.slot0 > 0) requantise_rows<D>(block, it.slot0, s_old / s_new, lane);
      if (lane == 0) a.c.scales[2 * blk + is_v] = s_new;
    }
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int r = rbase + p * kRpp;
      float y[16];
      item(p, y);
      if (r < it.nrow) store_codes(block + (it.slot0 + r) * D, ch, y, inv);
    }
  }
}

// ---------------------------------------------------------------------------
// reading back
// ---------------------------------------------------------------------------

struct BlockReadArgs {
  BlockPool c;
  Ragged rg;
  const int32_t *block_table;
  uint32_t *err_word;
  uint16_t *k_out, *v_out;
  int64_t k_stride, v_stride;
  int32_t MP;
};

// A warp takes 16 rows of one head's K or V in one page: 8 codes a lane and
// load, 8 bf16 a lane and store, both contiguous over a row.  Bandwidth-bound
// (D (1 + 2) bytes a token, head and tensor); the code times a power-of-two
// scale is exact in bf16, so nothing is rounded.
template <int D>
__global__ void __launch_bounds__(kBcThreads) block_read_kernel(BlockReadArgs a) {
  constexpr int kLanes = D / 8;
  constexpr int kRpp = 32 / kLanes;
  constexpr int kPasses = kRowsPerWarp / kRpp;
  __shared__ RunScan<kBcThreads> scan;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int P = a.c.P, H = a.c.H;
  const int i = lane % kLanes, r0 = lane / kLanes;
  grid_dependency_wait();
  allow_dependents();
  PageWalk walk = page_run<kBcThreads, false>(a.rg, a.c.ps, a.err_word, scan);
  PageItem it;
  while (next_page<false>(a.rg, a.block_table, a.MP, a.c.ps, a.c.num_pages, walk, it)) {
    if (it.page < 0) {
      if (threadIdx.x == 0) report(a.err_word, KVQ_ERRBIT_PAGE);
      continue;
    }
    const int slot0 = it.slot0, nrow = it.nrow;
    const int team = P / kRowsPerWarp;
    for (int u = warp; u < 2 * H * team; u += kBcWarps) {
      // neighbouring warps take neighbouring heads: whole rows are written together
      const int h = u % H, sub = (u / H) % team, is_v = u / (H * team);
      const int64_t blk = static_cast<int64_t>(it.page) * H + h;
      const uint8_t *src = (is_v ? a.c.v : a.c.k) + blk * P * D;
      uint2 w[kPasses];
#pragma unroll
      for (int p = 0; p < kPasses; ++p) {
        const int slot = kRowsPerWarp * sub + p * kRpp + r0;
        w[p] = make_uint2(0, 0);
        if (slot >= slot0 && slot < slot0 + nrow)
          w[p] = __ldg(reinterpret_cast<const uint2 *>(src + slot * D) + i);
      }
      const float s = __ldg(a.c.scales + 2 * blk + is_v);
      uint16_t *dst = (is_v ? a.v_out : a.k_out) + static_cast<int64_t>(h) * D + i * 8;
      const int64_t stride = is_v ? a.v_stride : a.k_stride;
#pragma unroll
      for (int p = 0; p < kPasses; ++p) {
        const int slot = kRowsPerWarp * sub + p * kRpp + r0;
        if (slot >= slot0 && slot < slot0 + nrow) {
          float x[8];
          e4m3x4_to_f32(w[p].x, x);
          e4m3x4_to_f32(w[p].y, x + 4);
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] *= s;
          *reinterpret_cast<uint4 *>(dst + (it.row0 + slot - slot0) * stride) = pack8(x);
        }
      }
    }
  }
}

namespace {

BlockPool block_pool(const kvq_block_cache *c) {
  return {static_cast<uint8_t *>(c->k_pool), static_cast<uint8_t *>(c->v_pool), c->scales,
          c->num_pages, c->page_size, c->num_kv_heads, c->page_size == 16 ? 4 : c->page_size == 32 ? 5 : 6};
}

// Pages that a step of n_tokens rows touches, at most: one a row, and
// n_tokens / P + 2 a request.
int64_t max_pages(int64_t n_tokens, int64_t B, int P) {
  const int64_t n = n_tokens / P + 2 * B;
  return n < n_tokens ? n : n_tokens;
}

int block_ctas(int64_t items, int per_sm, int sms) {
  const int64_t most = static_cast<int64_t>(per_sm) * sms;
  return static_cast<int>(items < most ? items : most);
}

// Rows a request, on average, up to which a step takes the short kernel.
constexpr int kShortRows = 16;

// [tokens][heads][D] bf16, strided by token; a box is P rows of hg heads.
bool rows_map(CUtensorMap *map, const void *p, int64_t stride, int64_t tokens, int heads, int D,
              int hg, int P) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(tokens)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(stride) * 2};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(D), static_cast<cuuint32_t>(hg),
                             static_cast<cuuint32_t>(P)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(p), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

using RingFn = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, BlockAppendArgs, int);

// Opt a ring kernel into its shared memory, once per device.
bool ring_opt_in(RingFn fn, int variant) {
  constexpr int kMaxDev = 64;
  static std::atomic<bool> done[kMaxDev][4];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return false;
  if (done[dev][variant].load(std::memory_order_acquire)) return true;
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 112 * 1024) != cudaSuccess)
    return false;
  done[dev][variant].store(true, std::memory_order_release);
  return true;
}

kvq_status append_impl(const kvq_block_cache *cache, const kvq_rope_desc *rope, const void *q,
                       int64_t q_stride, void *q_out, int64_t q_out_stride, int32_t Hq,
                       const void *k_new, int64_t k_stride, const void *v_new, int64_t v_stride,
                       const int32_t *tok_start, int32_t n_tokens, const int32_t *seq_lens,
                       const int32_t *block_table, int32_t B, int32_t MP, uint32_t *err_word,
                       kvq_stream_t stream) {
  kvq_status st = validate_block_cache(cache);
  if (st != KVQ_OK) return st;
  const int D = cache->head_dim;
  if (rope && (st = validate_rope(rope, D)) != KVQ_OK) return st;
  st = validate_ragged(tok_start, n_tokens, block_table, B, MP, cache->page_size);
  if (st != KVQ_OK) return st;
  if (Hq < 0) return KVQ_ERR_INVALID_ARG;
  if (n_tokens == 0 || B == 0) return KVQ_OK;
  if (!seq_lens || !rows_ok(k_new, k_stride, cache->num_kv_heads, D) ||
      !rows_ok(v_new, v_stride, cache->num_kv_heads, D))
    return KVQ_ERR_INVALID_ARG;
  if (Hq > 0 && (!rows_ok(q, q_stride, Hq, D) || !rows_ok(q_out, q_out_stride, Hq, D)))
    return KVQ_ERR_INVALID_ARG;
  BlockAppendArgs a;
  a.c = block_pool(cache);
  a.rg = {tok_start, seq_lens, B, n_tokens, static_cast<int64_t>(MP) * cache->page_size};
  a.block_table = block_table;
  a.err_word = err_word;
  a.k_new = static_cast<const uint16_t *>(k_new);
  a.v_new = static_cast<const uint16_t *>(v_new);
  a.q = static_cast<const uint16_t *>(q);
  a.q_out = static_cast<uint16_t *>(q_out);
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_stride = q_stride;
  a.q_out_stride = q_out_stride;
  a.MP = MP;
  a.Hq = Hq;
  a.rope = rope ? RopeArgs{rope->inv_freq, rope->rotary_dim, rope->layout, rope->mscale}
                : RopeArgs{nullptr, D, KVQ_ROPE_HALF, 1.f};
  int sms = 0;
  if (device_sm_count(&sms) != KVQ_OK) return KVQ_ERR_CUDA;
  const int P = cache->page_size, H = cache->num_kv_heads;
  const size_t angles = rope ? static_cast<size_t>(P) * rope->rotary_dim * 4 : 0;
  const int64_t pages = max_pages(n_tokens, B, P);
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (n_tokens <= kShortRows * static_cast<int64_t>(B) || pages <= 2 * sms) {
    // q's heads in one share for up to two rows a request, in shares of twice K's rows for
    // more (256 drafts of 1-8 rows, 32 heads over 8: 9.1 us, shares of 8 and of all heads 11.0
    // and 8.9; four parts of 300 rows 9.8, with all heads 14.8)
    const int qheads = n_tokens <= 2 * static_cast<int64_t>(B) ? Hq : 2 * H;
    const int shares = rope && Hq > 0 ? 2 + (Hq + qheads - 1) / qheads : 2;
    if (static_cast<int64_t>(B) * shares > INT32_MAX - 4 * sms) return KVQ_ERR_UNSUPPORTED;
    // pages a request that get CTAs of their own: what an average one fills,
    // up to 16 CTAs an SM in all
    const int64_t avg = (n_tokens + B - 1) / B;
    int64_t gy = (avg + P - 1) / P;
    const int64_t most = 16LL * sms / (static_cast<int64_t>(B) * shares) + 1;
    gy = gy < most ? gy : most;
    // a request's own CTAs do two pages each; what one can have beyond is shared: by further
    // CTAs, or by those of requests without rows, which there are where the rows are no more
    // than the requests and one has many
    const int64_t beyond = (static_cast<int64_t>(n_tokens) + P - 2) / P + 1 - 2 * gy;
    const bool shared = beyond > 0 && tok_start;
    const int own = shared ? 2 * static_cast<int>(gy) : INT32_MAX;
    const int64_t extra =
        shared && n_tokens > B ? (std::min<int64_t>(beyond * shares, 3 * sms) + gy - 1) / gy : 0;
    using ShortFn = void (*)(BlockAppendArgs, int, int, int);
    static constexpr ShortFn kFns[2][2] = {{block_append_short<64, false>, block_append_short<64, true>},
                                           {block_append_short<128, false>, block_append_short<128, true>}};
    e = launch_dependent(kFns[D == 128][rope != nullptr],
                         dim3(static_cast<unsigned>(B * shares + extra), static_cast<unsigned>(gy)), kBcThreads,
                         angles, cs, a, shares, qheads, own);
  } else if (H * P >= kBcWarps * kRowsPerWarp) {
    const auto fn = D == 128 ? (rope ? block_append_ring<128, true> : block_append_ring<128, false>)
                             : (rope ? block_append_ring<64, true> : block_append_ring<64, false>);
    const int ns = ring_stages(D, angles), hg = kBcWarps * kRowsPerWarp / P;
    const size_t smem = static_cast<size_t>(ns) * kBcWarps * kRowsPerWarp * D * 2 + angles;
    if (!ring_opt_in(fn, (D == 128 ? 2 : 0) + (rope ? 1 : 0))) return KVQ_ERR_CUDA;
    CUtensorMap km, vm, qm;
    if (!rows_map(&km, k_new, k_stride, n_tokens, H, D, hg, P) ||
        !rows_map(&vm, v_new, v_stride, n_tokens, H, D, hg, P))
      return KVQ_ERR_CUDA;
    qm = km;
    if (Hq > 0 && !rows_map(&qm, q, q_stride, n_tokens, Hq, D, hg, P)) return KVQ_ERR_CUDA;
    e = launch_dependent(fn, block_ctas(pages, 2, sms), kBcThreads + 32, smem, cs, km, vm, qm, a, ns);
  } else {
    const auto fn = D == 128 ? (rope ? block_append_wide<128, true> : block_append_wide<128, false>)
                             : (rope ? block_append_wide<64, true> : block_append_wide<64, false>);
    e = launch_dependent(fn, block_ctas(pages, rope ? 2 : 3, sms), kBcThreads, angles, cs, a);
  }
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

}  // namespace

}  // namespace kvq

using namespace kvq;

extern "C" kvq_status kvq_block_append(const kvq_block_cache *cache, const void *k_new,
                                       int64_t k_stride, const void *v_new, int64_t v_stride,
                                       const int32_t *tok_start, int32_t n_tokens,
                                       const int32_t *seq_lens, const int32_t *block_table,
                                       int32_t B, int32_t MP, uint32_t *err_word,
                                       kvq_stream_t stream) {
  return append_impl(cache, nullptr, nullptr, 0, nullptr, 0, 0, k_new, k_stride, v_new, v_stride,
                     tok_start, n_tokens, seq_lens, block_table, B, MP, err_word, stream);
}

extern "C" kvq_status kvq_rope_block_append(const kvq_block_cache *cache,
                                            const kvq_rope_desc *rope, const void *q,
                                            int64_t q_stride, void *q_out, int64_t q_out_stride,
                                            int32_t n_q_heads, const void *k_new,
                                            int64_t k_stride, const void *v_new, int64_t v_stride,
                                            const int32_t *tok_start, int32_t n_tokens,
                                            const int32_t *seq_lens, const int32_t *block_table,
                                            int32_t B, int32_t MP, uint32_t *err_word,
                                            kvq_stream_t stream) {
  if (!rope) return KVQ_ERR_INVALID_ARG;
  return append_impl(cache, rope, q, q_stride, q_out, q_out_stride, n_q_heads, k_new, k_stride,
                     v_new, v_stride, tok_start, n_tokens, seq_lens, block_table, B, MP, err_word,
                     stream);
}

extern "C" kvq_status kvq_block_read(const kvq_block_cache *cache, const int32_t *tok_start,
                                     int32_t n_tokens, const int32_t *first,
                                     const int32_t *block_table, int32_t B, int32_t MP,
                                     void *k_out, int64_t k_stride, void *v_out, int64_t v_stride,
                                     uint32_t *err_word, kvq_stream_t stream) {
  kvq_status st = validate_block_cache(cache);
  if (st != KVQ_OK) return st;
  const int D = cache->head_dim;
  st = validate_ragged(tok_start, n_tokens, block_table, B, MP, cache->page_size);
  if (st != KVQ_OK) return st;
  if (n_tokens == 0 || B == 0) return KVQ_OK;
  if (!rows_ok(k_out, k_stride, cache->num_kv_heads, D) ||
      !rows_ok(v_out, v_stride, cache->num_kv_heads, D))
    return KVQ_ERR_INVALID_ARG;
  BlockReadArgs a;
  a.c = block_pool(cache);
  a.rg = {tok_start, first, B, n_tokens, static_cast<int64_t>(MP) * cache->page_size};
  a.block_table = block_table;
  a.err_word = err_word;
  a.k_out = static_cast<uint16_t *>(k_out);
  a.v_out = static_cast<uint16_t *>(v_out);
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.MP = MP;
  int sms = 0;
  if (device_sm_count(&sms) != KVQ_OK) return KVQ_ERR_CUDA;
  // many short runs of pages keep more rows in flight than a few long ones (48
  // ragged prefixes: 230 us with 8 CTAs an SM, 215 with 32); a large batch, which
  // every CTA scans, takes fewer
  const int ctas = block_ctas(max_pages(n_tokens, B, cache->page_size), B <= 4096 ? 32 : 8, sms);
  const cudaError_t e =
      launch_dependent(D == 128 ? block_read_kernel<128> : block_read_kernel<64>, ctas, kBcThreads,
                       0, reinterpret_cast<cudaStream_t>(stream), a);
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}
