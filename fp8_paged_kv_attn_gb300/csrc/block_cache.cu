// kvq_block_append, kvq_rope_block_append, kvq_block_read: writing the
// block-scaled cache (rotation, scale, quantisation in one pass) and reading
// it back.
//
// Mathematics: include/kvq.h.  Work item: one (request, page) that the step
// touches, with all kv heads; every CTA scans the requests once and takes an
// equal run of items (find_run), so that one prompt among decode tokens
// does not leave the other SMs idle.
//
// Append: a warp takes 16 rows (tokens) of one head's K or V in one page, so
// the 16 x D values stay in registers between the maximum that sets the scale
// and the conversion: K and V are read once.  A 64-token page's block is four
// warps, which exchange their maxima through shared memory.  The page's
// angles are computed once into shared memory for all heads and q.
// Bandwidth-bound on prompts (2 D (2 + 1) bytes a token and kv head);
// latency-bound on a decode step.
#include "block_common.cuh"

namespace kvq {

constexpr int kBcThreads = 256;
constexpr int kBcWarps = kBcThreads / 32;
constexpr int kRowsPerWarp = 16;

struct BlockPool {
  uint8_t *k, *v;
  float *scales;
  int32_t num_pages, P, H;
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
__device__ __forceinline__ int64_t pages_touched(const Rows &r, int P) {
  return r.n == 0 || r.err ? 0 : (r.p0 + r.n - 1) / P - r.p0 / P + 1;
}

// Old codes of a block whose scale grew: rows [0, n_old) of this warp's 16.
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

template <int D, bool kRope>
__global__ void __launch_bounds__(kBcThreads, 2) block_append_kernel(BlockAppendArgs a) {
  constexpr int kItems = D / 16;           // lanes a row (two 8-dim chunks each)
  constexpr int kRpp = 32 / kItems;        // rows a pass of a warp
  constexpr int kPasses = kRowsPerWarp / kRpp;
  extern __shared__ float4 tab[];          // kRope: [P][rd / 4] angles of the page's rows
  __shared__ RunScan<kBcThreads> scan;
  __shared__ uint64_t s_freq[kRope ? D / 2 : 1];
  __shared__ float s_amax[2][kBcWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int P = a.c.P, H = a.c.H;
  const int team = P / kRowsPerWarp;       // warps a block: 1, 2 or 4
  const int sub = warp % team;             // this warp's 16 rows of the block
  const int i = lane % kItems, r0 = lane / kItems;
  const bool half = !kRope || a.rope.layout == KVQ_ROPE_HALF;
  const int rd = kRope ? a.rope.rd : D;
  const ItemChunks ch = item_chunks(i, D, rd, half);
  grid_dependency_wait();
  allow_dependents();
  if constexpr (kRope) {
    for (int j = threadIdx.x; j < rd / 2; j += kBcThreads)
      s_freq[j] = turns_per_token(a.rope.inv_freq[j]);
  }
  const RunStart run = find_run<kBcThreads>(
      a.rg.B, gridDim.x, blockIdx.x, scan, [&](int b) -> int64_t {
        const Rows r = request_rows<true>(a.rg, b);
        if (r.err && blockIdx.x == 0) report(a.err_word, r.err);
        return pages_touched(r, P);
      });
  int64_t left = min(run.per, run.total - blockIdx.x * run.per);
  int b = run.b;
  int64_t in = run.in;
  uint32_t round = 0;
  while (left > 0) {  // uniform over the CTA
    const Rows rq = request_rows<true>(a.rg, b);
    const int64_t have = pages_touched(rq, P);
    if (in >= have) {
      ++b;
      in = 0;
      continue;
    }
    const int lp = rq.p0 / P + static_cast<int>(in);
    ++in;
    --left;
    const int first = max(rq.p0, lp * P);              // the item's positions
    const int last = min(rq.p0 + rq.n, lp * P + P);    // [first, last)
    const int row0 = rq.row + (first - rq.p0);
    const int slot0 = first - lp * P, nrow = last - first;
    const int page = __ldg(a.block_table + static_cast<int64_t>(b) * a.MP + lp);
    if (page < 0 || page >= a.c.num_pages) {
      if (threadIdx.x == 0) report(a.err_word, KVQ_ERRBIT_PAGE);
      continue;
    }
    if constexpr (kRope) {
      __syncthreads();  // the previous item's angles are no longer read (and s_freq is set)
      for (int j = threadIdx.x; j < nrow * (rd / 4); j += kBcThreads) {
        const int r = j / (rd / 4), q = j % (rd / 4);
        const float2 x = rotation(first + r, s_freq[2 * q], a.rope.mscale);
        const float2 y = rotation(first + r, s_freq[2 * q + 1], a.rope.mscale);
        tab[r * (rd / 4) + angle_slot(q, rd, half)] = make_float4(x.x, x.y, y.x, y.y);
      }
      __syncthreads();
    }
    // this warp's rows of the page: slots [16 sub, 16 sub + 16)
    const int lo = max(slot0, kRowsPerWarp * sub), hi = min(slot0 + nrow, kRowsPerWarp * (sub + 1));
    const int units = 2 * H, step = kBcWarps / team;
    for (int u0 = 0; u0 < units; u0 += step, ++round) {
      const int u = u0 + warp / team;  // (head, K or V)
      const bool live = u < units;
      const int h = u >> 1, is_v = u & 1;
      uint4 w[kPasses][2];
      float amax = 0.f;
      if (live) {
        const uint16_t *src = (is_v ? a.v_new : a.k_new) + static_cast<int64_t>(h) * D;
        const int64_t stride = is_v ? a.v_stride : a.k_stride;
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
          const int slot = kRowsPerWarp * sub + p * kRpp + r0;
          w[p][0] = w[p][1] = make_uint4(0, 0, 0, 0);
          if (slot >= lo && slot < hi) {
            const uint16_t *s = src + (row0 + slot - slot0) * stride;
            w[p][0] = __ldg(reinterpret_cast<const uint4 *>(s + ch.c0 * 8));
            w[p][1] = __ldg(reinterpret_cast<const uint4 *>(s + ch.c1 * 8));
          }
        }
      }
      const int64_t blk = static_cast<int64_t>(page) * H + h;
      const float s_old = live && slot0 > 0 ? a.c.scales[2 * blk + is_v] : 0.f;
      // rotated K values are needed twice (maximum, conversion): kept in fp32
      float x[kRope ? kPasses : 1][16];
      if constexpr (kRope) {
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
          const int slot = kRowsPerWarp * sub + p * kRpp + r0;
          unpack8(w[p][0], x[p]);
          unpack8(w[p][1], x[p] + 8);
          if (!is_v && slot >= lo && slot < hi)
            rotate_item(x[p], tab + (slot - slot0) * (rd / 4), i, rd, half, ch);
#pragma unroll
          for (int j = 0; j < 16; ++j) amax = fmaxf(amax, finite_abs(x[p][j]));
        }
      } else {
#pragma unroll
        for (int p = 0; p < kPasses; ++p)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float y[8];
            unpack8(w[p][c], y);
#pragma unroll
            for (int j = 0; j < 8; ++j) amax = fmaxf(amax, finite_abs(y[j]));
          }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      if (team > 1) {  // uniform over the grid
        float *m = s_amax[round & 1];
        if (lane == 0) m[warp] = amax;
        __syncthreads();
        const int t0 = warp - sub;
        amax = fmaxf(m[t0], m[t0 + 1]);
        if (team == 4) amax = fmaxf(amax, fmaxf(m[t0 + 2], m[t0 + 3]));
      }
      if (!live) continue;
      const float s_new = fmaxf(pow2(block_exponent(amax)), s_old);
      const float inv = 1.0f / s_new;  // exact: a power of two
      uint8_t *block = (is_v ? a.c.v : a.c.k) + blk * P * D;
      if (s_new > s_old && slot0 > kRowsPerWarp * sub)
        requantise_rows<D>(block + static_cast<int64_t>(kRowsPerWarp * sub) * D,
                           min(slot0 - kRowsPerWarp * sub, kRowsPerWarp), s_old / s_new, lane);
      if (sub == 0 && lane == 0) a.c.scales[2 * blk + is_v] = s_new;
#pragma unroll
      for (int p = 0; p < kPasses; ++p) {
        const int slot = kRowsPerWarp * sub + p * kRpp + r0;
        if (slot >= lo && slot < hi) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float y[8];
            if constexpr (kRope) {
#pragma unroll
              for (int j = 0; j < 8; ++j) y[j] = x[p][8 * c + j];
            } else {
              unpack8(w[p][c], y);
            }
            uint32_t o[2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
              o[j] = static_cast<uint32_t>(f32x2_to_e4m3x2(y[4 * j] * inv, y[4 * j + 1] * inv)) |
                     (static_cast<uint32_t>(f32x2_to_e4m3x2(y[4 * j + 2] * inv,
                                                            y[4 * j + 3] * inv))
                      << 16);
            *reinterpret_cast<uint2 *>(block + slot * D + (c ? ch.c1 : ch.c0) * 8) =
                make_uint2(o[0], o[1]);
          }
        }
      }
    }
    if constexpr (kRope) {
      // q: rows of (token, head), kRpp a warp pass
      const int total = nrow * a.Hq;
      for (int base = warp * kRpp; base < total; base += kBcWarps * kRpp) {
        const int e = base + r0;
        if (e >= total) continue;
        const int r = e / a.Hq, h = e % a.Hq;
        const uint16_t *s = a.q + (row0 + r) * a.q_stride + static_cast<int64_t>(h) * D;
        uint16_t *d = a.q_out + (row0 + r) * a.q_out_stride + static_cast<int64_t>(h) * D;
        const uint4 w0 = *reinterpret_cast<const uint4 *>(s + ch.c0 * 8);
        const uint4 w1 = *reinterpret_cast<const uint4 *>(s + ch.c1 * 8);
        float x[16];
        unpack8(w0, x);
        unpack8(w1, x + 8);
        rotate_item(x, tab + r * (rd / 4), i, rd, half, ch);
        const int lim = half ? (i < rd / 16 ? D / 8 : 0) : rd / 8;
        *reinterpret_cast<uint4 *>(d + ch.c0 * 8) = ch.c0 < lim ? pack8(x) : w0;
        *reinterpret_cast<uint4 *>(d + ch.c1 * 8) = ch.c1 < lim ? pack8(x + 8) : w1;
      }
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
  const RunStart run = find_run<kBcThreads>(
      a.rg.B, gridDim.x, blockIdx.x, scan, [&](int b) -> int64_t {
        const Rows r = request_rows<false>(a.rg, b);
        if (r.err && blockIdx.x == 0) report(a.err_word, r.err);
        return pages_touched(r, P);
      });
  int64_t left = min(run.per, run.total - blockIdx.x * run.per);
  int b = run.b;
  int64_t in = run.in;
  while (left > 0) {
    const Rows rq = request_rows<false>(a.rg, b);
    const int64_t have = pages_touched(rq, P);
    if (in >= have) {
      ++b;
      in = 0;
      continue;
    }
    const int lp = rq.p0 / P + static_cast<int>(in);
    ++in;
    --left;
    const int first = max(rq.p0, lp * P), last = min(rq.p0 + rq.n, lp * P + P);
    const int slot0 = first - lp * P, nrow = last - first;
    const int64_t row0 = rq.row + (first - rq.p0);
    const int page = __ldg(a.block_table + static_cast<int64_t>(b) * a.MP + lp);
    if (page < 0 || page >= a.c.num_pages) {
      if (threadIdx.x == 0) report(a.err_word, KVQ_ERRBIT_PAGE);
      continue;
    }
    const int team = P / kRowsPerWarp;
    for (int u = warp; u < 2 * H * team; u += kBcWarps) {
      const int sub = u % team, h = (u / team) >> 1, is_v = (u / team) & 1;
      const int64_t blk = static_cast<int64_t>(page) * H + h;
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
          *reinterpret_cast<uint4 *>(dst + (row0 + slot - slot0) * stride) = pack8(x);
        }
      }
    }
  }
}

namespace {

BlockPool block_pool(const kvq_block_cache *c) {
  return {static_cast<uint8_t *>(c->k_pool), static_cast<uint8_t *>(c->v_pool), c->scales,
          c->num_pages, c->page_size, c->num_kv_heads};
}

// CTAs for a step of n_tokens rows: it touches at most one page a row, and at
// most n_tokens / P + 2 B pages; `per_sm` CTAs an SM at most.
int block_ctas(int64_t n_tokens, int64_t B, int P, int per_sm, int sms) {
  int64_t n = n_tokens / P + 2 * B;
  n = n < n_tokens ? n : n_tokens;
  const int64_t most = static_cast<int64_t>(per_sm) * sms;
  return static_cast<int>(n < most ? n : most);
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
  const int ctas = block_ctas(n_tokens, B, cache->page_size, 2, sms);
  // at most 64 rows x 32 words = 32 KB of angles
  const size_t smem = rope ? static_cast<size_t>(cache->page_size) * rope->rotary_dim * 4 : 0;
  const auto fn = D == 128 ? (rope ? block_append_kernel<128, true> : block_append_kernel<128, false>)
                           : (rope ? block_append_kernel<64, true> : block_append_kernel<64, false>);
  const cudaError_t e = launch_dependent(fn, ctas, kBcThreads, smem,
                                         reinterpret_cast<cudaStream_t>(stream), a);
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
  const int ctas = block_ctas(n_tokens, B, cache->page_size, 8, sms);
  const cudaError_t e =
      launch_dependent(D == 128 ? block_read_kernel<128> : block_read_kernel<64>, ctas, kBcThreads,
                       0, reinterpret_cast<cudaStream_t>(stream), a);
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}
