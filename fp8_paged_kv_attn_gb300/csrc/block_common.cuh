// What the block-scaled cache's kernels share: checks and walking of a ragged
// step, block scales, and rotary angles.
#pragma once

#include <cmath>

#include "kvq_internal.h"

namespace kvq {

// ---------------------------------------------------------------------------
// ragged steps
// ---------------------------------------------------------------------------

// Which rows and positions each request has (include/kvq.h, "Ragged steps").
struct Ragged {
  const int32_t *tok_start;  // [B+1] or null: one row a request
  const int32_t *at;         // [B]: length after the step, or (first) where the rows start; may
                             // be null for `first`
  int32_t B, n_tokens;
  int64_t cap;               // MP * page_size
};

// One request's rows: n of them from row `row`, at positions p0, p0 + 1, ...
struct Rows {
  int row, n, p0;
  uint32_t err;  // KVQ_ERRBIT_* of a request that is left out (n rows are still its own)
};

// kLens: `at` holds lengths after the step; else first positions.
template <bool kLens>
__device__ __forceinline__ Rows request_rows(const Ragged &r, int b) {
  Rows o;
  const int s0 = r.tok_start ? __ldg(r.tok_start + b) : b;
  const int s1 = r.tok_start ? __ldg(r.tok_start + b + 1) : b + 1;
  const int at = r.at ? __ldg(r.at + b) : 0;
  o.row = s0;
  o.n = s1 - s0;
  o.err = 0;
  if (s0 < 0 || s1 < s0 || s1 > r.n_tokens) {
    o.n = 0;
    o.p0 = 0;
    o.err = KVQ_ERRBIT_REQ;
    return o;
  }
  if (o.n == 0) {
    o.p0 = 0;
    return o;
  }
  if (kLens) {
    o.p0 = at - o.n;
    if (at < o.n || at > r.cap) o.err = KVQ_ERRBIT_SEQLEN;
  } else {
    o.p0 = at;
    if (at < 0 || static_cast<int64_t>(at) + o.n > r.cap) o.err = KVQ_ERRBIT_POS;
  }
  return o;
}

// Where one CTA's run of work items starts: `total` items over all requests
// are cut into runs of `per` items, CTA c taking items c * per, ...; the first
// of them is item `in` of request `b`.
struct RunStart {
  int64_t total, per, in;
  int b;
};

template <int NT>
struct RunScan {  // shared memory of find_run
  int64_t sum[NT / 32], in;
  int b;
};

// Every thread of the CTA calls it (NT threads).  items(b) is request b's item
// count; a thread counts a contiguous set of requests, so that any number of
// them takes one block scan, and the one thread whose set holds the CTA's
// first item walks its set once more.
template <int NT, typename Items>
__device__ __forceinline__ RunStart find_run(int B, int ctas, int cta, RunScan<NT> &scan,
                                             Items items) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (B + NT - 1) / NT;
  const int64_t b0l = min(static_cast<int64_t>(tid) * per, static_cast<int64_t>(B));
  const int b0 = static_cast<int>(b0l), b1 = static_cast<int>(min(b0l + per, static_cast<int64_t>(B)));
  int64_t sum = 0;
  for (int b = b0; b < b1; ++b) sum += items(b);
  int64_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) scan.sum[warp] = incl;
  __syncthreads();
  int64_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) before += scan.sum[w];
    total += scan.sum[w];
  }
  RunStart r;
  r.total = total;
  r.per = max(static_cast<int64_t>(1), (total + ctas - 1) / ctas);
  const int64_t u0 = cta * r.per;
  int64_t pre = before + incl - sum;
  if (u0 >= pre && u0 < pre + sum) {
    for (int b = b0; b < b1; ++b) {
      const int64_t n = items(b);
      if (u0 < pre + n) {
        scan.b = b;
        scan.in = u0 - pre;
        break;
      }
      pre += n;
    }
  }
  __syncthreads();
  r.b = scan.b;  // meaningful only when cta * per < total
  r.in = scan.in;
  return r;
}

// ---------------------------------------------------------------------------
// block scales: powers of two
// ---------------------------------------------------------------------------

// Exponent e of the smallest 2^e with amax <= 448 * 2^e (448 = 1.75 * 2^8), at
// least -126; amax finite and >= 0.  From the bits: amax = 1.m * 2^x needs
// e = x - 8, one more when 1.m > 1.75.  A power of two costs an e4m3 code no
// precision but at most one binade at the subnormal end; in return x / s and
// the requantisation of a block whose scale grew are exact shifts.
__device__ __forceinline__ int block_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return max(e, -126);
}

__device__ __forceinline__ float pow2(int e) {  // -126 <= e <= 127
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// |x| if finite, else 0: what a block's scale goes by.
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < INFINITY ? a : 0.f;
}

// ---------------------------------------------------------------------------
// rotary angles
// ---------------------------------------------------------------------------

// A pair's frequency as a 64-bit fraction of a turn per position.  Position
// times it, wrapping, is the angle's exact fraction of a turn: the reduction
// costs no precision however far the position (the table's own rounding, 2^-53
// relative, is what remains).
__device__ __forceinline__ uint64_t turns_per_token(double inv_freq) {
  double t = inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
  t -= floor(t);
  return __double2ull_rn(t * 18446744073709551616.0);
}

// (m cos, m sin) of position p's angle.
__device__ __forceinline__ float2 rotation(int p, uint64_t freq, float m) {
  const int64_t phase =
      static_cast<int64_t>(static_cast<uint64_t>(static_cast<int64_t>(p)) * freq);
  float s, c;
  sincospif(static_cast<float>(phase) * 0x1p-63f, &s, &c);  // phase 2^-64 turns = phase 2^-63 pi
  return make_float2(m * c, m * s);
}

struct RopeArgs {
  const double *inv_freq;
  int32_t rd, layout;  // rotary_dim; KVQ_ROPE_HALF or _INTERLEAVED
  float mscale;
};

// A row of D dims is D / 16 work items of two 8-dim chunks.  Half layout:
// item i < rd / 16 holds chunks i and i + rd / 16, i.e. pairs 8i .. 8i + 7
// whole; the remaining items hold the chunks past rd.  Interleaved: item i
// holds chunks i and i + D / 16, pairs 4c .. 4c + 3 being chunk c.  So no value of
// a pair is ever in another lane, and lanes next to each other read 16-byte
// words next to each other.
struct ItemChunks {
  int c0, c1;  // chunk numbers
};

__device__ __forceinline__ ItemChunks item_chunks(int i, int D, int rd, bool half) {
  ItemChunks o;
  const int h = rd / 16;
  if (half && i < h) {
    o.c0 = i;
    o.c1 = i + h;
  } else if (half) {
    o.c0 = i + h;
    o.c1 = i + D / 16;
  } else {
    o.c0 = i;
    o.c1 = i + D / 16;
  }
  return o;
}

// The angle table of one token in shared memory: rd / 4 float4 (cos, sin of
// pairs 2q and 2q + 1), ordered so that the items of a row read words next
// to each other (no bank conflicts): word q of the table lies at
// (q % w) * (rd / 4 / w) + q / w, w = 4 words an item (half), 2 a chunk.
__device__ __forceinline__ int angle_slot(int q, int rd, bool half) {
  const int w = half ? 4 : 2;
  return (q % w) * (rd / 4 / w) + q / w;
}

// Rotates the 16 values of item i in place: x[0..7] are chunk c0, x[8..15] c1.
__device__ __forceinline__ void rotate_item(float (&x)[16], const float4 *tab, int i, int rd,
                                            bool half, ItemChunks ch) {
  if (half) {
    if (i >= rd / 16) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 t = tab[j * (rd / 16) + i];
      const float a0 = x[2 * j], b0 = x[8 + 2 * j], a1 = x[2 * j + 1], b1 = x[8 + 2 * j + 1];
      x[2 * j] = a0 * t.x - b0 * t.y;
      x[8 + 2 * j] = b0 * t.x + a0 * t.y;
      x[2 * j + 1] = a1 * t.z - b1 * t.w;
      x[8 + 2 * j + 1] = b1 * t.z + a1 * t.w;
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int c = k ? ch.c1 : ch.c0;
    if (c >= rd / 8) continue;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float4 t = tab[j * (rd / 8) + c];
      float *v = x + 8 * k + 4 * j;
      const float a0 = v[0], b0 = v[1], a1 = v[2], b1 = v[3];
      v[0] = a0 * t.x - b0 * t.y;
      v[1] = b0 * t.x + a0 * t.y;
      v[2] = a1 * t.z - b1 * t.w;
      v[3] = b1 * t.z + a1 * t.w;
    }
  }
}

__device__ __forceinline__ void unpack8(uint4 w, float *x) {
  bf16x2_to_f32(w.x, x);
  bf16x2_to_f32(w.y, x + 2);
  bf16x2_to_f32(w.z, x + 4);
  bf16x2_to_f32(w.w, x + 6);
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {  // round to nearest even
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint4 pack8(const float *x) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// ---------------------------------------------------------------------------
// host checks
// ---------------------------------------------------------------------------

inline kvq_status validate_block_cache(const kvq_block_cache *c) {
  if (!c || !c->k_pool || !c->v_pool || !c->scales) return KVQ_ERR_INVALID_ARG;
  if (c->num_pages <= 0 || c->num_kv_heads <= 0) return KVQ_ERR_INVALID_ARG;
  if (!aligned16(c->k_pool) || !aligned16(c->v_pool) ||
      (reinterpret_cast<uintptr_t>(c->scales) & 7u))
    return KVQ_ERR_INVALID_ARG;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64) return KVQ_ERR_UNSUPPORTED;
  if (c->head_dim != 64 && c->head_dim != 128) return KVQ_ERR_UNSUPPORTED;
  return KVQ_OK;
}

inline kvq_status validate_rope(const kvq_rope_desc *r, int head_dim) {
  if (!r || !r->inv_freq || (reinterpret_cast<uintptr_t>(r->inv_freq) & 7u))
    return KVQ_ERR_INVALID_ARG;
  if (r->layout != KVQ_ROPE_HALF && r->layout != KVQ_ROPE_INTERLEAVED) return KVQ_ERR_INVALID_ARG;
  if (r->rotary_dim <= 0 || r->rotary_dim % 16 || r->rotary_dim > head_dim)
    return KVQ_ERR_INVALID_ARG;
  if (!std::isfinite(r->mscale)) return KVQ_ERR_INVALID_ARG;
  return KVQ_OK;
}

// A strided [tokens][heads][D] tensor: alignment and stride.
inline bool rows_ok(const void *p, int64_t stride, int64_t heads, int D) {
  return p && aligned16(p) && stride % 8 == 0 && stride >= heads * D;
}

// The ragged step's host-side arguments.
inline kvq_status validate_ragged(const int32_t *tok_start, int32_t n_tokens,
                                  const int32_t *block_table, int32_t B, int32_t MP,
                                  int32_t page_size) {
  if (n_tokens < 0 || B < 0 || MP <= 0) return KVQ_ERR_INVALID_ARG;
  if (static_cast<int64_t>(MP) * page_size > INT32_MAX) return KVQ_ERR_INVALID_ARG;
  if (!tok_start && n_tokens != B) return KVQ_ERR_INVALID_ARG;
  if (n_tokens > 0 && B > 0 && !block_table) return KVQ_ERR_INVALID_ARG;
  return KVQ_OK;
}

}  // namespace kvq
