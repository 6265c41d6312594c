// kvq_rope: rotary positions on q and k rows; kvq_rope_inv_freq: their tables.
//
// Mathematics: include/kvq.h.  Bandwidth-bound on long inputs (4 bytes an
// element: read and write bf16), launch-bound on a decode step.  A CTA takes
// one token with all its heads, so a pair's sine and cosine are computed once
// and used by every head; a thread owns one item (two 8-dim chunks that hold
// whole pairs, block_common.cuh) of every (blockDim / items)-th head and keeps
// that item's angles in registers.  The first heads' words are loaded before
// the angles are computed, so that their latency covers it.  32,768 rows of 32 + 8
// heads of 128: 180 us, 99% of the measured copy rate; 64 rows 2.5 us, one launch.
#include "block_common.cuh"

namespace kvq {

struct RopeRows {
  const uint16_t *src;
  uint16_t *dst;
  int64_t src_stride, dst_stride;
  int32_t heads;
};

constexpr int kRopeThreads = 320;  // at most

template <int D>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_kernel(RopeArgs r, const int32_t *pos,
                                                            RopeRows q, RopeRows k) {
  constexpr int kItems = D / 16;
  const int kStep = blockDim.x / kItems;  // heads a pass
  __shared__ float4 tab[D / 4];
  const int64_t t = blockIdx.x;
  const int i = threadIdx.x % kItems, h0 = threadIdx.x / kItems;
  const bool half = r.layout == KVQ_ROPE_HALF;
  const ItemChunks ch = item_chunks(i, D, r.rd, half);
  const int heads = q.heads + k.heads;
  grid_dependency_wait();
  allow_dependents();
  const int p = __ldg(pos + t);
  uint4 w[2][2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int h = h0 + j * kStep;
    if (h < heads) {
      const uint16_t *s = h < q.heads ? q.src + t * q.src_stride + static_cast<int64_t>(h) * D
                                      : k.src + t * k.src_stride +
                                            static_cast<int64_t>(h - q.heads) * D;
      w[j][0] = *reinterpret_cast<const uint4 *>(s + ch.c0 * 8);
      w[j][1] = *reinterpret_cast<const uint4 *>(s + ch.c1 * 8);
    }
  }
  for (int j = threadIdx.x; j < r.rd / 4; j += blockDim.x) {
    const float2 a = rotation(p, turns_per_token(r.inv_freq[2 * j]), r.mscale);
    const float2 b = rotation(p, turns_per_token(r.inv_freq[2 * j + 1]), r.mscale);
    tab[angle_slot(j, r.rd, half)] = make_float4(a.x, a.y, b.x, b.y);
  }
  __syncthreads();
  for (int hb = h0; hb < heads; hb += 2 * kStep) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int h = hb + j * kStep;
      if (h >= heads) continue;
      float x[16];
      unpack8(w[j][0], x);
      unpack8(w[j][1], x + 8);
      rotate_item(x, tab, i, r.rd, half, ch);
      uint16_t *o = h < q.heads ? q.dst + t * q.dst_stride + static_cast<int64_t>(h) * D
                                : k.dst + t * k.dst_stride +
                                      static_cast<int64_t>(h - q.heads) * D;
      // chunks past rotary_dim are stored as they came (NaN payloads included)
      const int lim = half ? (i < r.rd / 16 ? D / 8 : 0) : r.rd / 8;
      *reinterpret_cast<uint4 *>(o + ch.c0 * 8) = ch.c0 < lim ? pack8(x) : w[j][0];
      *reinterpret_cast<uint4 *>(o + ch.c1 * 8) = ch.c1 < lim ? pack8(x + 8) : w[j][1];
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int h = hb + (2 + j) * kStep;
      if (h < heads) {
        const uint16_t *s = h < q.heads ? q.src + t * q.src_stride + static_cast<int64_t>(h) * D
                                        : k.src + t * k.src_stride +
                                              static_cast<int64_t>(h - q.heads) * D;
        w[j][0] = *reinterpret_cast<const uint4 *>(s + ch.c0 * 8);
        w[j][1] = *reinterpret_cast<const uint4 *>(s + ch.c1 * 8);
      }
    }
  }
}

}  // namespace kvq

using namespace kvq;

extern "C" kvq_status kvq_rope_inv_freq(int32_t rotary_dim, double base, int32_t scaling,
                                        double factor, double orig_len, double low, double high,
                                        double *inv_freq_host, float *mscale_host) {
  if (!inv_freq_host || !mscale_host || rotary_dim <= 0 || rotary_dim % 16)
    return KVQ_ERR_INVALID_ARG;
  if (!(std::isfinite(base) && base > 1.0)) return KVQ_ERR_INVALID_ARG;
  if (scaling < KVQ_ROPE_PLAIN || scaling > KVQ_ROPE_BANDS) return KVQ_ERR_INVALID_ARG;
  if (scaling != KVQ_ROPE_PLAIN && !(std::isfinite(factor) && factor >= 1.0))
    return KVQ_ERR_INVALID_ARG;
  const bool mixes = scaling == KVQ_ROPE_RAMP || scaling == KVQ_ROPE_BANDS;
  if (mixes && !(std::isfinite(orig_len) && orig_len > 0 && low > 0 && high > low &&
                 std::isfinite(high)))
    return KVQ_ERR_INVALID_ARG;
  const double rd = rotary_dim, two_pi = 6.283185307179586477;
  if (scaling == KVQ_ROPE_BASE) base *= std::pow(factor, rd / (rd - 2.0));
  // RAMP: the (fractional) pair that makes r turns within orig_len
  auto pair_of = [&](double r) {
    return rd * std::log(orig_len / (r * two_pi)) / (2.0 * std::log(base));
  };
  double ramp_lo = 0, ramp_hi = 1;
  if (scaling == KVQ_ROPE_RAMP) {
    ramp_lo = std::fmax(std::floor(pair_of(high)), 0.0);
    ramp_hi = std::fmin(std::ceil(pair_of(low)), rd - 1.0);
  }
  for (int i = 0; i < rotary_dim / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / rd);
    double keep = 1.0;  // share of the unscaled frequency
    if (scaling == KVQ_ROPE_LINEAR) keep = 0.0;
    if (scaling == KVQ_ROPE_RAMP)
      keep = 1.0 - (i - ramp_lo) / std::fmax(ramp_hi - ramp_lo, 1e-3);
    if (scaling == KVQ_ROPE_BANDS) keep = (orig_len * f / two_pi - low) / (high - low);
    keep = std::fmin(std::fmax(keep, 0.0), 1.0);
    inv_freq_host[i] = keep >= 1.0 ? f : f / factor * (1.0 - keep) + f * keep;
  }
  *mscale_host = scaling == KVQ_ROPE_RAMP ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.f;
  return KVQ_OK;
}

extern "C" kvq_status kvq_rope(const kvq_rope_desc *rope, const int32_t *pos, int32_t n_tokens,
                               int32_t head_dim, const void *q, int64_t q_stride, void *q_out,
                               int64_t q_out_stride, int32_t n_q_heads, const void *k,
                               int64_t k_stride, void *k_out, int64_t k_out_stride,
                               int32_t n_k_heads, kvq_stream_t stream) {
  if (head_dim != 64 && head_dim != 128) return KVQ_ERR_UNSUPPORTED;
  const kvq_status st = validate_rope(rope, head_dim);
  if (st != KVQ_OK) return st;
  if (n_tokens < 0 || n_q_heads <= 0 || n_k_heads < 0) return KVQ_ERR_INVALID_ARG;
  if (n_tokens == 0) return KVQ_OK;
  if (!pos || !rows_ok(q, q_stride, n_q_heads, head_dim) ||
      !rows_ok(q_out, q_out_stride, n_q_heads, head_dim))
    return KVQ_ERR_INVALID_ARG;
  if (n_k_heads > 0 && (!rows_ok(k, k_stride, n_k_heads, head_dim) ||
                        !rows_ok(k_out, k_out_stride, n_k_heads, head_dim)))
    return KVQ_ERR_INVALID_ARG;
  const RopeArgs r{rope->inv_freq, rope->rotary_dim, rope->layout, rope->mscale};
  const RopeRows qr{static_cast<const uint16_t *>(q), static_cast<uint16_t *>(q_out), q_stride,
                    q_out_stride, n_q_heads};
  const RopeRows kr{static_cast<const uint16_t *>(k), static_cast<uint16_t *>(k_out), k_stride,
                    k_out_stride, n_k_heads};
  // two heads a thread, or a multiple
  const int items = (n_q_heads + n_k_heads) * (head_dim / 16);
  const int rounds = (items + 2 * kRopeThreads - 1) / (2 * kRopeThreads);
  const int threads = ((items + 2 * rounds - 1) / (2 * rounds) + 31) / 32 * 32;
  const cudaError_t e =
      launch_dependent(head_dim == 128 ? rope_kernel<128> : rope_kernel<64>, n_tokens,
                       threads, 0, reinterpret_cast<cudaStream_t>(stream), r, pos, qr, kr);
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}
