// kvq_copy_pages and kvq_block_copy_pages: whole pages copied by a list of pairs
// (include/kvq.h).
//
// Bound: HBM, every byte read and written once.  All pairs' pages are one sequence of
// 16-byte vectors (a page's K, then its V), cut into tiles of 16 KB that CTAs of 256
// threads take in turn, four vectors in flight a thread; so that one page is spread over
// several CTAs, and a CTA has as much to do whatever the page's size.  20,011 pages of 32 KB, K
// and V: 206 us, 95% of the measured copy rate; 48 pages 4.6, a launch.  A pair that is left out is found by each of
// its vectors: 150,000 of them, and nothing copied, take 561 us, and 20,011 pairs among as many 667.
#include <algorithm>

#include "block_common.cuh"

namespace kvq {

constexpr int kCpThreads = 256;
constexpr int kCpVecs = 4;  // vectors a thread has in flight

struct CopyArgs {
  uint4 *k, *v;
  float2 *scales;  // [num_pages][heads], or null
  const int32_t *src, *dst;
  uint32_t *err_word;
  int32_t num_pages, n, heads, vecs;  // vectors of one pool's page
};

// The pair's pages; false: it is left out.
__device__ __forceinline__ bool copy_pair(const CopyArgs &a, int pair, int64_t &s, int64_t &d) {
  const int from = __ldg(a.src + pair), to = __ldg(a.dst + pair);
  s = from;
  d = to;
  return from >= 0 && to >= 0 && from < a.num_pages && to < a.num_pages && from != to;
}

__global__ void __launch_bounds__(kCpThreads) copy_pages_kernel(CopyArgs a) {
  grid_dependency_wait();
  allow_dependents();
  const int both = 2 * a.vecs;
  const int64_t total = static_cast<int64_t>(a.n) * both;
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * (kCpThreads * kCpVecs); t0 < total;
       t0 += static_cast<int64_t>(gridDim.x) * (kCpThreads * kCpVecs)) {
    uint4 x[kCpVecs];
    uint4 *to[kCpVecs];
#pragma unroll
    for (int k = 0; k < kCpVecs; ++k) {
      const int64_t i = t0 + threadIdx.x + k * kCpThreads;
      to[k] = nullptr;
      if (i >= total) continue;
      const int pair = static_cast<int>(i / both), in = static_cast<int>(i - static_cast<int64_t>(pair) * both);
      int64_t s, d;
      if (!copy_pair(a, pair, s, d)) continue;
      uint4 *pool = in < a.vecs ? a.k : a.v;
      const int at = in < a.vecs ? in : in - a.vecs;
      x[k] = __ldcs(pool + s * a.vecs + at);
      to[k] = pool + d * a.vecs + at;
    }
#pragma unroll
    for (int k = 0; k < kCpVecs; ++k)
      if (to[k]) __stcs(to[k], x[k]);
  }
  const int per = a.scales ? a.heads : 1;  // (without scales: the check alone)
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kCpThreads + threadIdx.x;
       i < static_cast<int64_t>(a.n) * per; i += static_cast<int64_t>(gridDim.x) * kCpThreads) {
    const int pair = static_cast<int>(i / per), h = static_cast<int>(i - static_cast<int64_t>(pair) * per);
    int64_t s, d;
    if (copy_pair(a, pair, s, d)) {
      if (a.scales) a.scales[d * a.heads + h] = a.scales[s * a.heads + h];
    } else if (s >= a.num_pages || d >= a.num_pages) {
      report(a.err_word, KVQ_ERRBIT_PAGE);
    }
  }
}

static kvq_status copy_pages(CopyArgs a, cudaStream_t stream) {
  int sms = 0;
  if (device_sm_count(&sms) != KVQ_OK) return KVQ_ERR_CUDA;
  const int64_t vecs = static_cast<int64_t>(a.n) * 2 * a.vecs, tile = kCpThreads * kCpVecs;
  const int64_t ctas = std::min<int64_t>((vecs + tile - 1) / tile, static_cast<int64_t>(sms) * 8);
  const cudaError_t e = launch_dependent(copy_pages_kernel, static_cast<unsigned>(ctas), kCpThreads, 0, stream, a);
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

}  // namespace kvq

using namespace kvq;

extern "C" kvq_status kvq_copy_pages(const kvq_cache *cache, const int32_t *src, const int32_t *dst,
                                     int32_t n, uint32_t *err_word, kvq_stream_t stream) {
  const kvq_status st = validate_cache(cache);
  if (st != KVQ_OK) return st;
  if (n < 0) return KVQ_ERR_INVALID_ARG;
  if (n == 0) return KVQ_OK;
  if (!src || !dst) return KVQ_ERR_INVALID_ARG;
  const int64_t bytes = static_cast<int64_t>(cache->num_kv_heads) * cache->page_size * cache->head_dim *
                        (cache->kv_dtype == KVQ_KV_E4M3 ? 1 : 2);
  if (bytes / 16 > INT32_MAX / 2) return KVQ_ERR_INVALID_ARG;
  return copy_pages({static_cast<uint4 *>(cache->k_pool), static_cast<uint4 *>(cache->v_pool), nullptr, src, dst,
                     err_word, cache->num_pages, n, cache->num_kv_heads, static_cast<int32_t>(bytes / 16)},
                    reinterpret_cast<cudaStream_t>(stream));
}

extern "C" kvq_status kvq_block_copy_pages(const kvq_block_cache *cache, const int32_t *src,
                                           const int32_t *dst, int32_t n, uint32_t *err_word,
                                           kvq_stream_t stream) {
  const kvq_status st = validate_block_cache(cache);
  if (st != KVQ_OK) return st;
  if (n < 0) return KVQ_ERR_INVALID_ARG;
  if (n == 0) return KVQ_OK;
  if (!src || !dst) return KVQ_ERR_INVALID_ARG;
  const int64_t bytes = static_cast<int64_t>(cache->num_kv_heads) * cache->page_size * cache->head_dim;
  if (bytes / 16 > INT32_MAX / 2) return KVQ_ERR_INVALID_ARG;
  return copy_pages({static_cast<uint4 *>(cache->k_pool), static_cast<uint4 *>(cache->v_pool),
                     reinterpret_cast<float2 *>(cache->scales), src, dst, err_word, cache->num_pages, n,
                     cache->num_kv_heads, static_cast<int32_t>(bytes / 16)},
                    reinterpret_cast<cudaStream_t>(stream));
}
