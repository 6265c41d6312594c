// kvq_block_prefix_attn: causal attention over the block-scaled cache for a batch
// whose requests form groups with a shared prefix of whole pages.
#include <climits>

#include "block_common.cuh"

namespace kvq {

struct PfArgs {
  const uint16_t *q;
  int64_t q_stride;
  Ragged rg;
  const int32_t *block_table, *group_start, *prefix_pages;
  const uint8_t *abort_mask;
  const uint8_t *k_pool, *v_pool;
  const float2 *scales;  // [num_pages][Hkv]
  uint16_t *out;
  uint32_t *err_word;
  int32_t num_pages, p_shift, Hkv, Hq, G, MP, max_q, n_groups;
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

constexpr int kPfWarps = 8;

template <int D>
__global__ void __launch_bounds__(32 * kPfWarps) prefix_kernel(PfArgs a) {
  constexpr int V = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, b = blockIdx.x;
  grid_dependency_wait();
  allow_dependents();
  bool order = true;
  for (int g = threadIdx.x; g < a.n_groups; g += 32 * kPfWarps) order &= pf_group_ok(a, g);
  order = __syncthreads_and(order);
  PfReq rq = order ? pf_request(a, b) : PfReq{request_rows<true>(a.rg, b), 0, -1, false};
  if (!order) rq.r.err |= KVQ_ERRBIT_REQ;
  if (rq.r.err && blockIdx.y == 0 && threadIdx.x == 0) report(a.err_word, rq.r.err);
  const bool live = rq.live && order;
  int leader = b;
  if (live && rq.pre > 0)
    for (leader = __ldg(a.group_start + rq.group); leader < b && !pf_request(a, leader).live;) ++leader;
  const int32_t *mine = a.block_table + static_cast<int64_t>(b) * a.MP;
  const int32_t *first = a.block_table + static_cast<int64_t>(leader) * a.MP;
  for (int u = blockIdx.y * kPfWarps + warp; u < rq.r.n * a.Hq; u += gridDim.y * kPfWarps) {
    const int i = u / a.Hq, h = u - i * a.Hq, kvh = h / a.G;
    uint16_t *o = a.out + ((static_cast<int64_t>(rq.r.row) + i) * a.Hq + h) * D;
    float acc[V], q[V], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      acc[k] = 0.f;
      q[k] = live ? __uint_as_float(static_cast<uint32_t>(a.q[(static_cast<int64_t>(rq.r.row) + i) * a.q_stride +
                                                            h * D + lane + 32 * k]) << 16)
                  : 0.f;
    }
    bool bad = !live;
    const int L = rq.r.p0 + i + 1;
    for (int t = 0; !bad && t < L; ++t) {
      const int page = __ldg((t < rq.pre ? first : mine) + (t >> a.p_shift));
      if (page < 0 || page >= a.num_pages) {
        if (lane == 0) report(a.err_word, KVQ_ERRBIT_PAGE);
        bad = true;
        break;
      }
      const float2 sc = __ldg(a.scales + static_cast<int64_t>(page) * a.Hkv + kvh);
      const int64_t at = (((static_cast<int64_t>(page) * a.Hkv + kvh) << a.p_shift) + (t & ((1 << a.p_shift) - 1))) * D;
      float s = 0.f, v[V];
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const uint32_t c = __ldg(a.k_pool + at + lane + 32 * k) | (__ldg(a.v_pool + at + lane + 32 * k) << 8);
        const uint32_t f = e4m3x2_to_f16x2(static_cast<uint16_t>(c));
        const float2 kv = __half22float2(*reinterpret_cast<const __half2 *>(&f));
        s = fmaf(q[k], kv.x, s);
        v[k] = kv.y * sc.y;
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
      s *= sc.x * a.q_scale;
      const float M = fmaxf(m, s), f = exp2f(m - M), p = exp2f(s - M);
      m = M;
      l = l * f + p;
#pragma unroll
      for (int k = 0; k < V; ++k) acc[k] = acc[k] * f + p * v[k];
    }
#pragma unroll
    for (int k = 0; k < V; ++k)
      o[lane + 32 * k] = static_cast<uint16_t>(pack_bf16x2(bad ? 0.f : acc[k] / l, 0.f));
  }
}

}  // namespace kvq

using namespace kvq;

extern "C" size_t kvq_block_prefix_attn_workspace_size(int32_t n_tokens, int32_t Hq,
                                                       int32_t num_kv_heads, int32_t head_dim) {
  if (n_tokens < 0 || Hq <= 0 || num_kv_heads <= 0 || Hq % num_kv_heads) return 0;
  if (head_dim != 64 && head_dim != 128) return 0;
  return 256;
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
  const int64_t capacity = static_cast<int64_t>(MP) * cache->page_size;
  if (capacity > INT32_MAX - 255) return KVQ_ERR_INVALID_ARG;
  if (n_tokens == 0 || B == 0) return KVQ_OK;
  if (!seq_lens || !out || !workspace || !aligned16(out) || !rows_ok(q, q_stride, Hq, D)) return KVQ_ERR_INVALID_ARG;
  if (n_groups > 0 && (!group_start || !prefix_pages)) return KVQ_ERR_INVALID_ARG;
  if (!aligned256(workspace) || workspace_bytes < kvq_block_prefix_attn_workspace_size(n_tokens, Hq, Hkv, D))
    return KVQ_ERR_WORKSPACE;
  PfArgs a;
  a.q = static_cast<const uint16_t *>(q);
  a.q_stride = q_stride;
  a.rg = {tok_start, seq_lens, B, n_tokens, capacity};
  a.block_table = block_table;
  a.group_start = group_start;
  a.prefix_pages = prefix_pages;
  a.abort_mask = abort_mask;
  a.k_pool = static_cast<const uint8_t *>(cache->k_pool);
  a.v_pool = static_cast<const uint8_t *>(cache->v_pool);
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
  a.q_scale = sm_scale * 1.4426950408889634f;
  const dim3 grid(static_cast<unsigned>(B), static_cast<unsigned>((Hq + kPfWarps - 1) / kPfWarps));
  const cudaError_t e = launch_dependent(D == 128 ? prefix_kernel<128> : prefix_kernel<64>, grid, 32 * kPfWarps, 0,
                                         reinterpret_cast<cudaStream_t>(stream), a);
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}
