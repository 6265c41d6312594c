// kvq_block_attn: causal attention of one or several query rows a request over
// the block-scaled paged cache.
//
// Mathematics (include/kvq.h): with the page's scales ks, vs of the kv head,
//     x_j = sm_scale log2(e) ks (q . code_j),  out = sum_j 2^(x_j - m) vs code'_j / sum_j 2^(x_j - m)
// in one pass over the tokens.  Each row keeps two running references: m, the
// maximum of x, for the denominator l, and n, the maximum of x + log2(vs),
// for the accumulators o.  The weights of a tile are w_j = 2^(x_j - m) for l and
// w_j vs 2^(m - n) for o, so the f16 operand of p.v is at most 2^8 (lazy
// rescaling) however the scales of the V blocks differ, and a block of large
// values with a small softmax weight keeps its precision beside a block of
// small values with a large one.  out = 2^(n - m) o / l.
//
// Bound: HBM.  A request's K and V are read once for all query heads of a kv
// head and all its rows, in blocks of 32 rows x heads a kv head, or 128 (ba_shape).
// Measured: 64 requests of 8,193 - 9,216 tokens, 8 kv heads of 128, 4
// heads a kv head, one row: 174 us, 97% of the measured copy rate; 8 heads a kv head,
// 512 - 65,536 tokens, pages of 64: 294 us, 95%; 8 requests of 8,193 tokens: 30 us, 66%
// (3 us until the first bytes are asked for, 4 for the cut rows).
//
//   split   persistent CTAs; the requests' (kv-head group, row block) rows, in
//           units of 16 tokens, are laid end to end and cut into equal runs
//           (find_run: every CTA works out its own start, so the call needs no
//           plan kernel at any batch size).  A producer warp walks the run, stages
//           16 tokens of a group of HG heads per TMA copy into a ring (the pool
//           layout makes them one box) and the blocks' scales by 8-byte async
//           copies that count on the same barrier.  Consumer warps: HG
//           heads x RT 16-row tiles x TW teams that take the ring's stages in
//           turn, so that few heads or few rows still occupy every warp.  At
//           the end of a segment the teams' partials meet in shared memory.
//   combine merges rows that were cut across CTAs.
//
// head_dim 128 with many rows takes another split kernel (block_attn_tc.cuh).  Here q.k
// and p.v run on mma.sync m16n8k16 (f16 in, fp32 sums): at up to 16 rows a
// tile the tensor work is about half of what the memory time allows, and the
// operands come from registers in the layout that the byte conversion leaves
// them in.  e4m3 is exact in f16; a row of q is scaled by a power of two into
// f16's range (exact down to 2^-39 of its largest value); weights are split
// into an f16 and its f16 remainder (relative error 2^-22), because one f16
// alone (2^-11) would be visible in an fp32 output.
//
// Every wait is bounded; one that gives up raises KVQ_ERRBIT_TIMEOUT, and the
// CTA leaves after its copies have landed.
#include <algorithm>
#include <atomic>
#include <climits>

#include "block_common.cuh"
#include "decode_common.cuh"
#include "decode_attn_mma.cuh"
#include "tc_device.cuh"
#include "block_attn_split.cuh"

#include "block_attn_tc.cuh"

namespace kvq {

// ---------------------------------------------------------------------------
// combine: rows cut across CTAs
// ---------------------------------------------------------------------------

constexpr int kBcbWarps = 8;

// blockIdx.x: which of the cut rows, in the order of their CTAs (there are at
// most as many as rows of work, and fewer than CTAs); blockIdx.y: which of its output
// rows, eight a CTA and one a warp (kWide false), or one whose parts the eight
// warps share (kWide true: batches of so few rows that one has many parts).
//   out = 2^(N - M) sum_p 2^(n_p - N) o_p / sum_p 2^(m_p - M) l_p
template <int D, bool kWide>
__global__ void __launch_bounds__(32 * kBcbWarps) block_combine_kernel(BaArgs a, int rk_shift,
                                                                      int ctas) {
  constexpr int V = D / 32, RF = D + kStat, kBatch = 4;
  __shared__ float s_acc[kWide ? kBcbWarps : 1][D];
  __shared__ float4 s_st[kWide ? kBcbWarps : 1];
  __shared__ int s_cnt[kBcbWarps], s_cta;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int idx = kWide ? blockIdx.y : blockIdx.y * kBcbWarps + warp;  // (pair, row)
  const int ngrp = a.hg * a.rt, rk = 1 << rk_shift;
  const int pair = idx >> rk_shift, rr = idx & (rk - 1);
  const int head = pair / a.rt, tile = pair - head * a.rt;
  grid_dependency_wait();
  allow_dependents();
  // the CTA that holds cut row blockIdx.x's first part
  int before = 0;
  if (threadIdx.x == 0) s_cta = -1;
  for (int c = threadIdx.x; c - static_cast<int>(threadIdx.x) < ctas; c += 32 * kBcbWarps) {
    const bool is_cut = c < ctas && __ldcg(&a.cut[c].parts) > 0;
    const unsigned in_warp = __ballot_sync(0xffffffffu, is_cut);
    __syncthreads();
    if (lane == 0) s_cnt[warp] = __popc(in_warp);
    __syncthreads();
    int rank = before + __popc(in_warp & ((1u << lane) - 1));
#pragma unroll
    for (int w = 0; w < kBcbWarps; ++w) {
      if (w < warp) rank += s_cnt[w];
      before += s_cnt[w];
    }
    if (is_cut && rank == static_cast<int>(blockIdx.x)) s_cta = c;
  }
  __syncthreads();
  const int cta = s_cta;
  if (cta < 0) return;
  const int4 c0 = __ldcg(reinterpret_cast<const int4 *>(a.cut + cta));
  const int n = __ldcg(&a.cut[cta].n);
  const int parts = c0.x, grp = c0.y, rb = c0.z, row0 = c0.w;
  const int r = (rb * a.rt + tile) * rk + rr;
  if (pair >= ngrp || r >= n * a.G) return;
  float M = -INFINITY, N = -INFINITY, l = 0.f, acc[V];
  bool bad = false;
#pragma unroll
  for (int k = 0; k < V; ++k) acc[k] = 0.f;
  // part p lies in the p-th CTA from here on: the first in slot 1, others in slot 0
  const float *base = a.part + ((static_cast<int64_t>(2 * cta) * ngrp + pair) * rk + rr) * RF;
  const int64_t slot = static_cast<int64_t>(ngrp) * rk * RF;
  constexpr int kStep = kWide ? kBcbWarps : 1;
  for (int p0 = kWide ? warp : 0; p0 < parts; p0 += kBatch * kStep) {
    float4 s[kBatch];
    float v[kBatch][V];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int p = p0 + j * kStep;
      s[j] = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
      if (p < parts) {
        const float *q = base + (2 * p + (p == 0)) * slot;
        s[j] = __ldcg(reinterpret_cast<const float4 *>(q + D));
#pragma unroll
        for (int k = 0; k < V; ++k) v[j][k] = __ldcg(q + lane + 32 * k);
      }
    }
    float Mb = M, Nb = N;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      Mb = fmaxf(Mb, s[j].x);
      Nb = fmaxf(Nb, s[j].z);
      bad |= s[j].y < 0.f;
    }
    const float fl = M == -INFINITY ? 0.f : exp2f(M - Mb), fo = N == -INFINITY ? 0.f : exp2f(N - Nb);
    l *= fl;
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] *= fo;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (s[j].y == 0.f) continue;  // saw nothing
      l = fmaf(exp2f(s[j].x - Mb), s[j].y, l);
      const float f = exp2f(s[j].z - Nb);
#pragma unroll
      for (int k = 0; k < V; ++k) acc[k] = fmaf(f, v[j][k], acc[k]);
    }
    M = Mb;
    N = Nb;
  }
  const int i = r / a.G;
  float *out = a.out + ((static_cast<int64_t>(row0) + i) * a.Hq + (grp * a.hg + head) * a.G + r - i * a.G) * D;
  if constexpr (!kWide) {
    const float2 f = out_scale(N - M - 7.f, l);
#pragma unroll
    for (int k = 0; k < V; ++k) out[lane + 32 * k] = bad ? 0.f : acc[k] * f.x * f.y;
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) s_acc[warp][lane + 32 * k] = acc[k];
    if (lane == 0) s_st[warp] = make_float4(M, bad ? -1.f : l, N, 0.f);
    __syncthreads();
    if (threadIdx.x < D) {
      float Mr = -INFINITY, Nr = -INFINITY, lr = 0.f, o = 0.f;
      bool rbad = false;
#pragma unroll
      for (int w = 0; w < kBcbWarps; ++w) {
        Mr = fmaxf(Mr, s_st[w].x);
        Nr = fmaxf(Nr, s_st[w].z);
        rbad |= s_st[w].y < 0.f;
      }
#pragma unroll
      for (int w = 0; w < kBcbWarps; ++w) {
        if (s_st[w].y == 0.f) continue;
        lr = fmaf(exp2f(s_st[w].x - Mr), s_st[w].y, lr);
        o = fmaf(exp2f(s_st[w].z - Nr), s_acc[w][threadIdx.x], o);
      }
      const float2 f = out_scale(Nr - Mr - 7.f, lr);
      out[threadIdx.x] = rbad ? 0.f : o * f.x * f.y;
    }
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

namespace {

using BaFn = void (*)(CUtensorMap, CUtensorMap, BaArgs);

template <int D>
BaFn ba_kernel(int rk) {
  return rk == 4 ? block_split_kernel<D, 4>
                 : rk == 8 ? block_split_kernel<D, 8> : block_split_kernel<D, 16>;
}

// Opt a kernel into its shared memory, once per device.
bool ba_opt_in(BaFn fn, int variant, size_t smem) {
  constexpr int kMaxDev = 64;
  static std::atomic<bool> done[kMaxDev][7];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return false;
  if (done[dev][variant].load(std::memory_order_acquire)) return true;
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) !=
      cudaSuccess)
    return false;
  done[dev][variant].store(true, std::memory_order_release);
  return true;
}

size_t ba_cut_bytes(int ctas) {
  return (static_cast<size_t>(ctas) * sizeof(BaCut) + 255) & ~static_cast<size_t>(255);
}

size_t ba_kept_bytes(const BaShape &s, int ctas) {
  return s.tc ? sizeof(float) * ctas * kTcWarps * kTcKept : 0;
}

// [page][head][slot][dim] as a 4-D map; a box is 16 slots of hg heads.
bool ba_map(CUtensorMap *map, const void *pool, const kvq_block_cache &c, int hg) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t D = c.head_dim, P = c.page_size, H = c.num_kv_heads, NP = c.num_pages;
  const cuuint64_t dims[4] = {D, P, H, NP};
  const cuuint64_t strides[3] = {D, P * D, H * P * D};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(D), static_cast<cuuint32_t>(kTile),
                             static_cast<cuuint32_t>(hg), 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(pool), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

}  // namespace kvq

using namespace kvq;

extern "C" size_t kvq_block_attn_workspace_size(int32_t B, int32_t max_q, int32_t Hq,
                                                int32_t num_kv_heads, int32_t head_dim) {
  if (B < 0 || max_q <= 0 || Hq <= 0 || num_kv_heads <= 0 || Hq % num_kv_heads) return 0;
  if (head_dim != 64 && head_dim != 128) return 0;
  if (static_cast<int64_t>(max_q) * (Hq / num_kv_heads) > INT32_MAX / 2) return 0;
  int sms = 0;
  if (device_sm_count(&sms) != KVQ_OK) return 0;
  // the largest that a call of up to max_q rows may take, by either kernel: fewer rows can need
  // more (wider head groups, or mma.sync's partials where more rows go to tcgen05), and the
  // tilings change after 4, 8, 16 and 128 rows (ba_shape)
  const int rows = max_q * (Hq / num_kv_heads);
  size_t parts = 0;
  for (int most : {4, 8, 16, 128, INT32_MAX})
    for (int64_t capacity : {int64_t{0}, kTcLong}) {
      const BaShape s = ba_shape(std::min(most, rows), 1, num_kv_heads, head_dim, capacity);
      parts = std::max(parts, ba_part_bytes(s, head_dim, sms) + ba_kept_bytes(s, sms));
    }
  return ba_cut_bytes(sms) + parts;
}

extern "C" kvq_status kvq_block_attn(const kvq_block_cache *cache, const void *q, int64_t q_stride,
                                     int32_t Hq, const int32_t *tok_start, int32_t n_tokens,
                                     int32_t max_q, const int32_t *seq_lens,
                                     const int32_t *block_table, int32_t B, int32_t MP,
                                     const uint8_t *abort_mask, float sm_scale, float *out,
                                     void *workspace, size_t workspace_bytes, uint32_t *err_word,
                                     kvq_stream_t stream) {
  kvq_status st = validate_block_cache(cache);
  if (st != KVQ_OK) return st;
  const int D = cache->head_dim, Hkv = cache->num_kv_heads;
  st = validate_ragged(tok_start, n_tokens, block_table, B, MP, cache->page_size);
  if (st != KVQ_OK) return st;
  if (Hq <= 0 || Hq % Hkv || max_q <= 0 || !std::isfinite(sm_scale)) return KVQ_ERR_INVALID_ARG;
  const int G = Hq / Hkv;
  if (static_cast<int64_t>(max_q) * G > INT32_MAX / 2) return KVQ_ERR_INVALID_ARG;
  // the kernels' token counters are 32 bits and run on to the end of a tile (128) and past it
  const int64_t capacity = static_cast<int64_t>(MP) * cache->page_size;
  if (capacity > INT32_MAX - 255) return KVQ_ERR_INVALID_ARG;
  if (n_tokens == 0 || B == 0) return KVQ_OK;
  if (!seq_lens || !out || !workspace || !aligned16(out) || !rows_ok(q, q_stride, Hq, D))
    return KVQ_ERR_INVALID_ARG;
  int sms = 0;
  if (device_sm_count(&sms) != KVQ_OK) return KVQ_ERR_CUDA;
  const BaShape s = ba_shape(max_q, G, Hkv, D, capacity);
  const size_t cb = ba_cut_bytes(sms);
  if (!aligned256(workspace) || workspace_bytes < cb + ba_part_bytes(s, D, sms) + ba_kept_bytes(s, sms))
    return KVQ_ERR_WORKSPACE;
  BaArgs a;
  a.q = static_cast<const uint16_t *>(q);
  a.q_stride = q_stride;
  a.rg = {tok_start, seq_lens, B, n_tokens, capacity};
  a.block_table = block_table;
  a.abort_mask = abort_mask;
  a.scales = reinterpret_cast<const float2 *>(cache->scales);
  a.cut = static_cast<BaCut *>(workspace);
  a.part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + cb);
  a.kept = a.part + ba_part_bytes(s, D, sms) / sizeof(float);
  a.out = out;
  a.err_word = err_word;
  a.num_pages = cache->num_pages;
  a.p_shift = cache->page_size == 16 ? 4 : cache->page_size == 32 ? 5 : 6;
  a.Hkv = Hkv;
  a.Hq = Hq;
  a.G = G;
  a.MP = MP;
  a.max_q = max_q;
  a.hg = s.hg;
  a.rt = s.rt;
  a.tw = s.tw;
  a.rounds = 0;
  for (int t = s.tw; t > 1; t = (t + 1) / 2) ++a.rounds;
  a.groups = s.groups;
  a.stages = s.tc ? 0 : ba_stages(s, D);
  a.q_scale = sm_scale * kLog2e;
  const BaFn fn = s.tc ? block_tc_kernel : D == 128 ? ba_kernel<128>(s.rk) : ba_kernel<64>(s.rk);
  const size_t smem = s.tc ? tc_smem_bytes() : kBaSmem;
  const int variant = s.tc ? 6 : (D == 128 ? 3 : 0) + (s.rk == 4 ? 0 : s.rk == 8 ? 1 : 2);
  if (!ba_opt_in(fn, variant, smem)) return KVQ_ERR_CUDA;
  CUtensorMap kmap, vmap;
  if (!ba_map(&kmap, cache->k_pool, *cache, s.hg) || !ba_map(&vmap, cache->v_pool, *cache, s.hg))
    return KVQ_ERR_CUDA;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (launch_dependent(fn, sms, s.tc ? kTcThreads : kBaThreads, smem, cs, kmap, vmap, a) != cudaSuccess)
    return KVQ_ERR_CUDA;
  // fewer than a row of work for three CTAs: a row is cut into four parts or
  // more, and a CTA merges each of its output rows
  const int64_t work = static_cast<int64_t>(B) * s.row_blocks * s.groups;
  const bool wide = work * 3 < sms;
  const int outs = s.pairs() * s.rk;  // output rows of a row of work
  const dim3 grid(static_cast<unsigned>(work < sms - 1 ? work : sms - 1), wide ? outs : (outs + kBcbWarps - 1) / kBcbWarps);
  const auto cfn = D == 128 ? (wide ? block_combine_kernel<128, true> : block_combine_kernel<128, false>)
                            : (wide ? block_combine_kernel<64, true> : block_combine_kernel<64, false>);
  const int rk_shift = s.rk == 4 ? 2 : s.rk == 8 ? 3 : 4;
  if (launch_dependent(cfn, grid, 32 * kBcbWarps, 0, cs, a, rk_shift, sms) != cudaSuccess)
    return KVQ_ERR_CUDA;
  return KVQ_OK;
}
