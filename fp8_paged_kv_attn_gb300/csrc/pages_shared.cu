// Pages that several requests hold: kvq_pages_fork, kvq_pages_release,
// kvq_pages_compact (include/kvq.h).
//
// shares[p] counts the block-table entries that hold page p beyond the first, so
// a page that kvq_pages_update hands out needs no entry written: 0 is right.
//
// Each call is one cluster of up to 8 CTAs of 1,024 threads.  Its phases depend on
// one another (a fork's pages on the forks before it, a page's place on the stack on
// its last holder in the list) and are ordered by the cluster's hardware barrier, so that a
// call is one launch, whatever its sizes, and its work spreads over 8,192 threads.  What
// bounds it: a launch and a barrier a phase for short lists (5 - 9 us), and then the
// latency of its scattered accesses (holders of a page), of which a thread has several in flight.
//
// Lists are taken in rounds of 1,024 entries: every CTA scans a round's page counts, and
// the round's pages ("items", in list order) are spread over the cluster by a binary
// search of the scan.
#include <algorithm>
#include <climits>

#include <cooperative_groups.h>

#include "kvq_internal.h"

namespace kvq {

namespace cg = cooperative_groups;

constexpr int kShThreads = 1024;
constexpr int kShCtas = 8;
constexpr int kShBatch = 4;  // items a thread has in flight

struct ShSmem {
  long long pre[kShThreads];  // items of the round before each entry
  long long warp[33];
  int base[kShThreads];  // the entry's first logical page
  int req[kShThreads], other[kShThreads];
  uint8_t on[kShThreads];
  unsigned int bits;
  long long sum;
};

// Exclusive scan of v over the CTA; *total = the sum.
__device__ __forceinline__ long long sh_scan(long long v, ShSmem &sm, long long *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) sm.warp[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    const long long w = sm.warp[lane];
    long long wi = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, wi, o);
      if (lane >= o) wi += u;
    }
    sm.warp[lane] = wi - w;
    if (lane == 31) sm.warp[32] = wi;
  }
  __syncthreads();
  const long long r = sm.warp[warp] + incl - v;
  *total = sm.warp[32];
  __syncthreads();  // the scratch may be reused
  return r;
}

// The entry of a round of m entries that holds item e: the last with pre <= e.
__device__ __forceinline__ int sh_owner(const ShSmem &sm, int m, long long e) {
  int lo = 0, hi = m - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sm.pre[mid] <= e)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// The cluster's error bits together; every thread of the cluster calls it.
__device__ __forceinline__ unsigned int sh_bits(cg::cluster_group &cl, ShSmem &sm) {
  cl.sync();
  unsigned int all = 0;
  for (unsigned int r = 0; r < cl.num_blocks(); ++r)
    all |= *cl.map_shared_rank(&sm.bits, r);
  cl.sync();  // nobody's bits change, or go with their CTA, before all have read them
  return all;
}

// Memory that other CTAs of the cluster write: never through the read-only path.
template <typename T>
__device__ __forceinline__ T vol(const T *p) {
  return __ldcg(p);
}

// ---------------------------------------------------------------------------
// fork
// ---------------------------------------------------------------------------

struct ForkArgs {
  int32_t *stack, *count;
  uint32_t *tags;
  int32_t *shares, *table;
  uint32_t *expected;
  const int32_t *src, *dst, *tokens;
  int32_t *copy_src, *copy_dst;
  uint8_t *ok;
  int32_t *claim;  // [B]: the fork that writes a request's row, or INT_MAX
  uint32_t *err_word;
  int32_t num_pages, B, MP, page_size, n;
};

__global__ void __launch_bounds__(kShThreads, 1) fork_kernel(ForkArgs a) {
  __shared__ ShSmem sm;
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, cta = cl.block_rank(), ctas = cl.num_blocks();
  const int at = cta * kShThreads + tid, threads = ctas * kShThreads;
  grid_dependency_wait();
  allow_dependents();
  if (tid == 0) sm.bits = 0;
  const int count = *a.count;
  if (count < 0 || count > a.num_pages) {  // every CTA alike
    for (int i = at; i < a.n; i += threads) {
      a.ok[i] = 0;
      a.copy_src[i] = a.copy_dst[i] = -1;
    }
    if (at == 0) report(a.err_word, KVQ_ERRBIT_PAGE);
    return;
  }
  auto in_range = [&](int i, int &s, int &d) {
    s = a.src[i];
    d = a.dst[i];
    return s >= 0 && s < a.B && d >= 0 && d < a.B && s != d;
  };
  // ---- each request is written by one fork, and not read by another
  for (int i = at; i < a.n; i += threads) {
    int s, d;
    if (in_range(i, s, d)) a.claim[s] = a.claim[d] = INT_MAX;
  }
  cl.sync();
  for (int i = at; i < a.n; i += threads) {
    int s, d;
    if (in_range(i, s, d)) atomicMin(a.claim + d, i);
  }
  cl.sync();
  unsigned int bits = 0;
  for (int i = at; i < a.n; i += threads) {
    int s, d;
    bool valid = in_range(i, s, d) && vol(a.claim + d) == i && vol(a.claim + s) == INT_MAX;
    if (!valid) bits |= KVQ_ERRBIT_REQ;
    const long long t = a.tokens[i];
    if (valid && (t < 0 || t > static_cast<long long>(a.MP) * a.page_size)) {
      bits |= KVQ_ERRBIT_POS;
      valid = false;
    }
    a.ok[i] = valid;
  }
  cl.sync();
  // ---- every page that a fork takes, or copies, is a page
  for (int r0 = 0; r0 < a.n; r0 += kShThreads) {
    const int i = r0 + tid, m = min(kShThreads, a.n - r0);
    long long pages = 0, total;
    if (i < a.n && vol(a.ok + i)) {
      sm.req[tid] = a.src[i];
      pages = (static_cast<long long>(a.tokens[i]) + a.page_size - 1) / a.page_size;
    }
    sm.pre[tid] = sh_scan(pages, sm, &total);
    __syncthreads();
    for (long long e = at; e < total; e += threads) {
      const int o = sh_owner(sm, m, e);
      const int page = a.table[static_cast<int64_t>(sm.req[o]) * a.MP + (e - sm.pre[o])];
      if (page < 0 || page >= a.num_pages) {
        a.ok[r0 + o] = 0;
        bits |= KVQ_ERRBIT_PAGE;
      }
    }
    __syncthreads();
  }
  cl.sync();
  // ---- served in order until the first that finds the stack empty
  long long wanted = 0, taken = 0;
  for (int r0 = 0; r0 < a.n; r0 += kShThreads) {
    const int i = r0 + tid, m = min(kShThreads, a.n - r0);
    const bool valid = i < a.n && vol(a.ok + i) != 0;
    int s = 0, d = 0, full = 0, cut = 0;
    if (valid) {
      s = a.src[i];
      d = a.dst[i];
      full = a.tokens[i] / a.page_size;
      cut = a.tokens[i] % a.page_size != 0;
    }
    long long need, total;
    const long long pre = sh_scan(cut, sm, &need);
    const bool fits = valid && wanted + pre + cut <= count;
    if (valid && !fits) bits |= KVQ_ERRBIT_EXHAUSTED;
    sm.req[tid] = s;
    sm.other[tid] = d;
    sm.pre[tid] = sh_scan(fits ? full : 0, sm, &total);
    cl.sync();  // every CTA has read the round's flags
    if (cta == 0 && i < a.n) {
      int from = -1, to = -1;
      if (fits && cut) {
        const int page = a.stack[count - 1 - (wanted + pre)];
        if (page >= 0 && page < a.num_pages) {
          const uint32_t tag = a.tags[page] + 1u;
          const int64_t row = static_cast<int64_t>(d) * a.MP + full;
          a.tags[page] = tag;
          a.table[row] = page;
          a.expected[row] = tag;
          from = a.table[static_cast<int64_t>(s) * a.MP + full];
          to = page;
        } else {
          bits |= KVQ_ERRBIT_PAGE;
        }
      }
      a.ok[i] = fits;
      a.copy_src[i] = from;
      a.copy_dst[i] = to;
    }
    for (long long e0 = at; e0 < total; e0 += static_cast<long long>(kShBatch) * threads) {
      int64_t to[kShBatch];
      int page[kShBatch];
      uint32_t tag[kShBatch];
#pragma unroll
      for (int k = 0; k < kShBatch; ++k) {
        const long long e = e0 + static_cast<long long>(k) * threads;
        page[k] = -1;
        if (e < total) {
          const int o = sh_owner(sm, m, e);
          const int64_t col = e - sm.pre[o], from = static_cast<int64_t>(sm.req[o]) * a.MP + col;
          to[k] = static_cast<int64_t>(sm.other[o]) * a.MP + col;
          page[k] = a.table[from];
          tag[k] = a.expected[from];
        }
      }
#pragma unroll
      for (int k = 0; k < kShBatch; ++k)
        if (page[k] >= 0) {
          a.table[to[k]] = page[k];
          a.expected[to[k]] = tag[k];
          atomicAdd(a.shares + page[k], 1);
        }
    }
    long long served;
    sh_scan(fits ? cut : 0, sm, &served);  // (and the round's entries are read)
    wanted += need;  // above `count` once somebody was not served, so that nobody is from there on
    taken += served;
  }
  if (at == 0) *a.count = count - static_cast<int>(taken);
  if (bits) report(a.err_word, bits);
}

// ---------------------------------------------------------------------------
// release
// ---------------------------------------------------------------------------

struct ReleaseArgs {
  int32_t *stack, *count, *shares, *table;
  const int32_t *req, *first, *npages;
  int32_t *claim;         // [B]
  int32_t *gone, *last;   // [num_pages]: how many entries of the list hold a page, and the last one
  uint32_t *err_word;
  int32_t num_pages, B, MP, n;
};

// Calls f(item, its table entry) for the items [from, to) of the list.  Every thread of the CTA
// calls f together, with a null entry where it has no item.
template <typename F>
__device__ __forceinline__ void sh_items(const ReleaseArgs &a, ShSmem &sm, long long from, long long to, F f) {
  const int tid = threadIdx.x;
  long long carry = 0;
  for (int r0 = 0; r0 < a.n && carry < to; r0 += kShThreads) {
    const int j = r0 + tid, m = min(kShThreads, a.n - r0);
    long long total;
    const long long pre = sh_scan(j < a.n ? a.npages[j] : 0, sm, &total);
    sm.pre[tid] = pre;
    if (j < a.n) {
      sm.req[tid] = a.req[j];
      sm.base[tid] = a.first ? a.first[j] : 0;
    }
    __syncthreads();
    const long long lo = max(from, carry), hi = min(to, carry + total);
    for (long long e0 = lo; e0 < hi; e0 += kShThreads) {
      const long long e = e0 + tid;
      int32_t *entry = nullptr;
      if (e < hi) {
        const int o = sh_owner(sm, m, e - carry);
        entry = a.table + static_cast<int64_t>(sm.req[o]) * a.MP + sm.base[o] + (e - carry - sm.pre[o]);
      }
      f(static_cast<int>(e), entry);
    }
    carry += total;
    __syncthreads();
  }
}

__global__ void __launch_bounds__(kShThreads, 1) release_kernel(ReleaseArgs a) {
  __shared__ ShSmem sm;
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, cta = cl.block_rank(), ctas = cl.num_blocks();
  const int at = cta * kShThreads + tid, threads = ctas * kShThreads;
  grid_dependency_wait();
  allow_dependents();
  if (tid == 0) {
    sm.bits = 0;
    sm.sum = 0;
  }
  __syncthreads();
  const int count = *a.count;
  unsigned int bits = count < 0 || count > a.num_pages ? KVQ_ERRBIT_PAGE : 0;
  // ---- the list: requests named once, pages within their rows
  long long items = 0;
  for (int r0 = 0; r0 < a.n; r0 += kShThreads) {
    const int j = r0 + tid;
    long long n = 0, total;
    if (j < a.n) {
      const int b = a.req[j];
      const long long f = a.first ? a.first[j] : 0;
      n = a.npages[j];
      if (b < 0 || b >= a.B)
        bits |= KVQ_ERRBIT_REQ;
      else if (j % ctas == cta)
        a.claim[b] = INT_MAX;
      if (f < 0 || n < 0 || f + n > a.MP) {
        bits |= KVQ_ERRBIT_POS;
        n = 0;
      }
    }
    sh_scan(n, sm, &total);
    items += total;
  }
  if (items > INT_MAX) bits |= KVQ_ERRBIT_POS;
  if (bits) atomicOr(&sm.bits, bits);
  if (sh_bits(cl, sm)) {
    if (bits) report(a.err_word, bits);
    return;
  }
  for (int j = at; j < a.n; j += threads) atomicMin(a.claim + a.req[j], j);
  cl.sync();
  for (int j = at; j < a.n; j += threads)
    if (vol(a.claim + a.req[j]) != j) bits |= KVQ_ERRBIT_REQ;
  // ---- the items: pages, and their counters cleared
  const long long per = (items + ctas - 1) / ctas;
  const long long from = min(items, cta * per), to = min(items, from + per);
  sh_items(a, sm, from, to, [&](int, const int32_t *entry) {
    if (!entry) return;
    const int page = *entry;
    if (page < 0 || page >= a.num_pages) {
      bits |= KVQ_ERRBIT_PAGE;
    } else {
      a.gone[page] = 0;
      a.last[page] = -1;
    }
  });
  if (bits) atomicOr(&sm.bits, bits);
  if (sh_bits(cl, sm)) {
    if (bits) report(a.err_word, bits);
    return;
  }
  sh_items(a, sm, from, to, [&](int e, const int32_t *entry) {
    if (!entry) return;
    const int page = *entry;
    atomicAdd(a.gone + page, 1);
    atomicMax(a.last + page, e);
  });
  cl.sync();
  // ---- a page whose last holder goes is free, and lies on the stack where its last item stands
  int frees = 0;
  sh_items(a, sm, from, to, [&](int e, const int32_t *entry) {
    if (!entry) return;
    const int page = *entry;
    if (vol(a.last + page) != e) return;
    const int gone = vol(a.gone + page), shares = a.shares[page];
    if (shares < 0 || gone - 1 > shares) bits |= KVQ_ERRBIT_PAGE;  // more often than it is held
    frees += gone - 1 == shares;
  });
  long long freed;
  sh_scan(frees, sm, &freed);
  if (tid == 0) sm.sum = freed;
  if (bits) atomicOr(&sm.bits, bits);
  cl.sync();
  long long before = 0, all = 0;
  unsigned int any = 0;
  for (int r = 0; r < ctas; ++r) {
    const long long f = *cl.map_shared_rank(&sm.sum, r);
    any |= *cl.map_shared_rank(&sm.bits, r);
    before += r < cta ? f : 0;
    all += f;
  }
  cl.sync();
  if (!any && count + all > a.num_pages) any = bits = KVQ_ERRBIT_PAGE;
  if (any) {
    if (bits) report(a.err_word, bits);
    return;
  }
  sh_items(a, sm, from, to, [&](int e, int32_t *entry) {
    int push = -1;
    if (entry) {
      const int page = *entry;
      *entry = -1;
      if (vol(a.last + page) == e) {
        const int left = a.shares[page] - vol(a.gone + page);
        a.shares[page] = max(left, 0);
        if (left < 0) push = page;
      }
    }
    long long total;
    const long long pre = sh_scan(push >= 0, sm, &total);
    if (push >= 0) a.stack[count + before + pre] = push;
    before += total;
  });
  if (at == 0) *a.count = count + static_cast<int>(all);
}

// ---------------------------------------------------------------------------
// compaction
// ---------------------------------------------------------------------------

struct CompactArgs {
  int32_t *stack, *count;
  uint32_t *tags;
  int32_t *shares, *table;
  uint32_t *expected;
  const int32_t *held;
  int32_t *copy_src, *copy_dst, *moves;
  uint32_t *words;  // [words]: a bit for each free page
  int32_t *pre;     // [words]: free pages before a word, within its CTA's share
  uint32_t *err_word;
  int32_t num_pages, B, MP, cap;
};

__global__ void __launch_bounds__(kShThreads, 1) compact_kernel(CompactArgs a) {
  __shared__ ShSmem sm;
  __shared__ int s_base[kShCtas];
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, cta = cl.block_rank(), ctas = cl.num_blocks();
  const int at = cta * kShThreads + tid, threads = ctas * kShThreads;
  grid_dependency_wait();
  allow_dependents();
  if (tid == 0) sm.bits = 0;
  const int words = (a.num_pages + 31) / 32, count = *a.count;
  const int share = (words + ctas - 1) / ctas;  // words a CTA scans
  for (int w = at; w < words; w += threads) a.words[w] = 0;
  unsigned int bits = count < 0 || count > a.num_pages ? KVQ_ERRBIT_PAGE : 0;
  cl.sync();
  if (!bits)
    for (int i = at; i < count; i += threads) {
      const int page = a.stack[i];
      if (page < 0 || page >= a.num_pages)
        bits |= KVQ_ERRBIT_PAGE;
      else if (atomicOr(a.words + (page >> 5), 1u << (page & 31)) >> (page & 31) & 1)
        bits |= KVQ_ERRBIT_PAGE;  // free twice
    }
  for (int b = at; b < a.B; b += threads)
    if (a.held[b] < 0 || a.held[b] > a.MP) bits |= KVQ_ERRBIT_POS;
  if (bits) atomicOr(&sm.bits, bits);
  unsigned int any = sh_bits(cl, sm);
  if (!any) {
    // ---- free pages before each word, and held pages that are none or free
    const int w0 = min(words, cta * share), w1 = min(words, w0 + share);
    long long carry = 0;
    for (int r0 = w0; r0 < w1; r0 += kShThreads) {
      const int w = r0 + tid;
      long long total;
      const long long pre = sh_scan(w < w1 ? __popc(vol(a.words + w)) : 0, sm, &total);
      if (w < w1) a.pre[w] = static_cast<int>(carry + pre);
      carry += total;
    }
    if (tid == 0) sm.sum = carry;
    for (int b = cta; b < a.B; b += ctas) {
      const int32_t *row = a.table + static_cast<int64_t>(b) * a.MP;
      const int held = a.held[b];
      for (int j = tid; j < held; j += kShThreads) {
        const int page = row[j];
        if (page < 0 || page >= a.num_pages || (vol(a.words + (page >> 5)) >> (page & 31) & 1))
          bits |= KVQ_ERRBIT_PAGE;
      }
    }
    if (bits) atomicOr(&sm.bits, bits);
    any = sh_bits(cl, sm);
    if (tid == 0) {
      int base = 0;
      for (int r = 0; r < ctas; ++r) {
        s_base[r] = base;
        base += static_cast<int>(*cl.map_shared_rank(&sm.sum, r));
      }
    }
    cl.sync();
  }
  if (any) {  // nothing changes
    for (int k = at; k < a.cap; k += threads) a.copy_src[k] = a.copy_dst[k] = -1;
    if (at == 0) *a.moves = 0;
    if (bits) report(a.err_word, bits);
    return;
  }
  const int live = a.num_pages - count;
  // free pages below id, and whether id is one
  auto free_below = [&](int id, bool &is_free) {
    const int w = id >> 5;
    const uint32_t word = vol(a.words + w);
    is_free = word >> (id & 31) & 1;
    return s_base[w / share] + vol(a.pre + w) + __popc(word & ((1u << (id & 31)) - 1));
  };
  bool unused;
  const int holes = live < a.num_pages ? free_below(live, unused) : count;
  const int stay = live - holes;  // live pages below `live`
  for (int id = at; id < a.num_pages; id += threads) {
    bool is_free;
    const int f = free_below(id, is_free);
    if (is_free && id < live) {
      a.copy_dst[f] = id;
      a.tags[id] += 1u;
    } else if (!is_free && id >= live) {
      a.copy_src[id - f - stay] = id;
    }
  }
  for (int i = at; i < count; i += threads) a.stack[i] = a.num_pages - 1 - i;
  for (int k = holes + at; k < a.cap; k += threads) a.copy_src[k] = a.copy_dst[k] = -1;
  cl.sync();
  for (int k = at; k < holes; k += threads) {
    const int from = vol(a.copy_src + k), to = vol(a.copy_dst + k);
    a.shares[to] = a.shares[from];
    a.shares[from] = 0;
  }
  for (int b = cta; b < a.B; b += ctas) {
    const int64_t row = static_cast<int64_t>(b) * a.MP;
    const int held = a.held[b];
    for (int j = tid; j < held; j += kShThreads) {
      const int page = a.table[row + j];
      if (page < live) continue;
      bool is_free;
      const int to = vol(a.copy_dst + (page - free_below(page, is_free) - stay));
      a.table[row + j] = to;
      a.expected[row + j] = vol(a.tags + to);
    }
  }
  if (at == 0) *a.moves = holes;
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

namespace {

size_t up256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

// One cluster: a single CTA where a few thousand items at most are in hand (its barriers cost
// less), else eight.
template <typename Args>
cudaError_t launch_cluster(void (*kernel)(Args), int64_t items, cudaStream_t stream, const Args &args) {
  const unsigned ctas = items <= 4 * kShThreads ? 1 : kShCtas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = ctas;
  cfg.blockDim = kShThreads;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, args);
}

}  // namespace

}  // namespace kvq

using namespace kvq;

extern "C" size_t kvq_pages_workspace_size(int32_t num_pages, int32_t B) {
  if (num_pages <= 0 || B <= 0) return 0;
  return up256(4ull * B) + 2 * up256(4ull * num_pages);
}

extern "C" kvq_status kvq_pages_fork(int32_t *free_stack, int32_t *free_count, uint32_t *page_tags,
                                     int32_t *page_shares, int32_t num_pages, int32_t *block_table,
                                     uint32_t *expected_tags, int32_t B, int32_t MP,
                                     int32_t page_size, const int32_t *src_req,
                                     const int32_t *dst_req, const int32_t *n_tokens,
                                     int32_t n_fork, int32_t *copy_src, int32_t *copy_dst,
                                     uint8_t *fork_ok, void *workspace, size_t workspace_bytes,
                                     uint32_t *err_word, kvq_stream_t stream) {
  if (num_pages <= 0 || B <= 0 || MP <= 0 || page_size <= 0 || n_fork < 0) return KVQ_ERR_INVALID_ARG;
  if (!free_stack || !free_count || !page_tags || !page_shares || !block_table || !expected_tags)
    return KVQ_ERR_INVALID_ARG;
  if (n_fork == 0) return KVQ_OK;
  if (!src_req || !dst_req || !n_tokens || !copy_src || !copy_dst || !fork_ok || !workspace)
    return KVQ_ERR_INVALID_ARG;
  if (!aligned256(workspace) || workspace_bytes < kvq_pages_workspace_size(num_pages, B))
    return KVQ_ERR_WORKSPACE;
  const ForkArgs args{free_stack, free_count, page_tags, page_shares, block_table, expected_tags,
                      src_req,    dst_req,    n_tokens,  copy_src,    copy_dst,    fork_ok,
                      static_cast<int32_t *>(workspace), err_word, num_pages, B, MP, page_size, n_fork};
  const cudaError_t e = launch_cluster(fork_kernel, static_cast<int64_t>(n_fork) * MP,
                                       reinterpret_cast<cudaStream_t>(stream), args);
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

extern "C" kvq_status kvq_pages_release(int32_t *free_stack, int32_t *free_count,
                                        int32_t *page_shares, int32_t num_pages,
                                        int32_t *block_table, int32_t B, int32_t MP,
                                        const int32_t *rel_req, const int32_t *rel_first,
                                        const int32_t *rel_npages, int32_t n_rel, void *workspace,
                                        size_t workspace_bytes, uint32_t *err_word,
                                        kvq_stream_t stream) {
  if (num_pages <= 0 || B <= 0 || MP <= 0 || n_rel < 0) return KVQ_ERR_INVALID_ARG;
  if (!free_stack || !free_count || !page_shares || !block_table) return KVQ_ERR_INVALID_ARG;
  if (n_rel == 0) return KVQ_OK;
  if (!rel_req || !rel_npages || !workspace) return KVQ_ERR_INVALID_ARG;
  if (!aligned256(workspace) || workspace_bytes < kvq_pages_workspace_size(num_pages, B))
    return KVQ_ERR_WORKSPACE;
  int32_t *claim = static_cast<int32_t *>(workspace);
  int32_t *gone = claim + up256(4ull * B) / 4, *last = gone + up256(4ull * num_pages) / 4;
  const ReleaseArgs args{free_stack, free_count, page_shares, block_table, rel_req, rel_first,
                         rel_npages, claim,      gone,        last,        err_word, num_pages,
                         B,          MP,         n_rel};
  const cudaError_t e = launch_cluster(release_kernel, static_cast<int64_t>(n_rel) * MP,
                                       reinterpret_cast<cudaStream_t>(stream), args);
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

extern "C" kvq_status kvq_pages_compact(int32_t *free_stack, int32_t *free_count,
                                        uint32_t *page_tags, int32_t *page_shares,
                                        int32_t num_pages, int32_t *block_table,
                                        uint32_t *expected_tags, int32_t B, int32_t MP,
                                        const int32_t *held, int32_t *copy_src, int32_t *copy_dst,
                                        int32_t copy_cap, int32_t *n_moves, void *workspace,
                                        size_t workspace_bytes, uint32_t *err_word,
                                        kvq_stream_t stream) {
  if (num_pages <= 0 || B <= 0 || MP <= 0 || copy_cap < num_pages / 2) return KVQ_ERR_INVALID_ARG;
  if (!free_stack || !free_count || !page_tags || !page_shares || !block_table || !expected_tags)
    return KVQ_ERR_INVALID_ARG;
  if (!held || !n_moves || !workspace || (copy_cap > 0 && (!copy_src || !copy_dst)))
    return KVQ_ERR_INVALID_ARG;
  if (!aligned256(workspace) || workspace_bytes < kvq_pages_workspace_size(num_pages, B))
    return KVQ_ERR_WORKSPACE;
  uint32_t *words = static_cast<uint32_t *>(workspace);
  int32_t *pre = reinterpret_cast<int32_t *>(words) + up256(4ull * num_pages) / 4;
  const CompactArgs args{free_stack, free_count, page_tags, page_shares, block_table, expected_tags,
                         held,       copy_src,   copy_dst,  n_moves,     words,       pre,
                         err_word,   num_pages,  B,         MP,          copy_cap};
  const cudaError_t e = launch_cluster(compact_kernel, static_cast<int64_t>(num_pages),
                                       reinterpret_cast<cudaStream_t>(stream), args);
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}
