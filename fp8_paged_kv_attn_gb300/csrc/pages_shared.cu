// Pages that several requests hold: kvq_pages_fork, kvq_pages_release,
// kvq_pages_compact (include/kvq.h).
//
// shares[p] counts the block-table entries that hold page p beyond the first, so
// a page that kvq_pages_update hands out needs no entry written: 0 is right.
//
// Each call is one cluster of up to 16 CTAs of 1,024 threads.  Its phases depend on
// one another (a fork's pages on the forks before it, a page's place on the stack on
// its last holder in the list) and are ordered by the cluster's hardware barrier, so that a
// call is one launch, whatever its sizes.  What bounds it: for short lists a chain of four to
// seven phases, each a barrier and one or two loads that wait for one another (4 forks of 700
// tokens 9 us, 3 requests released 14, a pool of 2,048 pages moved together 15); for long ones
// the rate at which an SM takes scattered accesses, a 32-byte sector each for 4 or 8 bytes (200
// requests with 36,000 entries released: 47 us on 8 SMs, 25 on 16; a pool of 300,000 pages: 92
// and 54).  A thread has four entries in flight, a warp neighbouring ones (a request's entries a
// CTA at a time, one row behind the other, took 61 us for the pool of 2,048 pages).
//
// Lists are taken in rounds of 1,024 entries: every CTA scans a round's page counts, and
// the round's pages ("items", in list order) are spread over the cluster by a binary
// search of the scan, once a warp's batch.
#include <algorithm>
#include <atomic>
#include <climits>

#include <cooperative_groups.h>

#include "kvq_internal.h"

namespace kvq {

namespace cg = cooperative_groups;

constexpr int kShThreads = 1024;
constexpr int kShCtas = 16;
constexpr int kShBatch = 4;  // items a thread has in flight

struct ShSmem {
  long long pre[kShThreads];  // items of the round before each entry
  long long warp[33];
  int base[kShThreads];  // the entry's first logical page
  int req[kShThreads], other[kShThreads];
  uint8_t on[kShThreads];
  unsigned int bits[4];      // the cluster's error bits, a word a check
  long long sums[kShCtas];   // its CTAs' sums
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

// The same, from the owner `o` of an item a little before e.
__device__ __forceinline__ int sh_owner_from(const ShSmem &sm, int m, long long e, int o) {
#pragma unroll 1
  for (int k = 0; k < 4; ++k) {
    if (o + 1 >= m || sm.pre[o + 1] > e) return o;
    ++o;
  }
  return sh_owner(sm, m, e);
}

// The cluster's error bits up to check c; every thread of the cluster calls it.  Who has bits hands them to
// every CTA (reading the others' words took longer than a phase: 32 warps, eight remote loads each).  A
// check's word is its own: a later one's bits cannot come in while it is read.
__device__ __forceinline__ unsigned int sh_bits(cg::cluster_group &cl, ShSmem &sm, int c, unsigned int bits) {
  if (bits)
    for (unsigned int r = 0; r < cl.num_blocks(); ++r) atomicOr(cl.map_shared_rank(&sm.bits[c], r), bits);
  cl.sync();
  return sm.bits[c];
}

// A sum of this CTA for every CTA, read behind the next barrier of the cluster.
__device__ __forceinline__ void sh_sum(cg::cluster_group &cl, ShSmem &sm, long long sum) {
  if (threadIdx.x < cl.num_blocks()) *cl.map_shared_rank(&sm.sums[cl.block_rank()], threadIdx.x) = sum;
}

// Memory that other CTAs of the cluster write, read behind a barrier of the cluster: never through the
// read-only path.
template <typename T>
__device__ __forceinline__ T vol(const T *p) {
  return __ldcg(p);
}

// A warp takes kShBatch times 32 items in a row.  This thread's first, where the cluster's thread `at` begins;
__device__ __forceinline__ long long sh_first(int at) {
  return static_cast<long long>(at & ~31) * kShBatch + (at & 31);
}
// and the owners of its items e0, e0 + 32, .. below `to` (-1: there is none).
__device__ __forceinline__ void sh_batch(const ShSmem &sm, int m, long long e0, long long to, int (&o)[kShBatch]) {
  int from = sh_owner(sm, m, e0 & ~31ll);
#pragma unroll
  for (int k = 0; k < kShBatch; ++k) {
    const long long e = e0 + 32 * k;
    o[k] = -1;
    if (e < to) o[k] = from = sh_owner_from(sm, m, e, from);
  }
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

constexpr uint8_t kForkBad = 2;  // fork_ok while the call runs: 1 or this, for a fork with an entry that is no page

__global__ void __launch_bounds__(kShThreads, 1) fork_kernel(ForkArgs a) {
  __shared__ ShSmem sm;
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, cta = cl.block_rank(), ctas = cl.num_blocks();
  const int at = cta * kShThreads + tid, threads = ctas * kShThreads;
  grid_dependency_wait();
  allow_dependents();
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
  // ---- every page that a fork takes, or copies, is a page.  A fork that is found bad keeps a mark other than 0: the
  // CTAs lay a round's items out by its flags, each at its own time, and have to find the same ones.
  for (int r0 = 0; r0 < a.n; r0 += kShThreads) {
    const int i = r0 + tid, m = min(kShThreads, a.n - r0);
    long long pages = 0, total;
    if (i < a.n && vol(a.ok + i)) {
      sm.req[tid] = a.src[i];
      pages = (static_cast<long long>(a.tokens[i]) + a.page_size - 1) / a.page_size;
    }
    sm.pre[tid] = sh_scan(pages, sm, &total);
    __syncthreads();
    for (long long e0 = sh_first(at); e0 < total; e0 += static_cast<long long>(kShBatch) * threads) {
      int o[kShBatch], page[kShBatch];
      sh_batch(sm, m, e0, total, o);
#pragma unroll
      for (int k = 0; k < kShBatch; ++k)
        page[k] = o[k] < 0 ? 0 : a.table[static_cast<int64_t>(sm.req[o[k]]) * a.MP + (e0 + 32 * k - sm.pre[o[k]])];
#pragma unroll
      for (int k = 0; k < kShBatch; ++k)
        if (page[k] < 0 || page[k] >= a.num_pages) {
          a.ok[r0 + o[k]] = kForkBad;
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
    const bool valid = i < a.n && vol(a.ok + i) == 1;
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
    for (long long e0 = sh_first(at); e0 < total; e0 += static_cast<long long>(kShBatch) * threads) {
      int64_t to[kShBatch];
      int o[kShBatch], page[kShBatch];
      uint32_t tag[kShBatch];
      sh_batch(sm, m, e0, total, o);
#pragma unroll
      for (int k = 0; k < kShBatch; ++k) {
        page[k] = -1;
        if (o[k] >= 0) {
          const int64_t col = e0 + 32 * k - sm.pre[o[k]], from = static_cast<int64_t>(sm.req[o[k]]) * a.MP + col;
          to[k] = static_cast<int64_t>(sm.other[o[k]]) * a.MP + col;
          page[k] = a.table[from];
          tag[k] = a.expected[from];
        }
      }
#pragma unroll
      for (int k = 0; k < kShBatch; ++k)
        if (page[k] >= 0 && page[k] < a.num_pages) {
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
  int2 *gone;             // [num_pages]: how many entries of the list hold a page, and the last one
  uint32_t *err_word;
  int32_t num_pages, B, MP, n;
};

// Calls f(first item, the table entries of kShBatch items in a row) for the items [from, to) of the list.
// Every thread of the CTA calls f together, with null entries where it has no item.
template <typename F>
__device__ __forceinline__ void sh_items(const ReleaseArgs &a, ShSmem &sm, long long from, long long to,
                                         long long items, F f) {
  const int tid = threadIdx.x;
  long long carry = 0;
  for (int r0 = 0; r0 < a.n && carry < to; r0 += kShThreads) {
    const int j = r0 + tid, m = min(kShThreads, a.n - r0);
    long long total = items;
    if (a.n > kShThreads) {  // a single round is still there
      const long long pre = sh_scan(j < a.n ? a.npages[j] : 0, sm, &total);
      sm.pre[tid] = pre;
      if (j < a.n) {
        sm.req[tid] = a.req[j];
        sm.base[tid] = a.first ? a.first[j] : 0;
      }
      __syncthreads();
    }
    const long long lo = max(from, carry), hi = min(to, carry + total);
    for (long long e0 = lo; e0 < hi; e0 += kShBatch * kShThreads) {
      const long long e = e0 + kShBatch * tid;
      int32_t *entry[kShBatch];
      int o = e < hi ? sh_owner(sm, m, e - carry) : 0;
#pragma unroll
      for (int k = 0; k < kShBatch; ++k) {
        entry[k] = nullptr;
        if (e + k < hi) {
          o = sh_owner_from(sm, m, e + k - carry, o);
          entry[k] = a.table + static_cast<int64_t>(sm.req[o]) * a.MP + sm.base[o] + (e + k - carry - sm.pre[o]);
        }
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
  if (tid < 4) sm.bits[tid] = 0;
  cl.barrier_arrive();
  const int count = *a.count;
  unsigned int bits = count < 0 || count > a.num_pages ? KVQ_ERRBIT_PAGE : 0;
  // ---- the list: requests named once, pages within their rows
  long long items = 0;
  for (int r0 = 0; r0 < a.n; r0 += kShThreads) {
    const int j = r0 + tid;
    long long n = 0, total;
    if (j < a.n) {
      const int b = a.req[j];
      const int f = a.first ? a.first[j] : 0;
      n = a.npages[j];
      sm.req[tid] = b;
      sm.base[tid] = f;
      if (b < 0 || b >= a.B)
        bits |= KVQ_ERRBIT_REQ;
      else if (j % ctas == cta)
        a.claim[b] = INT_MAX;
      if (f < 0 || n < 0 || f + n > a.MP) {
        bits |= KVQ_ERRBIT_POS;
        n = 0;
      }
    }
    sm.pre[tid] = sh_scan(n, sm, &total);
    items += total;
  }
  if (items > INT_MAX) bits |= KVQ_ERRBIT_POS;
  cl.barrier_wait();  // every CTA's words are there
  if (sh_bits(cl, sm, 0, bits)) {
    if (bits) report(a.err_word, bits);
    return;
  }
  for (int j = at; j < a.n; j += threads) atomicMin(a.claim + a.req[j], j);
  // ---- the items: pages, and their counters cleared
  const long long per = (items + ctas - 1) / ctas;
  const long long from = min(items, cta * per), to = min(items, from + per);
  auto pages = [](int32_t *const(&entry)[kShBatch], int (&page)[kShBatch]) {
#pragma unroll
    for (int k = 0; k < kShBatch; ++k) page[k] = entry[k] ? *entry[k] : 0;
  };
  sh_items(a, sm, from, to, items, [&](int, int32_t *const(&entry)[kShBatch]) {
    int page[kShBatch];
    pages(entry, page);
#pragma unroll
    for (int k = 0; k < kShBatch; ++k) {
      if (page[k] < 0 || page[k] >= a.num_pages) {
        bits |= KVQ_ERRBIT_PAGE;
      } else if (entry[k]) {
        a.gone[page[k]] = make_int2(0, -1);
      }
    }
  });
  if (sh_bits(cl, sm, 1, bits)) {
    if (bits) report(a.err_word, bits);
    return;
  }
  for (int j = at; j < a.n; j += threads)  // (a request named twice spoils scratch alone)
    if (vol(a.claim + a.req[j]) != j) bits |= KVQ_ERRBIT_REQ;
  sh_items(a, sm, from, to, items, [&](int e, int32_t *const(&entry)[kShBatch]) {
    int page[kShBatch];
    pages(entry, page);
#pragma unroll
    for (int k = 0; k < kShBatch; ++k)
      if (entry[k]) {
        atomicAdd(&a.gone[page[k]].x, 1);
        atomicMax(&a.gone[page[k]].y, e + k);
      }
  });
  if (sh_bits(cl, sm, 2, bits)) {
    if (bits) report(a.err_word, bits);
    return;
  }
  // ---- a page whose last holder goes is free, and lies on the stack where its last item stands
  int frees = 0;
  // (of an item: whether it is its page's last, how many entries hold the page, its counter)
  struct Held {
    int page[kShBatch], last[kShBatch], gone[kShBatch], shares[kShBatch];
  };
  auto look = [&](int32_t *const(&entry)[kShBatch], Held &h) {
    pages(entry, h.page);
#pragma unroll
    for (int k = 0; k < kShBatch; ++k) {
      h.last[k] = -1;
      h.gone[k] = h.shares[k] = 0;
      if (entry[k]) {
        const int2 g = vol(a.gone + h.page[k]);
        h.gone[k] = g.x;
        h.last[k] = g.y;
        h.shares[k] = vol(a.shares + h.page[k]);
      }
    }
  };
  sh_items(a, sm, from, to, items, [&](int e, int32_t *const(&entry)[kShBatch]) {
    Held h;
    look(entry, h);
#pragma unroll
    for (int k = 0; k < kShBatch; ++k)
      if (entry[k] && h.last[k] == e + k) {
        if (h.shares[k] < 0 || h.gone[k] - 1 > h.shares[k]) bits |= KVQ_ERRBIT_PAGE;  // more often than it is held
        frees += h.gone[k] - 1 == h.shares[k];
      }
  });
  long long freed;
  sh_scan(frees, sm, &freed);
  sh_sum(cl, sm, freed);
  unsigned int any = sh_bits(cl, sm, 3, bits);
  long long before = 0, all = 0;
  for (int r = 0; r < ctas; ++r) {
    const long long f = sm.sums[r];
    before += r < cta ? f : 0;
    all += f;
  }
  if (!any && count + all > a.num_pages) any = bits = KVQ_ERRBIT_PAGE;
  if (any) {
    if (bits) report(a.err_word, bits);
    return;
  }
  sh_items(a, sm, from, to, items, [&](int e, int32_t *const(&entry)[kShBatch]) {
    Held h;
    look(entry, h);
    int free[kShBatch], pushes = 0;
#pragma unroll
    for (int k = 0; k < kShBatch; ++k) {
      free[k] = -1;
      if (!entry[k]) continue;
      *entry[k] = -1;
      if (h.last[k] == e + k) {  // (the page's counter is read here alone)
        const int left = h.shares[k] - h.gone[k];
        a.shares[h.page[k]] = max(left, 0);
        if (left < 0) {
          free[k] = h.page[k];
          ++pushes;
        }
      }
    }
    long long total;
    long long to_stack = count + before + sh_scan(pushes, sm, &total);
#pragma unroll
    for (int k = 0; k < kShBatch; ++k)
      if (free[k] >= 0) a.stack[to_stack++] = free[k];
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

// Calls f(indexes of kShBatch table entries, -1 for none) over the entries that requests hold, spread over
// the cluster.
template <typename F>
__device__ __forceinline__ void sh_held(const CompactArgs &a, ShSmem &sm, int at, int threads, F f) {
  const int tid = threadIdx.x;
  for (int r0 = 0; r0 < a.B; r0 += kShThreads) {
    const int b = r0 + tid, m = min(kShThreads, a.B - r0);
    long long total;
    const long long pre = sh_scan(b < a.B ? a.held[b] : 0, sm, &total);
    sm.pre[tid] = pre;
    __syncthreads();
    for (long long e0 = sh_first(at); e0 < total; e0 += static_cast<long long>(kShBatch) * threads) {
      int o[kShBatch];
      int64_t idx[kShBatch];
      sh_batch(sm, m, e0, total, o);
#pragma unroll
      for (int k = 0; k < kShBatch; ++k)
        idx[k] = o[k] < 0 ? -1 : static_cast<int64_t>(r0 + o[k]) * a.MP + (e0 + 32 * k - sm.pre[o[k]]);
      f(idx);
    }
    __syncthreads();
  }
}

__global__ void __launch_bounds__(kShThreads, 1) compact_kernel(CompactArgs a) {
  __shared__ ShSmem sm;
  __shared__ int s_base[kShCtas];
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, cta = cl.block_rank(), ctas = cl.num_blocks();
  const int at = cta * kShThreads + tid, threads = ctas * kShThreads;
  grid_dependency_wait();
  allow_dependents();
  if (tid < 4) sm.bits[tid] = 0;
  const int words = (a.num_pages + 31) / 32, count = *a.count;
  const int share = (words + ctas - 1) / ctas;  // words a CTA scans
  for (int w = at; w < words; w += threads) a.words[w] = 0;
  unsigned int bits = count < 0 || count > a.num_pages ? KVQ_ERRBIT_PAGE : 0;
  cl.sync();
  if (!bits)
    for (int i0 = at; i0 < count; i0 += kShBatch * threads) {
      int page[kShBatch];
#pragma unroll
      for (int k = 0; k < kShBatch; ++k) page[k] = i0 < count - k * threads ? a.stack[i0 + k * threads] : INT_MAX;
      uint32_t was[kShBatch];
#pragma unroll
      for (int k = 0; k < kShBatch; ++k) {
        was[k] = 0;
        if (page[k] >= 0 && page[k] < a.num_pages)
          was[k] = atomicOr(a.words + (page[k] >> 5), 1u << (page[k] & 31)) >> (page[k] & 31) & 1;
        else if (i0 < count - k * threads)
          bits |= KVQ_ERRBIT_PAGE;
      }
#pragma unroll
      for (int k = 0; k < kShBatch; ++k)
        if (was[k]) bits |= KVQ_ERRBIT_PAGE;  // free twice
    }
  for (int b = at; b < a.B; b += threads)
    if (a.held[b] < 0 || a.held[b] > a.MP) bits |= KVQ_ERRBIT_POS;
  unsigned int any = sh_bits(cl, sm, 0, bits);
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
    sh_sum(cl, sm, carry);
    sh_held(a, sm, at, threads, [&](const int64_t(&idx)[kShBatch]) {
      int page[kShBatch];
#pragma unroll
      for (int k = 0; k < kShBatch; ++k) page[k] = idx[k] < 0 ? INT_MIN : a.table[idx[k]];
#pragma unroll
      for (int k = 0; k < kShBatch; ++k) {
        if (idx[k] < 0) continue;
        if (page[k] < 0 || page[k] >= a.num_pages || (a.words[page[k] >> 5] >> (page[k] & 31) & 1))
          bits |= KVQ_ERRBIT_PAGE;
      }
    });
    any = sh_bits(cl, sm, 1, bits);
    if (tid == 0) {
      int base = 0;
      for (int r = 0; r < ctas; ++r) {
        s_base[r] = base;
        base += static_cast<int>(sm.sums[r]);
      }
    }
    __syncthreads();
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
    const uint32_t word = a.words[w];
    is_free = word >> (id & 31) & 1;
    return s_base[w / share] + a.pre[w] + __popc(word & ((1u << (id & 31)) - 1));
  };
  bool unused;
  const int holes = live < a.num_pages ? free_below(live, unused) : count;
  const int stay = live - holes;  // live pages below `live`
  for (int w = at; w < words; w += threads) {
    const uint32_t word = a.words[w];
    int f = s_base[w / share] + a.pre[w];  // free pages below
    const int first = 32 * w, here = min(32, a.num_pages - first), low = min(max(live - first, 0), here);
    const uint32_t below = low == 32 ? ~0u : (1u << low) - 1, all = here == 32 ? ~0u : (1u << here) - 1;
    for (uint32_t x = word & below; x; x &= x - 1) {
      const int id = first + __ffs(x) - 1;
      a.copy_dst[f++] = id;
      atomicAdd(a.tags + id, 1u);
    }
    for (uint32_t x = ~word & ~below & all; x; x &= x - 1) {
      const int bit = __ffs(x) - 1;
      a.copy_src[first + bit - (f + __popc(word & ~below & ((1u << bit) - 1))) - stay] = first + bit;
    }
  }
  for (int i = at; i < count; i += threads) a.stack[i] = a.num_pages - 1 - i;
  for (int k = holes + at; k < a.cap; k += threads) a.copy_src[k] = a.copy_dst[k] = -1;
  cl.sync();
  for (int i0 = at; i0 < holes; i0 += kShBatch * threads) {
    int from[kShBatch], to[kShBatch], held[kShBatch];
#pragma unroll
    for (int k = 0; k < kShBatch; ++k)
      if (i0 < holes - k * threads) {
        from[k] = a.copy_src[i0 + k * threads];
        to[k] = a.copy_dst[i0 + k * threads];
      }
#pragma unroll
    for (int k = 0; k < kShBatch; ++k)
      if (i0 < holes - k * threads) held[k] = a.shares[from[k]];
#pragma unroll
    for (int k = 0; k < kShBatch; ++k)
      if (i0 < holes - k * threads) {
        a.shares[to[k]] = held[k];
        a.shares[from[k]] = 0;
      }
  }
  sh_held(a, sm, at, threads, [&](const int64_t(&idx)[kShBatch]) {
    int page[kShBatch], to[kShBatch];
    uint32_t tag[kShBatch];
#pragma unroll
    for (int k = 0; k < kShBatch; ++k) page[k] = idx[k] < 0 ? -1 : a.table[idx[k]];
#pragma unroll
    for (int k = 0; k < kShBatch; ++k) {
      to[k] = -1;
      if (page[k] < live) continue;
      bool is_free;
      const int f = free_below(page[k], is_free);
      to[k] = a.copy_dst[page[k] - f - stay];
    }
#pragma unroll
    for (int k = 0; k < kShBatch; ++k)
      if (to[k] >= 0) tag[k] = a.tags[to[k]];
#pragma unroll
    for (int k = 0; k < kShBatch; ++k)
      if (to[k] >= 0) {
        a.table[idx[k]] = to[k];
        a.expected[idx[k]] = tag[k];
      }
  });
  if (at == 0) *a.moves = holes;
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

namespace {

// The kernels step through their lists with 32-bit counters, up to 65,536 ahead.
bool sh_sizes_ok(int32_t num_pages, int32_t B, int32_t list) {
  return std::max({num_pages, B, list}) <= 1 << 30;
}

size_t up256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

// The largest cluster of the current device: 16 CTAs have to be asked for, and may not fit.
template <typename Args>
unsigned cluster_ctas(void (*kernel)(Args)) {
  constexpr int kMaxDev = 64;
  static std::atomic<unsigned> most[kMaxDev];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return 8;
  unsigned ctas = most[dev].load(std::memory_order_acquire);
  if (ctas) return ctas;
  ctas = 8;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = kShCtas;
    cfg.blockDim = kShThreads;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = kShCtas;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int fit = 0;
    if (cudaOccupancyMaxActiveClusters(&fit, kernel, &cfg) != cudaSuccess)
      cudaGetLastError();
    else if (fit > 0)
      ctas = kShCtas;
  } else {
    cudaGetLastError();
  }
  most[dev].store(ctas, std::memory_order_release);
  return ctas;
}

// One cluster: a single CTA where a few thousand items at most are in hand, else the largest (16 CTAs
// against one: 176 entries forked 11.0 us and 9.0, 8,000 12.3 and 17.0, 32,000 15 and 40; 2,048 pages moved
// together 16 and 14.5, 8,192 18 and 20.5).  Items are what the lists may hold for forks and releases, and for
// compaction the pool's pages, which its tables hold many times over where most are shared: 4,096 pages held by 512
// requests of 1,000 entries take one CTA 616 us, 4,097 the cluster 51.
template <typename Args>
cudaError_t launch_cluster(void (*kernel)(Args), int64_t items, cudaStream_t stream, const Args &args) {
  const unsigned ctas = items <= 4 * kShThreads ? 1 : cluster_ctas(kernel);
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
  if (num_pages <= 0 || B <= 0 || !sh_sizes_ok(num_pages, B, 0)) return 0;
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
  if (num_pages <= 0 || B <= 0 || MP <= 0 || page_size <= 0 || n_fork < 0 || !sh_sizes_ok(num_pages, B, n_fork))
    return KVQ_ERR_INVALID_ARG;
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
  if (num_pages <= 0 || B <= 0 || MP <= 0 || n_rel < 0 || !sh_sizes_ok(num_pages, B, n_rel)) return KVQ_ERR_INVALID_ARG;
  if (!free_stack || !free_count || !page_shares || !block_table) return KVQ_ERR_INVALID_ARG;
  if (n_rel == 0) return KVQ_OK;
  if (!rel_req || !rel_npages || !workspace) return KVQ_ERR_INVALID_ARG;
  if (!aligned256(workspace) || workspace_bytes < kvq_pages_workspace_size(num_pages, B))
    return KVQ_ERR_WORKSPACE;
  int32_t *claim = static_cast<int32_t *>(workspace);
  int2 *gone = reinterpret_cast<int2 *>(claim + up256(4ull * B) / 4);
  const ReleaseArgs args{free_stack, free_count, page_shares, block_table, rel_req, rel_first,
                         rel_npages, claim,      gone,        err_word,    num_pages,
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
  if (num_pages <= 0 || B <= 0 || MP <= 0 || copy_cap < num_pages / 2 || !sh_sizes_ok(num_pages, B, copy_cap))
    return KVQ_ERR_INVALID_ARG;
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
