// What the kernels of kvq_block_prefix_attn share: the plan of a call, and how a row's sums are kept
// until they are merged.
#pragma once

#include "block_common.cuh"

namespace kvq {

// A row's sums are D floats and four statistics: m, l, n (block_attn.cu), and where they are.
constexpr int kStat = 4;
// The fourth: here; in the parts of several CTAs (then the first two are the first CTA and how many);
// or nowhere, the row is written.
constexpr float kHere = 1.f, kCut = 2.f, kDone = 3.f;

// An item: the prefix of a group for all its rows, or a request's own tokens for its rows.
struct __align__(16) PxItem {
  int b;           // whose block table
  int row0, n;     // token rows
  int rows;        // rows: token rows times heads a kv head
  int first, end;  // tokens [first, end)
  int p0;          // position of its first row (own tokens)
  int nb;          // blocks of rows
  int own, pre;    // pre: own tokens behind a prefix
  int live;        // 0: a request whose rows are zeros
  int row_pre;     // the first row of its group
};

struct PxPlan {
  int64_t total, per;  // units, and units a CTA
  int n_grp, n_req;    // items
};

__device__ __forceinline__ PxItem px_load_item(const PxItem *at) {
  PxItem o;
  const int4 *p = reinterpret_cast<const int4 *>(at);
  int4 *q = reinterpret_cast<int4 *>(&o);
#pragma unroll
  for (int k = 0; k < 3; ++k) q[k] = __ldcg(p + k);
  return o;
}

}  // namespace kvq
