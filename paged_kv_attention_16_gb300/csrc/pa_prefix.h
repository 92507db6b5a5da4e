// pa_prefix.h -- what the kernels of pa_forward_shared_prefix share: the plan
// of the prefix part and its work items (not part of the public C ABI).
#pragma once

#include "pa_internal.h"

namespace pa {

// Rows of one work item of the prefix part: two 128-row query tiles, a row
// being one (token, query head) of the item's KV head.
constexpr int kPrefixRows = 256;
// KV positions per tile; splits are whole tiles.
constexpr int kPrefixTile = 128;
// Items the splits may add on top of one per (KV head, 256 rows, group):
// four per SM of a 160-SM part.  Bounds the partials' storage.
constexpr int kPrefixSplitItems = 640;

struct PrefixGroup {
  int q_start;      // first token row of the group's requests
  int q_len;        // their token rows
  int req0;         // first request: its block-table row names the prefix's pages
  int prefix;       // shared positions (0: no prefix part)
  int nrp;          // 256-row blocks of a KV head: ceil(q_len * G / 256)
  int nsplit;       // splits of the prefix
  int split_len;    // positions per split, a multiple of kPrefixTile
  int item0;        // first item; item = item0 + (kv head * nsplit + split) * nrp + block
};

struct PrefixPlan {
  int n_items;
  int all_bad;  // bad query_start_loc or group_start_loc, or no room: every row is zero
};

// Partials of the prefix part: row r (0 .. 255) of item x is row x * 256 + r of
// part_o [.., head_dim] (normalised by its own weights' sum) and part_lse
// (base 2; NaN marks a bad page in the item's range).
struct PrefixParams {
  FwdParams f;  // the call, and the plan of the positions behind the prefixes
  const void *k_cache, *v_cache;
  const int32_t *group_start, *prefix_lens;
  int num_groups, max_prefix_len, num_sms;
  PrefixPlan *plan;
  PrefixGroup *grp;     // [num_groups]
  int *grp_end;         // [num_groups] inclusive prefix sum of the items
  int *req_grp;         // [num_seqs] group of each request
  float *part_o, *part_lse;
  long long item_cap;
};

struct PrefixItem {
  int q_start, q_len, req0;  // the group's rows, and the row of its pages
  int kvh, t0;               // first token of the item (within the group)
  int kv_lo, kv_hi;          // positions of its split
};

// g0: group 0, loaded beside the number of items (most batches have one group).
__device__ inline PrefixItem prefix_item(const PrefixParams &p, const PrefixGroup &g0, int item,
                                         int G) {
  int lo = 0, hi = p.num_groups - 1;
  while (lo < hi) {  // the first group that ends behind the item
    const int mid = (lo + hi) >> 1;
    if (p.grp_end[mid] > item) hi = mid; else lo = mid + 1;
  }
  PrefixGroup g = g0;
  if (lo) g = p.grp[lo];
  const unsigned local = item - g.item0, rest = local / (unsigned)g.nrp;
  PrefixItem it;
  it.q_start = g.q_start;
  it.q_len = g.q_len;
  it.req0 = g.req0;
  it.t0 = (int)(local - rest * g.nrp) * (kPrefixRows / G);
  it.kvh = (int)(rest / (unsigned)g.nsplit);
  it.kv_lo = (int)(rest % (unsigned)g.nsplit) * g.split_len;
  it.kv_hi = min(it.kv_lo + g.split_len, g.prefix);
  return it;
}

// The prefix part of bf16 calls (tensor cores).
cudaError_t launch_prefix_mma(const PrefixParams &p, int kv_layout, int num_sms,
                              cudaStream_t stream);

}  // namespace pa
