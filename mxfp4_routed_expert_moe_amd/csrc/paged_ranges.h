// Which rows, keys and pages a sequence of the paged operators has, from the
// caller's int32 arrays.  Host and device code, so that every value those arrays
// can hold is tested on the CPU.
#pragma once

#include <cstdint>

#include "attention_ranges.h"

namespace moe {

struct PagedRange {
  int q0, lq;    // rows of q
  int diag;      // Lk - Lq of the lengths as given: row i is at position i + diag
  int own, end;  // the keys behind the shared prefix: own .. end - 1
};

// The keys of a prefix that are read once for all of its group: the pages that it
// fills.
__host__ __device__ inline int shared_keys(int prefix_len, int max_prefix, int page_shift) {
  return min_of(max_of(prefix_len, 0), max_prefix) >> page_shift << page_shift;
}

// The keys of a sequence (rows and diag are set) behind its prefix.
__host__ __device__ inline void behind_prefix(PagedRange& s, int prefix, int max_prefix, int max_kv, int capacity,
                                              int page_shift) {
  s.own = shared_keys(prefix, max_prefix, page_shift);
  s.end = min_of(s.diag + s.lq, min_of(capacity, min_of(max_of(prefix, 0), max_prefix) + max_kv));
}

// Sequence b, whose group's prefix_len is `prefix` (0: no group).  capacity =
// table_pages * page_size; max_prefix, max_kv <= capacity < 2^30.  Both ends of
// the rows are cut before one is taken from the other: the difference of two
// entries as they come may need 33 bits.
__host__ __device__ inline PagedRange paged_range(const int32_t* cu_q, const int32_t* kv_len, int b, int q_rows,
                                                  int capacity, int prefix, int max_prefix, int max_kv,
                                                  int page_shift) {
  PagedRange s;
  s.q0 = min_of(max_of(cu_q[b], 0), q_rows);
  s.lq = min_of(max_of(cu_q[b + 1], s.q0), q_rows) - s.q0;
  s.diag = max_of(kv_len[b], 0) - s.lq;
  behind_prefix(s, prefix, max_prefix, max_kv, capacity, page_shift);
  return s;
}

// The last key that row pos < lq sees (-1 or less: none).
__host__ __device__ inline int last_key(const PagedRange& s, int pos) { return min_of(pos + s.diag, s.end - 1); }

// The first and one past the last sequence of group g.
struct GroupRange {
  int first, past;
};
__host__ __device__ inline GroupRange group_range(const int32_t* cu_group, int g, int n_seqs) {
  GroupRange r;
  r.first = min_of(max_of(cu_group[g], 0), n_seqs);
  r.past = min_of(max_of(cu_group[g + 1], r.first), n_seqs);
  return r;
}

// What a block does with split `split` of a tile that sees the keys of `splits` splits (0: none), where a row
// has `slots` shares: attend to it, write an empty share in its place, or nothing.  every_slot: the join reads all
// of a row's shares, so each of them is written.  A row of one share has no shares in the workspace, which there
// may be none of: its tile writes the output itself, also where it sees nothing.
enum class SplitWork { kAttend, kEmpty, kNothing };
__host__ __device__ inline SplitWork split_work(int split, int splits, int slots, bool every_slot) {
  const bool shares = every_slot && slots > 1;
  if (split < splits || (split == 0 && !shares)) return SplitWork::kAttend;
  return shares ? SplitWork::kEmpty : SplitWork::kNothing;
}

}  // namespace moe
