// Which rows and keys a sequence of moe_attention has, from the caller's int32
// arrays.  Host and device code, so that every value those arrays can hold is
// tested on the CPU.
#pragma once

#include <cstdint>

namespace moe {

// By value: references to the fields would keep a struct in scratch memory.
__host__ __device__ inline int min_of(int a, int b) { return a < b ? a : b; }
__host__ __device__ inline int max_of(int a, int b) { return a > b ? a : b; }

struct SeqRange {
  int q0, lq;  // rows of q
  int k0, lk;  // rows of k and v that there are to see
  int diag;    // Lk - Lq of the lengths as given: query i sees keys j <= i + diag
};

// Rows cu_q[b] .. cu_q[b + 1] - 1 of q and the keys kv_start[b] .. of length
// kv_len[b] (NULL: the rows of q), cut to the tensors and to max_kv.  Both ends of
// the rows are cut before one is taken from the other: the difference of two
// entries as they come may need 33 bits.  A cut of the keys takes keys away, and does
// not move the diagonal.
__host__ __device__ inline SeqRange seq_range(const int32_t* cu_q, const int32_t* kv_start, const int32_t* kv_len, int b,
                                              int q_rows, int kv_rows, int max_kv) {
  SeqRange s;
  s.q0 = min_of(max_of(cu_q[b], 0), q_rows);
  s.lq = min_of(max_of(cu_q[b + 1], s.q0), q_rows) - s.q0;
  s.k0 = kv_start ? min_of(max_of(kv_start[b], 0), kv_rows) : min_of(s.q0, kv_rows);
  const int lk = kv_start ? max_of(kv_len[b], 0) : s.lq;
  s.lk = min_of(lk, min_of(kv_rows - s.k0, max_kv));
  s.diag = lk - s.lq;
  return s;
}

// The last key that query pos < lq sees (-1 or less: none).
__host__ __device__ inline int last_key(const SeqRange& s, int causal, int pos) {
  return causal ? min_of(pos + s.diag, s.lk - 1) : s.lk - 1;
}

}  // namespace moe
