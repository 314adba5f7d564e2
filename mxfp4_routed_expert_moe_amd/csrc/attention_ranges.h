// Which rows and keys a sequence of moe_attention has, from the caller's int32
// arrays.  Host and device code, so that every value those arrays can hold is
// tested on the CPU.
#pragma once

#include <algorithm>
#include <cstdint>

namespace moe {

struct SeqRange {
  int q0, lq;  // rows of q
  int k0, lk;  // rows of k and v
};

// Rows cu_q[b] .. cu_q[b + 1] - 1 of q and the keys kv_start[b] .. of length
// kv_len[b] (NULL: the rows of q), cut to the tensors and to max_kv.  Both ends of
// the rows are cut before one is taken from the other: the difference of two
// entries as they come may need 33 bits.
__host__ __device__ inline SeqRange seq_range(const int32_t* cu_q, const int32_t* kv_start, const int32_t* kv_len, int b,
                                              int q_rows, int kv_rows, int max_kv) {
  SeqRange s;
  s.q0 = std::min(std::max(cu_q[b], 0), q_rows);
  s.lq = std::min(std::max(cu_q[b + 1], s.q0), q_rows) - s.q0;
  if (kv_start) {
    s.k0 = std::min(std::max(kv_start[b], 0), kv_rows);
    s.lk = std::max(std::min(kv_len[b], kv_rows - s.k0), 0);
  } else {
    s.k0 = std::min(s.q0, kv_rows);
    s.lk = std::min(s.lq, kv_rows - s.k0);
  }
  s.lk = std::min(s.lk, max_kv);
  return s;
}

}  // namespace moe
