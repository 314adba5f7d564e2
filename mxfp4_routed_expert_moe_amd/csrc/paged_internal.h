// What the paged operators share: the sequences of a call and their pages, on the
// device, and the host's checks of them.
#pragma once

#include "../../include/moe_paged.h"
#include "moe_internal.h"
#include "paged_ranges.h"

namespace moe {

struct PagedSeqs {
  const int32_t *cu_q, *kv_len, *table;
  int64_t table_stride;
  int n_seqs, q_rows, n_pages, shift, table_pages, capacity;
};

// Uniform loads of the caller's arrays through the scalar cache: nothing that a kernel
// here writes overlaps them.
typedef const __attribute__((address_space(4))) int32_t* ConstInts;
__device__ __forceinline__ ConstInts const_ints(const int32_t* p) { return (ConstInts)p; }

// Inclusive prefix sum over the 64 lanes of a wave, in the vector unit alone: every
// block of these kernels looks its work up, before it can load anything.
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_or_zero(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 15, false);
}
__device__ __forceinline__ int wave_prefix(int v) {
  v += dpp_or_zero<0x111, 15>(v);  // row_shr 1, 2, 4, 8: inside 16 lanes
  v += dpp_or_zero<0x112, 15>(v);
  v += dpp_or_zero<0x114, 15>(v);
  v += dpp_or_zero<0x118, 15>(v);
  v += dpp_or_zero<0x142, 10>(v);  // lane 15 of rows 0 and 2 to rows 1 and 3
  v += dpp_or_zero<0x143, 12>(v);  // lane 31 to rows 2 and 3
  return v;
}
// The value of a lane that all lanes name.
__device__ __forceinline__ int lane_value(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }

__host__ inline bool paged_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

inline int check_paged_heads(const moe_heads& h) {
  if (!h.base || h.row_stride <= 0 || h.head_stride <= 0) return MOE_EINVAL;
  if (!paged_aligned16(h.base) || h.row_stride % 8 != 0 || h.head_stride % 8 != 0) return MOE_EALIGN;
  return MOE_OK;
}

inline int check_pages(const moe_pages& h) {
  if (!h.base || h.page_stride <= 0 || h.row_stride <= 0 || h.head_stride <= 0) return MOE_EINVAL;
  if (!paged_aligned16(h.base) || h.page_stride % 8 != 0 || h.row_stride % 8 != 0 || h.head_stride % 8 != 0)
    return MOE_EALIGN;
  return h.row_stride > (1 << 22) ? MOE_ESHAPE : MOE_OK;  // a page spans less than 2^31 bytes
}

// The shape fields.
inline int check_paged_shape(const moe_paged& p, bool q_optional) {
  if (p.abi_version != MOE_ABI_VERSION) return MOE_ELAYOUT;
  if (p.n_seqs < 0 || p.q_rows < 0 || p.n_pages < 0 || p.table_pages < 0 || p.q_heads < 0 || p.reserved != 0)
    return MOE_EINVAL;
  if (p.head_dim != 64 && p.head_dim != 128 && p.head_dim != 256) return MOE_ESHAPE;
  if (p.page_size != 16 && p.page_size != 32 && p.page_size != 64 && p.page_size != 128) return MOE_ESHAPE;
  if (p.kv_heads < 1 || p.kv_heads > 1024 || p.q_heads > 1024 || p.q_heads % p.kv_heads != 0) return MOE_ESHAPE;
  if (p.q_heads == 0 && !q_optional) return MOE_ESHAPE;
  if (p.n_seqs > 65536 || p.q_rows > MOE_MAX_TOKENS) return MOE_ESHAPE;
  if (static_cast<int64_t>(p.table_pages) * p.page_size >= (1 << 30)) return MOE_ESHAPE;
  return MOE_OK;
}

// The arrays (of a call that has rows and sequences).
inline int check_paged_arrays(const moe_paged& p) {
  if (!p.cu_q || !p.kv_len) return MOE_EINVAL;
  if (p.table_pages > 0 && (!p.page_table || p.table_stride < p.table_pages)) return MOE_EINVAL;
  return MOE_OK;
}

inline PagedSeqs paged_seqs(const moe_paged& p) {
  PagedSeqs s;
  s.cu_q = p.cu_q, s.kv_len = p.kv_len, s.table = p.page_table, s.table_stride = p.table_stride;
  s.n_seqs = p.n_seqs, s.q_rows = p.q_rows, s.n_pages = p.n_pages;
  s.shift = __builtin_ctz(static_cast<unsigned>(p.page_size));
  s.table_pages = p.n_pages > 0 ? p.table_pages : 0;  // a cache without pages holds nothing
  s.capacity = s.table_pages << s.shift;
  return s;
}

}  // namespace moe
