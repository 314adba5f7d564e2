// The blocks of a paged cache that each token's queries promise to need
// (include/moe_paged.h, moe_select_blocks).
//
// For a query element x and bounds low <= k <= high, x k is at most max(x low, x high)
// = max(x, 0) high + min(x, 0) low.  Summed over the query heads of a key head, the
// score of a page is Q+ . high + Q- . low with Q+ = sum max(x, 0), Q- = sum min(x, 0): one
// dot product of 2 D columns per token, key head and page, whatever the group.
//
// Two tokens' scores that differ in the last bits of float32 must still be ordered as
// defined, so everything is summed in float64 (products of bf16 values are exact there), which
// this card does at the rate of float32.
//
// Scores go to the workspace as integers that order as they do; then a wave (or a block,
// for many pages) holds a token's scores in registers, finds the n-th largest by
// bisecting its bits with counts over the wave, and writes the blocks at or above it in
// order, the first ones of those that are equal to it.
#include <algorithm>

#include "paged_internal.h"

namespace moe {

namespace {

struct SelectArgs {
  PagedSeqs s;
  moe_heads q;
  const uint16_t* bounds;
  int32_t* blocks;
  uint64_t* keys;  // [rows of this launch, kv_heads, stride]
  int q_heads, kv_heads, group, max_q, max_kv, n_blocks, first, last;
  int row0, rows, stride;
};

// Orders: a block that the row does not see, a page that is none, finite scores, scores that are
// not finite, blocks that are always taken.
constexpr uint64_t kHidden = 0, kNone = 1, kLargest = ~uint64_t{1}, kAlways = ~uint64_t{0};

__device__ __forceinline__ uint64_t order_key(double score) {
  const uint64_t b = __builtin_bit_cast(uint64_t, score + 0.0);  // -0 and 0 are equal
  if ((b & 0x7ff0000000000000u) == 0x7ff0000000000000u) return kLargest;
  return b >> 63 ? ~b : b | 0x8000000000000000u;
}

__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }

// A row's sequence and its last key (-1: it sees none, -2: it is no sequence's).
struct RowWork {
  int seq, last;
};
__device__ __forceinline__ RowWork find_row(const SelectArgs& a, int row) {
  int lo = 0, hi = a.s.n_seqs;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.s.cu_q[mid] <= row) lo = mid; else hi = mid;
  }
  const PagedRange r = paged_range(a.s.cu_q, a.s.kv_len, lo, a.s.q_rows, a.s.capacity, 0, 0, a.max_kv, a.s.shift);
  const int pos = row - r.q0;
  RowWork w;
  w.seq = lo;
  w.last = pos < 0 || pos >= min(r.lq, a.max_q) ? -2 : max(last_key(r, pos), -1);
  return w;
}

__device__ __forceinline__ void unpack8(u32x4 w, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ double shfl_xor_f64(double v, int mask) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __shfl_xor(static_cast<uint32_t>(b), mask, 64);
  const uint32_t hi = __shfl_xor(static_cast<uint32_t>(b >> 32), mask, 64);
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

// ---------------------------------------------------------------- scores
// Block x: pages kPages x .. of one row and key head.  A group of L = D / 8 lanes takes
// a page at a time, eight columns a lane.
constexpr int kPages = 64;

template <int L>
__global__ __launch_bounds__(256) void score_kernel(SelectArgs a) {
  constexpr int D = 8 * L, kGroups = 256 / L, kEach = kPages / kGroups;
  const int item = blockIdx.y, head = item % a.kv_heads, row = a.row0 + item / a.kv_heads;
  const RowWork w = find_row(a, row);
  const int n = (w.last >> a.s.shift) + 1;  // blocks that the row sees (last = -2: 0)
  const int b0 = blockIdx.x * kPages;
  if (n <= a.n_blocks || b0 >= n) return;  // all of them are taken
  const int grp = threadIdx.x / L, e0 = 8 * (threadIdx.x % L);
  const int32_t* table = a.s.table + w.seq * a.s.table_stride;
  int page[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int b = b0 + i * kGroups + grp;
    page[i] = table[min(b, n - 1)];
  }
  u32x4 low[kEach], high[kEach];
  bool ok[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    ok[i] = page[i] >= 0 && page[i] < a.s.n_pages;
    const uint16_t* p = a.bounds + (static_cast<int64_t>(ok[i] ? page[i] : 0) * 2 * a.kv_heads + head) * D + e0;
    low[i] = ld16(p);
    high[i] = ld16(p + static_cast<int64_t>(a.kv_heads) * D);
  }
  double up[8], down[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) up[j] = down[j] = 0.0;
  const uint16_t* q = a.q.base + row * a.q.row_stride + head * a.group * a.q.head_stride + e0;
  for (int g = 0; g < a.group; ++g) {
    float x[8];
    unpack8(ld16(q + g * a.q.head_stride), x);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // NaN goes to both
      up[j] += x[j] < 0.f ? 0.0 : static_cast<double>(x[j]);
      down[j] += x[j] > 0.f ? 0.0 : static_cast<double>(x[j]);
    }
  }
  uint64_t* out = a.keys + static_cast<int64_t>(item) * a.stride;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    float l[8], h[8];
    unpack8(low[i], l);
    unpack8(high[i], h);
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sum = __builtin_fma(up[j], static_cast<double>(h[j]), sum);
      sum = __builtin_fma(down[j], static_cast<double>(l[j]), sum);
    }
#pragma unroll
    for (int off = 1; off < L; off <<= 1) sum += shfl_xor_f64(sum, off);
    const int b = b0 + i * kGroups + grp;
    if (threadIdx.x % L == 0 && b < n) out[b] = ok[i] ? order_key(sum) : kNone;
  }
}

// ---------------------------------------------------------------- choice
// WAVES waves hold 64 * PER scores each, wave w those from 64 * PER * w on.  Blocks of
// one wave per token and head stand four in a workgroup.
template <int WAVES, int PER>
__global__ __launch_bounds__(WAVES == 1 ? 256 : 64 * WAVES) void choose_kernel(SelectArgs a) {
  __shared__ int s_count[2][WAVES == 1 ? 1 : WAVES];
  const int lane = threadIdx.x & 63;
  const int wave = WAVES == 1 ? 0 : uni(threadIdx.x >> 6);
  const int item = WAVES == 1 ? uni(blockIdx.x * 4 + (threadIdx.x >> 6)) : blockIdx.x;
  if (item >= a.rows * a.kv_heads) return;
  const int head = item % a.kv_heads, row = a.row0 + item / a.kv_heads;
  const RowWork w = find_row(a, row);
  if (w.last == -2) return;
  const int n = (w.last >> a.s.shift) + 1;
  int32_t* out = a.blocks + (static_cast<int64_t>(row) * a.kv_heads + head) * a.n_blocks;
  if (n <= a.n_blocks) {
    for (int i = threadIdx.x & (64 * WAVES - 1); i < a.n_blocks; i += 64 * WAVES) out[i] = i < n ? i : -1;
    return;
  }
  const uint64_t* keys = a.keys + static_cast<int64_t>(item) * a.stride;
  const int base = 64 * PER * wave;
  uint64_t key[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int b = base + 64 * j + lane;
    key[j] = kHidden;
    if (b < n) key[j] = b < a.first || b >= n - a.last ? kAlways : keys[b];
  }
  int parity = 0;
  // the sum of a wave's count over the waves
  auto total = [&](int c) {
    if (WAVES == 1) return c;
    if (lane == 0) s_count[parity][wave] = c;
    __syncthreads();
    int sum = 0;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) sum += s_count[parity][i];
    parity ^= 1;  // the next call writes the other half, so one barrier a call is enough
    return sum;
  };
  auto count = [&](uint64_t from) {
    int c = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) c += __popcll(__ballot(key[j] >= from));
    return total(uni(c));
  };
  // The largest t with at least n_blocks keys from t on; n > n_blocks, so t >= kNone.
  // One with exactly n_blocks ends the search.
  uint64_t t = 0;
  for (int bit = 63; bit >= 0; --bit) {
    const uint64_t c = t | uint64_t{1} << bit;
    const int m = count(c);
    if (m >= a.n_blocks) t = c;
    if (m == a.n_blocks) break;
  }
  // keys above t are all taken; of those equal to t the first ones
  int above = 0, equal = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    above += __popcll(__ballot(key[j] > t));
    equal += __popcll(__ballot(key[j] == t));
  }
  above = uni(above), equal = uni(equal);
  int above_before = 0, equal_before = 0, above_all = above;
  if (WAVES > 1) {
    __syncthreads();
    if (lane == 0) s_count[0][wave] = above, s_count[1][wave] = equal;
    __syncthreads();
    above_all = 0;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) {
      if (i < wave) above_before += s_count[0][i], equal_before += s_count[1][i];
      above_all += s_count[0][i];
    }
  }
  const int want = a.n_blocks - above_all;  // of the equal ones
  const uint64_t below = (uint64_t{1} << lane) - 1;
  int at = above_before + min(equal_before, want), seen = equal_before;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const uint64_t gt = __ballot(key[j] > t), eq = __ballot(key[j] == t);
    const bool take_eq = key[j] == t && seen + __popcll(eq & below) < want;
    const uint64_t take = gt | __ballot(take_eq);
    if (take >> lane & 1) out[at + __popcll(take & below)] = base + 64 * j + lane;
    at += __popcll(take);
    seen += __popcll(eq);
  }
}

// ---------------------------------------------------------------- host
constexpr int kMaxPages = 32768;
constexpr size_t kBatchBytes = size_t{1} << 28;  // of scores at a time

inline int score_stride(const moe_select& d) {
  const int pages = (d.max_kv + d.p.page_size - 1) / d.p.page_size;
  return std::max((pages + 7) / 8 * 8, 8);
}
// Rows of a launch: their scores fit kBatchBytes, and the grid 65535 blocks along y.
inline int batch_rows(const moe_select& d) {
  const size_t row = static_cast<size_t>(d.p.kv_heads) * score_stride(d) * 8;
  const size_t rows = std::min(std::max(kBatchBytes / row, size_t{1}), static_cast<size_t>(65535 / d.p.kv_heads));
  return static_cast<int>(std::min(rows, static_cast<size_t>(std::max(d.p.q_rows, 1))));
}
inline size_t ws_bytes_for(const moe_select& d) {
  return static_cast<size_t>(batch_rows(d)) * d.p.kv_heads * score_stride(d) * 8;
}

int check_shape(const moe_select* a) {
  if (!a) return MOE_EINVAL;
  const int st = check_paged_shape(a->p, false);
  if (st != MOE_OK) return st;
  const int64_t capacity = static_cast<int64_t>(a->p.table_pages) * a->p.page_size;
  if (a->max_q < 0 || a->max_q > a->p.q_rows || a->max_kv < 0 || a->max_kv > capacity || a->reserved != 0)
    return MOE_EINVAL;
  if (a->n_blocks < 1 || a->first < 0 || a->last < 1) return MOE_EINVAL;
  if (a->n_blocks > 1024 || a->max_kv > static_cast<int64_t>(kMaxPages) * a->p.page_size) return MOE_ESHAPE;
  if (a->first > a->n_blocks || a->last > a->n_blocks - a->first) return MOE_EINVAL;
  return MOE_OK;
}

template <int L>
void launch(SelectArgs a, int step, hipStream_t s) {
  const int rows = a.rows, pages = a.stride;
  for (int r = 0; r < rows; r += step) {
    a.row0 = r;
    a.rows = std::min(step, rows - r);
    const unsigned items = static_cast<unsigned>(a.rows) * a.kv_heads;
    score_kernel<L><<<dim3((pages + kPages - 1) / kPages, items), 256, 0, s>>>(a);
    if (pages <= 512)
      choose_kernel<1, 8><<<(items + 3) / 4, 256, 0, s>>>(a);
    else if (pages <= 2048)
      choose_kernel<16, 2><<<items, 1024, 0, s>>>(a);
    else if (pages <= 8192)
      choose_kernel<16, 8><<<items, 1024, 0, s>>>(a);
    else
      choose_kernel<16, 32><<<items, 1024, 0, s>>>(a);
  }
}

}  // namespace
}  // namespace moe

extern "C" {

size_t moe_select_blocks_workspace_size(const moe_select* a) {
  if (moe::check_shape(a) != MOE_OK || a->p.n_seqs == 0 || a->p.q_rows == 0 || a->max_q == 0) return 0;
  return moe::ws_bytes_for(*a);
}

int moe_select_blocks(const moe_select* a, void* ws, size_t ws_bytes, void* stream) {
  int st = moe::check_shape(a);
  if (st != MOE_OK) return st;
  const moe_paged& p = a->p;
  if (p.n_seqs == 0 || p.q_rows == 0 || a->max_q == 0) return MOE_OK;
  if ((st = moe::check_paged_arrays(p)) != MOE_OK || (st = moe::check_paged_heads(a->q)) != MOE_OK) return st;
  if ((p.n_pages > 0 && !a->bounds) || !a->blocks || !ws) return MOE_EINVAL;
  if (!moe::paged_aligned16(a->bounds) || (reinterpret_cast<uintptr_t>(ws) & 255)) return MOE_EALIGN;
  if (ws_bytes < moe::ws_bytes_for(*a)) return MOE_EWORKSPACE;
  moe::SelectArgs k;
  k.s = moe::paged_seqs(p);
  k.q = a->q, k.bounds = a->bounds, k.blocks = a->blocks, k.keys = static_cast<uint64_t*>(ws);
  k.q_heads = p.q_heads, k.kv_heads = p.kv_heads, k.group = p.q_heads / p.kv_heads;
  k.max_q = a->max_q, k.max_kv = std::min(a->max_kv, k.s.capacity);
  k.n_blocks = a->n_blocks, k.first = a->first, k.last = a->last;
  k.row0 = 0, k.rows = p.q_rows, k.stride = moe::score_stride(*a);
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const int step = moe::batch_rows(*a);
  switch (p.head_dim) {
    case 64: moe::launch<8>(k, step, s); break;
    case 128: moe::launch<16>(k, step, s); break;
    default: moe::launch<32>(k, step, s); break;
  }
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_EHIP;
}

}  // extern "C"
