// The blocks of a paged cache that each token's queries promise to need
// (include/moe_paged.h, moe_select_blocks).
//
// For a query element x and bounds low <= k <= high, x k is at most max(x low, x high)
// = max(x, 0) high + min(x, 0) low.  Summed over the query heads of a key head, the
// score of a page is Q+ . high + Q- . low with Q+ = sum max(x, 0), Q- = sum min(x, 0): one
// dot product of 2 D columns per token, key head and page, whatever the group.
//
// Two tokens' scores that differ in the last bits of float32 must still be ordered as
// defined, so everything is summed in float64 (products of bf16 values are exact there).  The vector
// unit multiplies and adds it at the rate of single float32 values (76 TFLOP/s both, measured), the
// matrix cores at half of theirs (68 against 128 TFLOP/s, 4096^3).
//
// Scores are kept as integers that order as they do.  A wave holds those of a token and
// key head in registers, finds the n-th largest by bisecting its bits with counts over
// the wave, and writes the blocks at or above it in order, the first ones of those that are
// equal to it.  For a few tokens of many sequences one block scores a token's pages into LDS and
// chooses (one launch, the pages read once); with many pages for few tokens the scores go
// through the workspace, so that more of the card reads; for chunks of a sequence tiles of
// 16 tokens x 16 pages go through the float64 matrix cores, so a page is read once per 16 tokens.
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
__device__ __forceinline__ RowWork row_work(const SelectArgs& a, int seq, int row) {
  const PagedRange r = paged_range(a.s.cu_q, a.s.kv_len, seq, a.s.q_rows, a.s.capacity, 0, 0, a.max_kv, a.s.shift);
  const int pos = row - r.q0;
  RowWork w;
  w.seq = uni(seq);
  w.last = uni(pos < 0 || pos >= min(r.lq, a.max_q) ? -2 : max(last_key(r, pos), -1));
  return w;
}
// The last sequence that begins at or before a row; one row each is the common case.
__device__ __forceinline__ int find_seq(const SelectArgs& a, int row) {
  const int guess = min(row, a.s.n_seqs - 1);
  if (a.s.cu_q[guess] <= row && (guess + 1 == a.s.n_seqs || a.s.cu_q[guess + 1] > row)) return guess;
  int lo = 0, hi = a.s.n_seqs;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.s.cu_q[mid] <= row) lo = mid; else hi = mid;
  }
  return lo;
}
__device__ __forceinline__ RowWork find_row(const SelectArgs& a, int row) {
  return row_work(a, find_seq(a, row), row);
}

__device__ __forceinline__ void unpack8(u32x4 w, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// The sum over a group of L = 8, 16 or 32 lanes, in every lane of it.
template <int CTRL>
__device__ __forceinline__ double dpp_add(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const int lo = __builtin_amdgcn_mov_dpp(static_cast<int>(b), CTRL, 15, 15, true);
  const int hi = __builtin_amdgcn_mov_dpp(static_cast<int>(b >> 32), CTRL, 15, 15, true);
  return v + __builtin_bit_cast(double, static_cast<uint64_t>(static_cast<uint32_t>(hi)) << 32 | static_cast<uint32_t>(lo));
}
template <int L>
__device__ __forceinline__ double group_sum(double v) {
  v = dpp_add<0xb1>(v);   // quad_perm 1 0 3 2
  v = dpp_add<0x4e>(v);   // quad_perm 2 3 0 1
  v = dpp_add<0x141>(v);  // mirror within 8
  if (L >= 16) v = dpp_add<0x140>(v);  // mirror within 16
  if (L >= 32) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = static_cast<uint32_t>(b), hi = static_cast<uint32_t>(b >> 32);
    const auto l = __builtin_amdgcn_permlane16_swap(lo, lo, false, false);
    const auto h = __builtin_amdgcn_permlane16_swap(hi, hi, false, false);
    v = __builtin_bit_cast(double, static_cast<uint64_t>(h[0]) << 32 | l[0]) +
        __builtin_bit_cast(double, static_cast<uint64_t>(h[1]) << 32 | l[1]);
  }
  return v;
}

// ---------------------------------------------------------------- scores of one token
// Q+ and Q- of eight columns a lane.
struct Sides {
  double up[8], down[8];
};
__device__ __forceinline__ Sides query_sides(const uint16_t* q, int64_t head_stride, int group) {
  Sides s;
#pragma unroll
  for (int j = 0; j < 8; ++j) s.up[j] = s.down[j] = 0.0;
#pragma unroll 4
  for (int g = 0; g < group; ++g) {
    float x[8];
    unpack8(ld16(q + g * head_stride), x);
#pragma unroll
    for (int j = 0; j < 8; ++j) {  // NaN goes up
      const double d = static_cast<double>(x[j]);
      const bool below = x[j] < 0.f;
      s.up[j] += below ? 0.0 : d;
      s.down[j] += below ? d : 0.0;
    }
  }
  return s;
}

// Pages begin .. end - 1 of one row and key head, by THREADS threads: a group of L = D / 8
// lanes takes a page at a time, eight columns a lane, four pages in flight.  put(b, key).
template <int L, int THREADS, typename Put>
__device__ __forceinline__ void score_pages(const SelectArgs& a, const RowWork& w, int row, int head, int begin, int end,
                                            Put put) {
  constexpr int D = 8 * L, kGroups = THREADS / L, kEach = 4, kStep = kEach * kGroups;
  const int grp = threadIdx.x / L, e0 = 8 * (threadIdx.x % L);
  const int32_t* table = a.s.table + w.seq * a.s.table_stride;
  const int64_t to_high = static_cast<int64_t>(a.kv_heads) * D;
  int page[kEach];
  u32x4 low[kEach], high[kEach];
  auto pages = [&](int b0) {
#pragma unroll
    for (int i = 0; i < kEach; ++i) page[i] = table[min(b0 + i * kGroups + grp, end - 1)];
  };
  bool ok[kEach];
  auto load = [&] {
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      ok[i] = page[i] >= 0 && page[i] < a.s.n_pages;
      const uint16_t* p = a.bounds + (static_cast<int64_t>(ok[i] ? page[i] : 0) * 2 * a.kv_heads + head) * D + e0;
      low[i] = ld16(p);
      high[i] = ld16(p + to_high);
    }
  };
  pages(begin);
  load();
  if (begin + kStep < end) pages(begin + kStep);
  const Sides s =
      query_sides(a.q.base + row * a.q.row_stride + head * a.group * a.q.head_stride + e0, a.q.head_stride, a.group);
  for (int b0 = begin; b0 < end; b0 += kStep) {
    u32x4 l4[kEach], h4[kEach];
    bool there[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) l4[i] = low[i], h4[i] = high[i], there[i] = ok[i];
    if (b0 + kStep < end) {
      load();
      if (b0 + 2 * kStep < end) pages(b0 + 2 * kStep);
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      float l[8], h[8];
      unpack8(l4[i], l);
      unpack8(h4[i], h);
      double sum = 0.0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sum = __builtin_fma(s.up[j], static_cast<double>(h[j]), sum);
        sum = __builtin_fma(s.down[j], static_cast<double>(l[j]), sum);
      }
      sum = group_sum<L>(sum);
      const int b = b0 + i * kGroups + grp;
      if (threadIdx.x % L == 0 && b < end) put(b, there[i] ? order_key(sum) : kNone);
    }
  }
}

// ---------------------------------------------------------------- choice
// The n_blocks largest of 64 * PER keys of a wave, key j of a lane block base + 64 j + lane; more
// than n_blocks of them are visible.  `total` sums a count over the waves that share the keys.
// Counts are made per lane and summed over the wave once.
template <int CTRL>
__device__ __forceinline__ int dpp_add_int(int v) {
  return v + __builtin_amdgcn_mov_dpp(v, CTRL, 15, 15, true);
}
__device__ __forceinline__ int wave_sum(int v) {
  v = dpp_add_int<0xb1>(v);   // quad_perm 1 0 3 2
  v = dpp_add_int<0x4e>(v);   // quad_perm 2 3 0 1
  v = dpp_add_int<0x141>(v);  // mirror within 8
  v = dpp_add_int<0x140>(v);  // mirror within 16
  const auto r = __builtin_amdgcn_permlane16_swap(static_cast<unsigned>(v), static_cast<unsigned>(v), false, false);
  const unsigned half = r[0] + r[1];
  const auto t = __builtin_amdgcn_permlane32_swap(half, half, false, false);
  return uni(static_cast<int>(t[0] + t[1]));
}

template <int PER, typename Total, typename Range>
__device__ __forceinline__ uint64_t nth_largest(const uint64_t (&key)[PER], int n_blocks, Total total, Range range) {
  auto count_high = [&](uint32_t from) {
    int c = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) c += static_cast<uint32_t>(key[j] >> 32) >= from;
    return total(wave_sum(c));
  };
  auto count = [&](uint64_t from) {
    int c = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) c += key[j] >= from;
    return total(wave_sum(c));
  };
  // The bits that the scores' upper halves have in common need no counts.  kAlways and
  // kHidden are no scores.
  uint32_t least = ~0u, most = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    if (key[j] == kHidden || key[j] == kAlways) continue;
    least = min(least, static_cast<uint32_t>(key[j] >> 32));
    most = max(most, static_cast<uint32_t>(key[j] >> 32));
  }
  range(least, most);
  if (most < least) return kAlways;  // the blocks that are always taken are all that are wanted, or there
  // The largest t with at least n_blocks keys from t on, its upper half first; one with
  // exactly n_blocks ends the search.
  const int same = most == least ? 32 : __clz(most ^ least);
  uint32_t high = same == 0 ? 0 : most >> (32 - same) << (32 - same);
  for (int bit = 31 - same; bit >= 0; --bit) {
    const uint32_t c = high | 1u << bit;
    const int m = count_high(c);
    if (m >= n_blocks) high = c;
    if (m == n_blocks) return static_cast<uint64_t>(high) << 32;
  }
  uint64_t t = static_cast<uint64_t>(high) << 32;
  for (int bit = 31; bit >= 0; --bit) {
    const uint64_t c = t | uint64_t{1} << bit;
    const int m = count(c);
    if (m >= n_blocks) t = c;
    if (m == n_blocks) break;
  }
  return t;
}

__device__ __forceinline__ void wave_range(uint32_t& least, uint32_t& most) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    least = min(least, static_cast<uint32_t>(__shfl_xor(static_cast<int>(least), off, 64)));
    most = max(most, static_cast<uint32_t>(__shfl_xor(static_cast<int>(most), off, 64)));
  }
  least = static_cast<uint32_t>(uni(static_cast<int>(least)));
  most = static_cast<uint32_t>(uni(static_cast<int>(most)));
}

// Writes the blocks above t, and the first of those equal to t that are still wanted;
// at: place of the wave's first, seen: equal ones before the wave.
template <int PER>
__device__ __forceinline__ void write_blocks(const uint64_t (&key)[PER], uint64_t t, int base, int at, int seen, int want,
                                             int32_t* out) {
  const int lane = threadIdx.x & 63;
  const uint64_t below = (uint64_t{1} << lane) - 1;
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

// One wave, all keys.
template <int PER>
__device__ __forceinline__ void choose(const uint64_t (&key)[PER], int n_blocks, int32_t* out) {
  const uint64_t t = nth_largest(key, n_blocks, [](int c) { return c; }, wave_range);
  int above = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) above += __popcll(__ballot(key[j] > t));
  write_blocks(key, t, 0, 0, 0, n_blocks - uni(above), out);
}

// Key of block b of n from where its score is kept.
__device__ __forceinline__ uint64_t kept_key(const SelectArgs& a, const uint64_t* keys, int b, int n) {
  if (b >= n) return kHidden;
  return b < a.first || b >= n - a.last ? kAlways : keys[b];
}

// No more blocks than are wanted: all of them.
__device__ __forceinline__ void take_all(int n, int n_blocks, int thread, int threads, int32_t* out) {
  for (int i = thread; i < n_blocks; i += threads) out[i] = i < n ? i : -1;
}

__device__ __forceinline__ int32_t* out_row(const SelectArgs& a, int row, int head) {
  return a.blocks + (static_cast<int64_t>(row) * a.kv_heads + head) * a.n_blocks;
}

// ---------------------------------------------------------------- a token in a block
// Bound by the vector unit: eight columns of a page are 8 conversions and 8 FMAs of float64 for each bound.  64 tokens of
// 32 heads of 128 over 8, 512 pages of 64: 24 us for 67 MB (13 at the copy rate), vector pipes busy half of the
// time; scored by several blocks and chosen by a second launch 26.
constexpr int kFusedThreads = 512;

template <int L, int PER>
__global__ __launch_bounds__(kFusedThreads, 2) void token_kernel(SelectArgs a) {
  __shared__ uint64_t s_key[64 * PER];
  const int head = blockIdx.x % a.kv_heads, row = blockIdx.x / a.kv_heads;
  const RowWork w = find_row(a, row);
  if (w.last == -2) return;
  const int n = (w.last >> a.s.shift) + 1;
  int32_t* out = out_row(a, row, head);
  if (n <= a.n_blocks) return take_all(n, a.n_blocks, threadIdx.x, kFusedThreads, out);
  score_pages<L, kFusedThreads>(a, w, row, head, 0, n, [&](int b, uint64_t key) { s_key[b] = key; });
  __syncthreads();
  if (threadIdx.x >= 64) return;
  uint64_t key[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) key[j] = kept_key(a, s_key, 64 * j + static_cast<int>(threadIdx.x), n);
  choose(key, a.n_blocks, out);
}

// ---------------------------------------------------------------- a token over many blocks
constexpr int kPages = 128;  // of a block

template <int L>
__global__ __launch_bounds__(256) void score_kernel(SelectArgs a) {
  const int item = blockIdx.y, head = item % a.kv_heads, row = a.row0 + item / a.kv_heads;
  const RowWork w = find_row(a, row);
  const int n = (w.last >> a.s.shift) + 1;  // blocks that the row sees (last = -2: 0)
  const int b0 = blockIdx.x * kPages;
  if (n <= a.n_blocks || b0 >= n) return;  // all of them are taken
  uint64_t* out = a.keys + static_cast<int64_t>(item) * a.stride;
  score_pages<L, 256>(a, w, row, head, b0, min(n, b0 + kPages), [&](int b, uint64_t key) { out[b] = key; });
}

// ---------------------------------------------------------------- tiles of tokens
// 16 rows (of q, from a multiple of 16 on) x 16 pages of a key head per matrix product of
// float64: lane l gives Q+ or Q- of row l % 16 and the bound of page l % 16, in four columns
// l / 16 at a time, and gets rows l / 16 + 4 r of page l % 16.  The order of the columns is free: lane l
// takes eight neighbouring ones, 32 c + 8 (l / 16) + e, as they are loaded.  Q+ and Q- of
// the rows are made once by the block and kept in LDS; the waves take 16 pages in turn.
// 1021 tokens of 16 heads of 128 over 2, 1024 pages: 40 us with the choice, 16 at the rate of a large float64
// product (28 for the scores, matrix pipes busy 38 %, making Q+ and Q- is 12 of them; 12 for the choice); one token at a time 281.
typedef double f64x4 __attribute__((ext_vector_type(4)));
constexpr int kTileRows = 16, kTilePages = 256;

template <int L>
__global__ __launch_bounds__(256) void tile_kernel(SelectArgs a) {
  constexpr int D = 8 * L, kChunks = D / 32;
  __shared__ double s_q[kChunks * 16 * 64];
  const int head = blockIdx.y % a.kv_heads, row0 = a.row0 + kTileRows * (blockIdx.y / a.kv_heads);
  const int rows = min(kTileRows, a.row0 + a.rows - row0);
  const int wave = uni(threadIdx.x >> 6), lane = threadIdx.x & 63, col = lane & 15, kq = lane >> 4;
  // the sequences that rows of the tile belong to
  const int seq0 = find_seq(a, row0), seq1 = find_seq(a, row0 + rows - 1);
  bool work = false;
  for (int seq = seq0; seq <= seq1 && !work; ++seq) {
    const PagedRange r = paged_range(a.s.cu_q, a.s.kv_len, seq, a.s.q_rows, a.s.capacity, 0, 0, a.max_kv, a.s.shift);
    const int past = min(row0 + rows, r.q0 + min(r.lq, a.max_q));
    const int n = past > max(row0, r.q0) ? (max(last_key(r, past - 1 - r.q0), -1) >> a.s.shift) + 1 : 0;
    work = n > a.n_blocks && static_cast<int>(blockIdx.x) * kTilePages < n;
  }
  if (!work) return;
  const uint16_t* q = a.q.base + (row0 + min(col, rows - 1)) * a.q.row_stride + head * a.group * a.q.head_stride + 8 * kq;
  for (int c = wave; c < kChunks; c += 4) {
    const Sides s = query_sides(q + 32 * c, a.q.head_stride, a.group);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      s_q[(16 * c + e) * 64 + lane] = s.up[e];
      s_q[(16 * c + 8 + e) * 64 + lane] = s.down[e];
    }
  }
  __syncthreads();
  const int64_t to_high = static_cast<int64_t>(a.kv_heads) * D;
  for (int seq = seq0; seq <= seq1; ++seq) {
    const PagedRange r = paged_range(a.s.cu_q, a.s.kv_len, seq, a.s.q_rows, a.s.capacity, 0, 0, a.max_kv, a.s.shift);
    const int from = uni(max(row0, r.q0)), past = uni(min(row0 + rows, r.q0 + min(r.lq, a.max_q)));
    if (past <= from) continue;
    const int n = uni((max(last_key(r, past - 1 - r.q0), -1) >> a.s.shift) + 1);  // the last row sees the most
    const int end = min(n, (static_cast<int>(blockIdx.x) + 1) * kTilePages);
    const int32_t* table = a.s.table + seq * a.s.table_stride;
    // the bounds of a wave's next pages are loaded while these are used, their numbers one step before
    int page = 0;
    bool ok = false;
    u32x4 low[kChunks], high[kChunks];
    auto number = [&](int b) { return table[min(b, n - 1)]; };
    auto load = [&] {
      ok = page >= 0 && page < a.s.n_pages;
      const uint16_t* p = a.bounds + (static_cast<int64_t>(ok ? page : 0) * 2 * a.kv_heads + head) * D + 8 * kq;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) low[c] = ld16(p + 32 * c), high[c] = ld16(p + to_high + 32 * c);
    };
    int b0 = blockIdx.x * kTilePages + 16 * wave;
    if (b0 < end) {
      page = number(b0 + col);
      load();
      page = number(b0 + 64 + col);
    }
    for (; b0 < end; b0 += 64) {
      const int b = b0 + col;
      const bool there = ok;
      u32x4 l4[kChunks], h4[kChunks];
#pragma unroll
      for (int c = 0; c < kChunks; ++c) l4[c] = low[c], h4[c] = high[c];
      if (b0 + 64 < end) {
        load();
        page = number(b + 128);
      }
      f64x4 up = {0, 0, 0, 0}, down = {0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        float l[8], h[8];
        unpack8(l4[c], l);
        unpack8(h4[c], h);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          up = __builtin_amdgcn_mfma_f64_16x16x4f64(s_q[(16 * c + e) * 64 + lane], static_cast<double>(h[e]), up, 0, 0, 0);
          down = __builtin_amdgcn_mfma_f64_16x16x4f64(s_q[(16 * c + 8 + e) * 64 + lane], static_cast<double>(l[e]), down, 0,
                                                      0, 0);
        }
      }
      if (b >= n) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = row0 + kq + 4 * i;
        if (row < from || row >= past) continue;
        const int64_t item = static_cast<int64_t>(row - a.row0) * a.kv_heads + head;
        a.keys[item * a.stride + b] = there ? order_key(up[i] + down[i]) : kNone;
      }
    }
  }
}

// ---------------------------------------------------------------- choice from the workspace
// WAVES waves hold 64 * PER scores each, wave w those from 64 * PER * w on.  Where a token
// and head has one wave, four of them stand in a workgroup.  Bound by the counts'
// vector work: two bits at a time, three thresholds in half as many counts, took longer (1021 tokens of 1024 pages
// 42.9 us for the call against 42.0, one of 16384 pages 44.0 against 39.9).
template <int WAVES, int PER>
__global__ __launch_bounds__(WAVES == 1 ? 256 : 64 * WAVES) void choose_kernel(SelectArgs a) {
  __shared__ int s_count[2][WAVES];
  __shared__ uint32_t s_range[2][WAVES];
  const int lane = threadIdx.x & 63;
  const int wave = WAVES == 1 ? 0 : uni(threadIdx.x >> 6);
  const int item = WAVES == 1 ? uni(blockIdx.x * 4 + (threadIdx.x >> 6)) : blockIdx.x;
  if (item >= a.rows * a.kv_heads) return;
  const int head = item % a.kv_heads, row = a.row0 + item / a.kv_heads;
  const RowWork w = find_row(a, row);
  if (w.last == -2) return;
  const int n = (w.last >> a.s.shift) + 1;
  int32_t* out = out_row(a, row, head);
  if (n <= a.n_blocks) return take_all(n, a.n_blocks, threadIdx.x & (64 * WAVES - 1), 64 * WAVES, out);
  const uint64_t* keys = a.keys + static_cast<int64_t>(item) * a.stride;
  const int base = 64 * PER * wave;
  uint64_t key[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) key[j] = kept_key(a, keys, base + 64 * j + lane, n);
  if (WAVES == 1) return choose(key, a.n_blocks, out);
  int parity = 0;
  const uint64_t t = nth_largest(key, a.n_blocks, [&](int c) {
    if (lane == 0) s_count[parity][wave] = c;
    __syncthreads();
    int sum = 0;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) sum += s_count[parity][i];
    parity ^= 1;  // the next count goes to the other half, so one barrier each is enough
    return uni(sum);
  }, [&](uint32_t& least, uint32_t& most) {
    wave_range(least, most);
    if (lane == 0) s_range[0][wave] = least, s_range[1][wave] = most;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < WAVES; ++i) least = min(least, s_range[0][i]), most = max(most, s_range[1][i]);
    least = static_cast<uint32_t>(uni(static_cast<int>(least)));
    most = static_cast<uint32_t>(uni(static_cast<int>(most)));
  });
  // keys above t are all taken; of those equal to t the first ones
  int above = 0, equal = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    above += __popcll(__ballot(key[j] > t));
    equal += __popcll(__ballot(key[j] == t));
  }
  __syncthreads();
  if (lane == 0) s_count[0][wave] = above, s_count[1][wave] = equal;
  __syncthreads();
  int above_before = 0, equal_before = 0, above_all = 0;
#pragma unroll
  for (int i = 0; i < WAVES; ++i) {
    if (i < wave) above_before += s_count[0][i], equal_before += s_count[1][i];
    above_all += s_count[0][i];
  }
  const int want = a.n_blocks - uni(above_all);  // of the equal ones
  write_blocks(key, t, base, uni(above_before) + min(uni(equal_before), want), uni(equal_before), want, out);
}

// ---------------------------------------------------------------- host
constexpr int kMaxPages = 32768;
constexpr size_t kBatchBytes = size_t{1} << 28;  // of scores at a time

enum Way { kTokenBlock, kTokenSplit, kTiles };

inline int score_stride(const moe_select& d) {
  const int pages = (d.max_kv + d.p.page_size - 1) / d.p.page_size;
  return std::max((pages + 7) / 8 * 8, 8);
}
// How the scores are made, from the shape fields, as the workspace.  32 query heads of 128 over
// 8, pages of 64 (us: one block a token and head; several and the workspace; tiles):
//   64 rows of one sequence, 512 pages 23.4, 26.4, 23.1; 128 rows 40.3, 42.7, 24.1; four sequences of
//   32 rows 26.9, 33.8, 34.1, of 64 rows 47.3, 57.5, 35.2; 16 heads of 64 over 2, 256 pages, 128 rows 10.6,
//   12.6, 16.8, 512 rows 26.8, 24.7, 17.9: tiles from 64 rows a sequence and 512 rows x heads on;
//   single tokens, 4 of 256 pages 10.1, 10.6; 4 of 512 13.1, 10.9; 16 of 512 14.9, 15.0; 16 of 1024 26.6, 23.1;
//   64 of 1024 46.8, 57.4; 16 of 2048 38.8, 34.9; 64 of 2048 77.4, 106.6: several blocks each where
//   there are fewer rows x heads than a quarter of the pages, and more than 256 of those.
inline Way pick_way(const moe_select& d) {
  const int64_t items = static_cast<int64_t>(d.p.q_rows) * d.p.kv_heads;
  if (d.max_q >= 64 && d.p.q_rows >= 64 * static_cast<int64_t>(d.p.n_seqs) && items >= 512) return kTiles;
  const int pages = score_stride(d);
  return pages <= 256 || (pages <= 2048 && items >= pages / 4) ? kTokenBlock : kTokenSplit;
}
// Rows of a launch: their scores fit kBatchBytes, and the grid 65535 blocks along y; whole tiles.
inline int batch_rows(const moe_select& d) {
  const size_t row = static_cast<size_t>(d.p.kv_heads) * score_stride(d) * 8;
  const size_t rows = std::min(std::max(kBatchBytes / row, size_t{1}), static_cast<size_t>(65535 / d.p.kv_heads));
  const size_t whole = rows >= kTileRows ? rows / kTileRows * kTileRows : rows;
  return static_cast<int>(std::min(whole, static_cast<size_t>(std::max(d.p.q_rows, 1))));
}
inline size_t ws_bytes_for(const moe_select& d) {
  if (pick_way(d) == kTokenBlock) return 0;
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
  if (static_cast<int64_t>(a->p.q_rows) * a->p.kv_heads >= (1 << 23)) return MOE_ESHAPE;  // 2^32 threads
  if (a->first > a->n_blocks || a->last > a->n_blocks - a->first) return MOE_EINVAL;
  return MOE_OK;
}

template <int L>
void launch(SelectArgs a, Way way, int step, hipStream_t s) {
  const int rows = a.rows, pages = a.stride;
  if (way == kTokenBlock) {
    const unsigned blocks = static_cast<unsigned>(rows) * a.kv_heads;
    if (pages <= 512)
      token_kernel<L, 8><<<blocks, kFusedThreads, 0, s>>>(a);
    else
      token_kernel<L, 32><<<blocks, kFusedThreads, 0, s>>>(a);
    return;
  }
  for (int r = 0; r < rows; r += step) {
    a.row0 = r;
    a.rows = std::min(step, rows - r);
    const unsigned items = static_cast<unsigned>(a.rows) * a.kv_heads;
    const unsigned tiles = static_cast<unsigned>((a.rows + kTileRows - 1) / kTileRows) * a.kv_heads;
    if (way == kTiles)
      tile_kernel<L><<<dim3((pages + kTilePages - 1) / kTilePages, tiles), 256, 0, s>>>(a);
    else
      score_kernel<L><<<dim3((pages + kPages - 1) / kPages, items), 256, 0, s>>>(a);
    if (pages <= 512)
      choose_kernel<1, 8><<<(items + 3) / 4, 256, 0, s>>>(a);
    else if (pages <= 1024)
      choose_kernel<1, 16><<<(items + 3) / 4, 256, 0, s>>>(a);
    else if (pages <= 2048)
      choose_kernel<1, 32><<<(items + 3) / 4, 256, 0, s>>>(a);
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
  if ((p.n_pages > 0 && !a->bounds) || !a->blocks) return MOE_EINVAL;
  if (!moe::paged_aligned16(a->bounds)) return MOE_EALIGN;
  const size_t need = moe::ws_bytes_for(*a);
  if (need) {
    if (!ws) return MOE_EINVAL;
    if (reinterpret_cast<uintptr_t>(ws) & 255) return MOE_EALIGN;
    if (ws_bytes < need) return MOE_EWORKSPACE;
  }
  moe::SelectArgs k;
  k.s = moe::paged_seqs(p);
  k.q = a->q, k.bounds = a->bounds, k.blocks = a->blocks, k.keys = static_cast<uint64_t*>(ws);
  k.q_heads = p.q_heads, k.kv_heads = p.kv_heads, k.group = p.q_heads / p.kv_heads;
  k.max_q = a->max_q, k.max_kv = std::min(a->max_kv, k.s.capacity);
  k.n_blocks = a->n_blocks, k.first = a->first, k.last = a->last;
  k.row0 = 0, k.rows = p.q_rows, k.stride = moe::score_stride(*a);
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const int step = moe::batch_rows(*a);
  const moe::Way way = moe::pick_way(*a);
  switch (p.head_dim) {
    case 64: moe::launch<8>(k, way, step, s); break;
    case 128: moe::launch<16>(k, way, step, s); break;
    default: moe::launch<32>(k, way, step, s); break;
  }
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_EHIP;
}

}  // extern "C"
