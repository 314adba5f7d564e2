// Softmax attention over a paged cache (include/moe_paged.h, moe_paged_attention).
//
// Rows, tiles and their arithmetic are those of the attention over a contiguous cache
// (attention_core.h): the query heads of a key head are folded into rows, row r
// is query r / G, head r % G.  What differs is where keys come from.  A DMA instruction
// fills at most 16 rows of a tile, and a page holds a multiple of 16 keys, so every
// instruction has one page and the tile's keys need one lookup per 16 ("half" below: 16 keys).
//
// Two kernels write shares of rows, a third joins them:
//  token  32 rows of a sequence (its new tokens' heads, few of them), the waves split
//         the keys; the sequence's own keys, or those of listed blocks
//  rows   128 rows of a sequence over its own keys, or over listed blocks; in the same launch
//         128 rows of a whole group over the prefix that its sequences share
// With a shared prefix a row has shares of both: slots 0 .. prefix_splits - 1 are the
// prefix's, the others the sequence's own.  Every slot of a row is written, if only
// with a sum of 0, so the join needs to know nothing about groups or lists.
//
// A sequence alone costs what it does over a contiguous cache (us, pages of 64; contiguous): 64 tokens over up to
// 8192 keys 216, 212; 4 over 1024 10.9, 10.5; one over 65536 57 to 60, 57 to 61; a prompt of 4096 147 to 152, 146 to
// 151; with pages of 16, a lookup per 16 keys, 219 and 142 to 147.  Heads of 256 lose more, 25 and 22 for one token over
// 32768 keys, 202 and 177 for a prompt of 4096: the addresses are made anew for every tile, and some 50 registers
// still spill (the contiguous kernel's do not).
#include <math.h>

#include <algorithm>

#include "attention_core.h"
#include "paged_internal.h"

namespace moe {

namespace {

struct PagedArgs {
  PagedSeqs s;
  moe_heads q, out;
  moe_pages k, v;
  const int32_t *cu_group, *prefix_len, *blocks;
  float* lse;
  float* part_o;    // [slots, q_rows, q_heads, D]
  float2* part_ml;  // [slots, q_rows, q_heads]: maximum, sum
  int q_heads, kv_heads, group, max_q, max_kv, n_groups, max_prefix, n_blocks;
  int chunk, splits; // own keys of a split (listed blocks: the fewest), and how many there are at most
  int prefix_chunk;  // prefix keys of a split
  int prefix_splits, slots;
  int tiles, prefix_tiles, units, prefix_units;  // of the rows kernel: row tiles, and (tile, split) pairs
  int token;         // the token kernel did the own keys: every sequence is one tile of it
  int tile_rows;     // rows of a tile of the kernel that did the own keys
  int join_rows;     // rows of a block of the join
  float scale, c;    // c = scale * log2(e)
  __host__ __device__ bool every_slot() const { return n_groups > 0 || n_blocks > 0; }
};

// ---------------------------------------------------------------- work
// A lane's group of the first 64, loaded before anything is known.
struct LaneGroup {
  GroupRange range;
  int prefix;
};
__device__ __forceinline__ LaneGroup lane_group(const PagedArgs& a, int base) {
  const int g = min(base + static_cast<int>(threadIdx.x & 63), a.n_groups - 1);
  return LaneGroup{group_range(a.cu_group, g, a.s.n_seqs), a.prefix_len[g]};
}
// The prefix length that sequence b's group names (0 without one): the last group that
// begins at or before b.  For a whole wave, 64 groups at a time; mine: the first of them.
__device__ __forceinline__ int prefix_of(const PagedArgs& a, int b, LaneGroup mine) {
  for (int base = 0; base < a.n_groups; base += 64) {
    if (base > 0) mine = lane_group(a, base);
    const uint64_t holds = __ballot(b >= mine.range.first && b < mine.range.past);
    if (holds) return lane_value(mine.prefix, 63 - __clzll(static_cast<long long>(holds)));
  }
  return 0;
}

__device__ __forceinline__ PagedRange sequence(const PagedArgs& a, int b, int prefix) {
  return paged_range(a.s.cu_q, a.s.kv_len, b, a.s.q_rows, a.s.capacity, prefix, a.max_prefix, a.max_kv, a.s.shift);
}

struct PagedTile : PagedRange {
  int seq;  // whose row of the table names the pages
  int tile, tiles;
};

// Tile t over all sequences (each sequence's tiles in a row), 64 of them at a time.
__device__ bool find_tile(const PagedArgs& a, int t, int rows, PagedTile& w) {
  const int lane = threadIdx.x & 63;
  for (int base = 0; base < a.s.n_seqs; base += 64) {
    const bool there = base + lane < a.s.n_seqs;
    const PagedRange r = sequence(a, there ? base + lane : base, 0);
    const int nt = there ? (min(r.lq, a.max_q) * a.group + rows - 1) / rows : 0;
    const int incl = wave_prefix(nt);
    const uint64_t past = __ballot(incl > t);
    if (past) {
      const int src = __ffsll(static_cast<unsigned long long>(past)) - 1;
      w.seq = base + src;
      w.q0 = lane_value(r.q0, src), w.lq = lane_value(r.lq, src), w.diag = lane_value(r.diag, src);
      w.own = lane_value(r.own, src), w.end = lane_value(r.end, src);
      w.tiles = lane_value(nt, src);
      w.tile = t - (lane_value(incl, src) - w.tiles);
      return true;
    }
    t -= lane_value(incl, 63);
  }
  return false;
}

// Tile t over all groups: 128-row tiles of the rows of a group's sequences, in groups
// that share something.
__device__ bool find_group_tile(const PagedArgs& a, int t, int rows, PagedTile& w, GroupRange& g) {
  const int lane = threadIdx.x & 63;
  for (int base = 0; base < a.n_groups; base += 64) {
    int nt = 0, q0 = 0, lq = 0, keys = 0;
    GroupRange x = {0, 0};
    if (base + lane < a.n_groups) {
      x = group_range(a.cu_group, base + lane, a.s.n_seqs);
      keys = shared_keys(a.prefix_len[base + lane], a.max_prefix, a.s.shift);
      q0 = min(max(a.s.cu_q[x.first], 0), a.s.q_rows);
      lq = min(max(a.s.cu_q[x.past], q0), a.s.q_rows) - q0;
      nt = keys > 0 ? (lq * a.group + rows - 1) / rows : 0;
    }
    const int incl = wave_prefix(nt);
    const uint64_t past = __ballot(incl > t);
    if (past) {
      const int src = __ffsll(static_cast<unsigned long long>(past)) - 1;
      g.first = lane_value(x.first, src), g.past = lane_value(x.past, src);
      w.seq = g.first;
      w.q0 = lane_value(q0, src), w.lq = lane_value(lq, src);
      w.own = 0, w.end = lane_value(keys, src), w.diag = 0;
      w.tiles = lane_value(nt, src);
      w.tile = t - (lane_value(incl, src) - w.tiles);
      return true;
    }
    t -= lane_value(incl, 63);
  }
  return false;
}

// A lane's row: the query row and head it reads and writes, and the last key it sees.
struct LaneRow {
  int64_t q_row;
  int head, limit;
  bool valid;
};
__device__ __forceinline__ LaneRow lane_row(const PagedArgs& a, const PagedTile& w, int kv_head, int r, int n_rows) {
  LaneRow x;
  x.valid = r < n_rows;
  const int rc = min(r, n_rows - 1);
  const int pos = rc / a.group;
  x.q_row = w.q0 + pos;
  x.head = kv_head * a.group + rc - pos * a.group;
  x.limit = last_key(w, pos);
  return x;
}

template <int D>
__device__ __forceinline__ void load_q(const PagedArgs& a, const LaneRow& x, bf16x8 (&q)[D / 16]) {
  const uint16_t* p = a.q.base + x.q_row * a.q.row_stride + x.head * a.q.head_stride + 8 * ((threadIdx.x & 63) >> 5);
#pragma unroll
  for (int i = 0; i < D / 16; ++i) q[i] = __builtin_bit_cast(bf16x8, ld16(p + 16 * i));
}

// Outputs d .. d + 3 of a row from the sums o and l over the maximum m; l is 0 only
// where the row saw no score above -infinity: zeros then, whatever o holds.
__device__ __forceinline__ void store_quad(const PagedArgs& a, int64_t q_row, int head, int d, f32x4 o, float m,
                                           float l) {
  if (l == 0.f) o = f32x4{0.f, 0.f, 0.f, 0.f};
  const float inv = l == 0.f ? 0.f : 1.f / l;
  u32x2 v;
#pragma unroll
  for (int e = 0; e < 2; ++e)
    v[e] = float_to_bf16_bits(o[2 * e] * inv) | static_cast<uint32_t>(float_to_bf16_bits(o[2 * e + 1] * inv)) << 16;
  *reinterpret_cast<u32x2*>(a.out.base + q_row * a.out.row_stride + head * a.out.head_stride + d) = v;
  if (a.lse && d == 0) a.lse[q_row * a.q_heads + head] = l == 0.f ? kNegInf : m * a.scale + logf(l);
}

// A slot's share of a row: the unscaled output, the maximum and the sum.
__device__ __forceinline__ int64_t part_row(const PagedArgs& a, int slot, int64_t q_row, int head) {
  return (static_cast<int64_t>(slot) * a.s.q_rows + q_row) * a.q_heads + head;
}
__device__ __forceinline__ void empty_share(const PagedArgs& a, int slot, int64_t q_row, int head) {
  a.part_ml[part_row(a, slot, q_row, head)] = make_float2(kNegInf, 0.f);
}

// Heads of 256 leave no registers for the LDS addresses (kept, the loops spilled).
template <int D>
constexpr bool kKeep = D < 256;

// A tile whose rows see some of its 16-key halves only, or none: as attend_masked of the
// contiguous kernels, with a limit per half; row(i): the values of half i's first key.
// scan = false: every value of the tile is taken for finite.
template <int D, int NT, typename Row>
__device__ __forceinline__ void attend_halves(const uint8_t* ks, const uint8_t* vs, const bf16x8 (&q)[D / 16],
                                              RowState<D>& st, float c, const Limits<NT>& lim, bool scan,
                                              int64_t row_stride, Row row) {
  const bool dirty = scan && any_not_finite(vs, NT * 32 * 2 * D);
  attend<D, NT, true, kKeep<D>>(ks, vs, q, st, c, lim, dirty);
  if (!dirty) return;
  const int h = (threadIdx.x & 63) >> 5;
  for (int r = 0; r < NT * 32; ++r) {
    int last = lim.at[0];
#pragma unroll
    for (int i = 1; i < 2 * NT; ++i) last = r >= 16 * i ? lim.at[i] : last;
    if (r > last) continue;
    add_not_finite<D>(row(r >> 4) + (r & 15) * row_stride + 4 * h, st);
  }
}

// LDS-DMA: an instruction fills 1 KiB, 512 / D rows; the lane that lands in slot s of
// row r loads the chunk whose slot that is (the XOR is its own inverse, and the same
// for rows 16 apart).  Byte offset for instruction i of a half.
template <int D, bool VALUE>
__device__ __forceinline__ int half_offset(int i, int row_bytes) {
  constexpr int kChunks = D / 8;
  const int lane = threadIdx.x & 63;
  const int r = i * (64 / kChunks) + lane / kChunks, s = lane % kChunks;
  return r * row_bytes + 16 * (VALUE ? v_slot<D>(r, s) : k_slot<D>(r, s));
}

// Whether an output of the wave is not finite.
template <int D>
__device__ __forceinline__ bool not_finite(const RowState<D>& st) {
  float zero = 0.f;  // 0 times what is finite
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) zero = __builtin_fmaf(st.o[i][j], 0.f, zero);
  return __any(zero != 0.f);
}

// Neighbouring keys of one page: 16, or a tile where a page holds whole tiles.
struct Spot {
  int page, key;     // a page that there is, the position of the first key
  uint32_t visible;  // of the rows' tokens: bit (token - the first); 0 where the page is none
};
// A tile's N spots.
template <int N>
struct Spots {
  Spot at[N];
};

__device__ __forceinline__ const uint16_t* spot_base(const moe_pages& p, const Spot& x, int slot_mask, int kv_head) {
  return p.base + x.page * p.page_stride + (x.key & slot_mask) * p.row_stride + kv_head * p.head_stride;
}

// What a lookup brings: used one tile later, so that nothing waits for it.
struct Found {
  int page, key;
  uint32_t tokens;
};
template <int N>
struct FoundAll {
  Found at[N];
};

// The spot at key `key` of the table row, for every token.
__device__ __forceinline__ Found look_up(const PagedArgs& a, ConstInts table, int key) {
  return Found{table[min(key >> a.s.shift, a.s.table_pages - 1)], key, ~0u};
}
__device__ __forceinline__ Spot to_spot(const PagedArgs& a, Found f) {
  const int page = uniform(f.page);
  const bool ok = page >= 0 && page < a.s.n_pages;
  return Spot{ok ? page : 0, uniform(f.key), ok ? static_cast<uint32_t>(uniform(static_cast<int>(f.tokens))) : 0u};
}
template <int N>
__device__ __forceinline__ Spots<N> to_spots(const PagedArgs& a, const FoundAll<N>& f) {
  Spots<N> p;
#pragma unroll
  for (int i = 0; i < N; ++i) p.at[i] = to_spot(a, f.at[i]);
  return p;
}

// Last keys that a row sees in the tile's halves, given the last that it sees at all and
// its token.
template <int NT, int N>
__device__ __forceinline__ Limits<NT> spot_limits(const Spots<N>& p, int limit, int token) {
  constexpr int kEach = 2 * NT / N;  // halves of a spot
  Limits<NT> lim;
#pragma unroll
  for (int i = 0; i < 2 * NT; ++i) {
    const Spot& x = p.at[i / kEach];
    lim.at[i] = x.visible >> token & 1 ? limit - x.key + 16 * (i / kEach * kEach) : -1;
  }
  return lim;
}

// ---------------------------------------------------------------- few rows
constexpr int kRowsT = 32;  // rows of a tile
constexpr int kKeysT = 32;  // keys of a wave's tile
constexpr int kList = 512;  // listed blocks of a split
constexpr int kWords = 1024;  // 32-block words of the marks: blocks per sequence / 32

// The listed blocks of a tile's tokens, each once and ascending, of which the splits
// take equal shares (as many as `least` there are, or less in the last).  An entry is a
// page (-1: none), its block, and for each 32 rows of the tile the tokens that list it,
// from the first of those rows on.
template <int PARTS>
struct ListEntry {
  int page, block;
  uint32_t tokens[PARTS];
};

// Marks are set with integer atomics (their order changes nothing) in LDS, one bit a
// block; a block's place in the list is the number of marks below it.  A thread keeps its
// first kHeld ids and their pages in registers, so a list costs three loads in a row.
// scratch: at least 2 * kWords + 16 ints; r0: the tile's first row, rows: its rows.  Returns
// the number of entries of this split's share (at most kList: the plan sees to it).
template <int THREADS, int PARTS>
__device__ int build_list(const PagedArgs& a, const PagedTile& w, int kv_head, int r0, int rows, int split,
                          ListEntry<PARTS>* list, uint32_t* scratch) {
  constexpr int kPer = kWords / THREADS, kHeld = 4;
  const int tid = threadIdx.x;
  uint32_t* marks = scratch;
  int* below = reinterpret_cast<int*>(scratch + kWords);
  int* wave_sum = reinterpret_cast<int*>(scratch + 2 * kWords);
  const int tok0 = r0 / a.group, n_tok = (r0 + rows - 1) / a.group - tok0 + 1;
  const int total = n_tok * a.n_blocks;
  const int32_t* ids = a.blocks + (static_cast<int64_t>(w.q0 + tok0) * a.kv_heads + kv_head) * a.n_blocks;
  const int64_t to_next = static_cast<int64_t>(a.kv_heads) * a.n_blocks;
  const int32_t* table = a.s.table + w.seq * a.s.table_stride;
  // id i of the tile: a block that its token sees a key of, or -1
  auto load_id = [&](int i) {
    if (i >= total) return -1;
    const int t = i / a.n_blocks;
    const int id = ids[t * to_next + i - t * a.n_blocks];
    return id >= 0 && id < 32 * kWords && id << a.s.shift <= last_key(w, tok0 + t) ? id : -1;
  };
  int id[kHeld], page[kHeld];
#pragma unroll
  for (int j = 0; j < kHeld; ++j) id[j] = load_id(tid + j * THREADS);
#pragma unroll
  for (int i = 0; i < kPer; ++i) marks[tid + i * THREADS] = 0;
  for (int i = tid; i < kList; i += THREADS) {
    list[i].page = -1;
#pragma unroll
    for (int j = 0; j < PARTS; ++j) list[i].tokens[j] = 0;
  }
  __syncthreads();
  auto mark = [&](int i) {
    if (i >= 0) atomicOr(&marks[i >> 5], 1u << (i & 31));
  };
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    mark(id[j]);
    page[j] = id[j] >= 0 ? table[id[j]] : -1;
  }
  for (int i = tid + kHeld * THREADS; i < total; i += THREADS) mark(load_id(i));
  __syncthreads();
  int mine[kPer], local = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    mine[i] = __popc(marks[tid * kPer + i]);
    local += mine[i];
  }
  const int incl = wave_prefix(local);
  if ((tid & 63) == 63) wave_sum[tid >> 6] = incl;
  __syncthreads();
  int run = incl - local, all = 0;
#pragma unroll
  for (int i = 0; i < THREADS / 64; ++i) {
    if (i < (tid >> 6)) run += wave_sum[i];
    all += wave_sum[i];
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    below[tid * kPer + i] = run;
    run += mine[i];
  }
  __syncthreads();
  const int count = min(max((all + a.splits - 1) / a.splits, a.chunk), kList), lo = split * count;
  auto enter = [&](int i, int block, int p) {
    if (block < 0) return;
    const int r = below[block >> 5] + __popc(marks[block >> 5] & ((1u << (block & 31)) - 1)) - lo;
    if (r < 0 || r >= count) return;
    list[r].block = block;  // threads that hold the same block write the same
    if (p < 0 || p >= a.s.n_pages) return;
    list[r].page = p;
    const int t = i / a.n_blocks;
#pragma unroll
    for (int j = 0; j < PARTS; ++j) {
      const int from = (r0 + 32 * j) / a.group - tok0, to = (r0 + 32 * j + 31) / a.group - tok0;
      if (t >= from && t <= to) atomicOr(&list[r].tokens[j], 1u << (t - from));
    }
  };
#pragma unroll
  for (int j = 0; j < kHeld; ++j) enter(tid + j * THREADS, id[j], page[j]);
  for (int i = tid + kHeld * THREADS; i < total; i += THREADS) {
    const int block = load_id(i);
    enter(i, block, block >= 0 ? table[block] : -1);
  }
  __syncthreads();
  return min(max(all - lo, 0), count);
}

// Spot i of a list, of SPAN keys: those at i % (page_size / SPAN) of entry i / (page_size / SPAN).
template <int SPAN, int PARTS>
__device__ __forceinline__ Found list_look_up(const PagedArgs& a, const ListEntry<PARTS>* list, int entries, int i,
                                              int part) {
  const int per = a.s.shift - (SPAN == 16 ? 4 : SPAN == 32 ? 5 : 6);  // log2 of the spots in a page
  const int e = i >> per;
  const ListEntry<PARTS>& entry = list[min(e, entries - 1)];
  return Found{entry.page, (entry.block << a.s.shift) + SPAN * (i & ((1 << per) - 1)), e < entries ? entry.tokens[part] : 0u};
}

// Where the token kernel's keys come from.
enum Keys {
  kTable,      // the table: the sequence's own keys
  kListOne,    // listed blocks, tiles of one token
  kListSeveral // listed blocks, tiles of several tokens, which see different blocks
};

// A block per sequence, key head and split; each wave takes every NW-th tile of 32 keys through two stages of
// its own, so no wave waits for another before the merge.  Bound by HBM where there are many keys (32 tokens over 64
// of 512 pages each, 494 MB: 93 us, 5.3 TB/s), by the latency of a list, a tile and the join where there are few (4
// tokens, 16 pages each: 12.7 us).  A tile's pages are looked up one tile before its loads go out: looked up with them, every
// tile waited for the table (4 tokens over 1024 keys 13.3 against 12.9).
// N: spots of a tile, 1 where a page holds whole tiles.
template <int D, Keys KEYS, int NW, int N>
__global__ __launch_bounds__(64 * NW, 1) void paged_token_kernel(PagedArgs a) {
  constexpr bool LISTED = KEYS != kTable;
  constexpr int kTile = kKeysT * 2 * D;
  constexpr int kSpan = kKeysT / N;           // keys of a spot
  constexpr int kHalfOps = kTile / 2048;      // DMA instructions per 16 keys
  // The stages are variables of their own: the compiler then knows that the
  // DMA in flight into one does not write the other, and does not wait for it.
  __shared__ __attribute__((aligned(1024))) uint8_t smem0[NW][2][kTile];
  __shared__ __attribute__((aligned(1024))) uint8_t smem1[NW][2][kTile];
  __shared__ float s_m[NW][32], s_l[NW][32];
  __shared__ ListEntry<1> s_list[LISTED ? kList : 1];
  static_assert(NW * 32 * D * 4 == sizeof(smem0), "the merge uses a stage");
  static_assert(!LISTED || sizeof(smem0) >= 4 * (2 * kWords + 16), "and so does the list's scratch");
  const int t_block = blockIdx.x / a.kv_heads, split = blockIdx.y;
  // the heads of each sequence and split begin on another XCD
  const int kv_head = (blockIdx.x + t_block + split) % a.kv_heads;
  PagedTile w;
  w.seq = t_block, w.tile = 0, w.tiles = 1;
  const PagedRange range = sequence(a, w.seq, 0);  // no groups here: the keys begin at 0
  w.q0 = uniform(range.q0), w.lq = uniform(range.lq), w.diag = uniform(range.diag);
  w.own = 0, w.end = uniform(range.end);
  const int r0 = 0, n_rows = min(w.lq, a.max_q) * a.group;
  if (n_rows == 0) return;
  const int here = n_rows;  // at most 32
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int tok0 = r0 / a.group, tok1 = (r0 + here - 1) / a.group;
  const LaneRow x = lane_row(a, w, kv_head, r0 + (lane & 31), n_rows);
  const int lim_first = last_key(w, tok0);
  auto empty = [&](int at) {
    if (wave == 0 && lane < here) empty_share(a, at, x.q_row, x.head);
  };

  int n_tiles, kbeg = 0, splits = 1, entries = 0;
  if (LISTED) {
    entries = uniform(build_list<64 * NW>(a, w, kv_head, r0, here, split, s_list,
                                          reinterpret_cast<uint32_t*>(&smem0[0][0][0])));
    n_tiles = ((entries << (a.s.shift - 4)) + 1) / 2;
    if (n_tiles == 0 && a.slots > 1) return empty(split);
  } else {
    const int all = max(last_key(w, tok1) + 1 - w.own, 0);
    splits = (all + a.chunk - 1) / a.chunk;
    if (split >= max(splits, 1)) return;
    kbeg = w.own + split * a.chunk;
    n_tiles = (min(all - split * a.chunk, a.chunk) + kKeysT - 1) / kKeysT;
  }

  bf16x8 q[D / 16];
  load_q<D>(a, x, q);
  const int slot_mask = (1 << a.s.shift) - 1;
  ConstInts table = const_ints(a.s.table + w.seq * a.s.table_stride);
  int koff[kHalfOps], voff[kHalfOps];
#pragma unroll
  for (int i = 0; i < kHalfOps; ++i) {
    koff[i] = half_offset<D, false>(i, static_cast<int>(a.k.row_stride) * 2);
    voff[i] = half_offset<D, true>(i, static_cast<int>(a.v.row_stride) * 2);
  }
  const uint32_t every = tok1 - tok0 == 31 ? ~0u : (2u << (tok1 - tok0)) - 1;
  auto find = [&](int t, int i) -> Found {
    return LISTED ? list_look_up<kSpan>(a, s_list, entries, N * t + i, 0)
                  : look_up(a, table, kbeg + kKeysT * t + kSpan * i);
  };
  auto find_all = [&](int t) {
    FoundAll<N> p;
#pragma unroll
    for (int i = 0; i < N; ++i) p.at[i] = find(t, i);
    return p;
  };
  const int k16 = 32 * static_cast<int>(a.k.row_stride), v16 = 32 * static_cast<int>(a.v.row_stride);  // bytes of 16 rows
  auto issue = [&](uint8_t (&to)[2][kTile], const Spots<N>& p) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const __amdgpu_buffer_rsrc_t kr = raw_buffer(spot_base(a.k, p.at[i], slot_mask, kv_head), 0x7fffffff);
      const __amdgpu_buffer_rsrc_t vr = raw_buffer(spot_base(a.v, p.at[i], slot_mask, kv_head), 0x7fffffff);
#pragma unroll
      for (int hh = 0; hh < 2 / N; ++hh) {
        const int half = i * (2 / N) + hh;
#pragma unroll
        for (int j = 0; j < kHalfOps; ++j) dma16(kr, koff[j], hh * k16, &to[0][1024 * (kHalfOps * half + j)]);
#pragma unroll
        for (int j = 0; j < kHalfOps; ++j) dma16(vr, voff[j], hh * v16, &to[1][1024 * (kHalfOps * half + j)]);
      }
    }
  };

  RowState<D> st;
  st.clear();
  Spots<N> now, next;  // the tile in use, the one that is loaded
  FoundAll<N> after;   // the one behind it
  // Tile t is in one stage; the reads of the other have returned: refill it.
  auto turn = [&](uint8_t (&to)[2][kTile], int t) {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0), other counters untouched
    if (t + NW < n_tiles) {
      next = to_spots(a, after);
      issue(to, next);
      after = find_all(min(t + 2 * NW, n_tiles - 1));
      wait_vmcnt<4 * kHalfOps>();
    } else {
      wait_vmcnt<0>();
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
    __builtin_amdgcn_sched_barrier(0);
  };
  // whether every row sees all of the tile
  auto whole = [&](const Spots<N>& p) {
    bool all = true;
#pragma unroll
    for (int i = 0; i < N; ++i) all &= p.at[i].key + kSpan - 1 <= lim_first && (p.at[i].visible & every) == every;
    return all;
  };
  const int tk = static_cast<int>(x.q_row) - w.q0 - tok0;  // the lane's token
  // Tiles that end behind some row's last key may hold anything there.  Where rows differ in
  // the blocks that they list, what is hidden from one is some other's value, and all but
  // always finite: these tiles are only looked through if an output says otherwise, in a second pass.
  bool careful = false;
  auto masked = [&](const uint8_t (&from)[2][kTile], int t) {
    bool ends = false;
#pragma unroll
    for (int i = 0; i < N; ++i) ends |= now.at[i].key + kSpan - 1 > lim_first;
    attend_halves<D, 1>(from[0], from[1], q, st, a.c, spot_limits<1>(now, x.limit, tk),
                        KEYS != kListSeveral || careful || ends, a.v.row_stride, [&](int i) {
                          return spot_base(a.v, to_spot(a, find(t, i * N / 2)), slot_mask, kv_head) + i % (2 / N) * 16 * a.v.row_stride;
                        });
  };
  int t = wave;
  auto start = [&] {
    if (t < n_tiles) {
      now = to_spots(a, find_all(t));
      issue(smem0[wave], now);
      after = find_all(min(t + NW, n_tiles - 1));
    }
  };
  start();
  if (KEYS == kListSeveral) {
    for (;;) {
      for (; t < n_tiles; t += 2 * NW) {
        turn(smem1[wave], t);
        masked(smem0[wave], t);
        now = next;
        if (t + NW >= n_tiles) break;
        turn(smem0[wave], t + NW);
        masked(smem1[wave], t + NW);
        now = next;
      }
      if (careful || !not_finite(st)) break;
      careful = true;
      st.clear();
      t = wave;
      __builtin_amdgcn_s_waitcnt(0xc07f);  // the reads of both stages have returned
      start();
    }
  } else {
    // tiles that every row sees whole, in pairs; the rest
    int stage = 0;
    while (t < n_tiles && whole(now)) {
      turn(smem1[wave], t);
      attend<D, 1, false, kKeep<D>>(smem0[wave][0], smem0[wave][1], q, st, a.c, 0, false);
      now = next;
      t += NW;
      stage = 1;
      if (t >= n_tiles || !whole(now)) break;
      turn(smem0[wave], t);
      attend<D, 1, false, kKeep<D>>(smem1[wave][0], smem1[wave][1], q, st, a.c, 0, false);
      now = next;
      t += NW;
      stage = 0;
    }
    for (; t < n_tiles; t += NW, stage ^= 1) {
      uint8_t(&from)[2][kTile] = stage ? smem1[wave] : smem0[wave];
      turn(stage ? smem0[wave] : smem1[wave], t);
      masked(from, t);
      now = next;
    }
  }
  __syncthreads();

  // the merge: quad d of row r of a wave is at slot d ^ (r mod 16), off the other rows' banks
  auto merge = [&](int wv, int r, int quad) {
    return reinterpret_cast<f32x4*>(&smem0[0][0][0]) + (wv * 32 + r) * (D / 4) + (quad ^ (r & 15));
  };
  const int n = lane & 31, h = lane >> 5;
  const float lsum = sum_halves(st.l);
  if (n < here) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *merge(wave, n, 8 * i + 2 * j + h) =
            f32x4{st.o[i][4 * j], st.o[i][4 * j + 1], st.o[i][4 * j + 2], st.o[i][4 * j + 3]};
    if (h == 0) s_m[wave][n] = st.m, s_l[wave][n] = lsum;
  }
  __syncthreads();
  const bool direct = a.every_slot() ? a.slots == 1 : splits <= 1;
  for (int u = threadIdx.x; u < here * (D / 4); u += 64 * NW) {
    const int r = u / (D / 4), d = 4 * (u % (D / 4));
    float m = kNegInf, l = 0.f;
#pragma unroll
    for (int i = 0; i < NW; ++i) m = fmaxf(m, s_m[i][r]);
    const float ms = m == kNegInf ? 0.f : m;
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      const float f = __builtin_amdgcn_exp2f((s_m[i][r] - ms) * a.c);
      l += f * s_l[i][r];
      o += f * *merge(i, r, d / 4);
    }
    const int pos = (r0 + r) / a.group;
    const int64_t q_row = w.q0 + pos;
    const int head = kv_head * a.group + r0 + r - pos * a.group;
    if (direct) {
      store_quad(a, q_row, head, d, o, m, l);
    } else {
      const int64_t row = part_row(a, split, q_row, head);
      *reinterpret_cast<f32x4*>(a.part_o + row * D + d) = o;
      if (d == 0) a.part_ml[row] = make_float2(m, l);
    }
  }
}

// ---------------------------------------------------------------- many rows
constexpr int kRowsP = 128;  // rows of a block: 4 waves x 32
constexpr int kKeysP = 64;   // keys of a tile

// 4 waves x 32 rows and tiles of 64 keys that all of them read: 2 x 32 KB of LDS at heads of 128, two blocks on a
// CU, one's softmax under the other's products.  A prefix of 16384 keys under 1003 rows of 32 heads: 293 to 304 us for the
// whole call, 0.94 to 0.90 PFLOP/s (matrix pipes busy 45 %, vector pipes 41 %).  Listed blocks are masked
// tiles throughout, also the third of them that every token of a wave lists whole (509 tokens, 40 pages of 32 each: 48 us; in
// 32-row tiles 94).
// A launch has units of kv_heads blocks each: (tile, split) pairs of sequences over their
// own keys, or over listed blocks, and behind them those of groups over their prefixes.
// (64 single tokens behind a prefix of 16384, whole call, before its pieces had their present sizes, 99 now: 101 us;
// prefix first 113; the kinds evenly mixed 113 to 126, as a block that multiplies then waits for its keys behind
// those that stream the caches.)
template <int D, bool LISTED, int N>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void paged_rows_kernel(PagedArgs a) {
  constexpr int kTile = kKeysP * 2 * D;
  constexpr int kOps = kTile / 4096;  // DMA instructions per wave and tile
  constexpr int kSpan = kKeysP / N;   // keys of a spot
  // two variables: see paged_token_kernel
  __shared__ __attribute__((aligned(1024))) uint8_t smem0[2][kTile];
  __shared__ __attribute__((aligned(1024))) uint8_t smem1[2][kTile];
  __shared__ ListEntry<4> s_list[LISTED ? kList : 1];
  static_assert(sizeof(smem0) >= 4 * (2 * kWords + 16), "the list's scratch is in a stage");
  const int kv_head = blockIdx.x % a.kv_heads;
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63;
  int unit = blockIdx.x / a.kv_heads;
  bool prefix = false;
  if (!LISTED && a.prefix_units > 0) {
    const int own = a.units - a.prefix_units;
    prefix = unit >= own;
    unit -= prefix ? own : 0;
  }
  const int tiles = prefix ? a.prefix_tiles : a.tiles;
  const int split = uniform(unit / tiles), tile = unit - split * tiles;
  PagedTile w;
  LaneRow x;
  int r0 = 0, n_rows = 0;
  // the last key that some row of the wave sees; the last that every row of the block sees; keys of the
  // block; the last key that every row of the wave sees
  int lim_last, block_first, all, lim_first = 0;
  if (prefix) {
    GroupRange g;
    if (!find_group_tile(a, tile, kRowsP, w, g)) return;
    x = lane_row(a, w, kv_head, w.tile * kRowsP + 32 * wave + (lane & 31), w.lq * a.group);
    // the row's sequence: the last one that begins at or before it; often they have a row each
    int lo = min(g.first + static_cast<int>(x.q_row) - w.q0, g.past - 1), hi = lo + 1;
    PagedRange s = sequence(a, lo, 0);
    if (x.q_row < s.q0 || (hi < g.past && x.q_row >= s.q0 + s.lq)) {
      lo = g.first, hi = g.past;
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (a.s.cu_q[mid] <= x.q_row) lo = mid; else hi = mid;
      }
      s = sequence(a, lo, 0);
    }
    const int pos = static_cast<int>(x.q_row) - s.q0;
    x.limit = min(pos + s.diag, w.end - 1);
    if (pos < 0 || pos >= min(s.lq, a.max_q)) x.valid = false, x.limit = w.end - 1;
    block_first = lim_last = x.limit;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      block_first = min(block_first, __shfl_xor(block_first, off, 64));
      lim_last = max(lim_last, __shfl_xor(lim_last, off, 64));
    }
    lim_last = uniform(lim_last);
    __shared__ int s_first[4];
    if (lane == 0) s_first[wave] = block_first;
    __syncthreads();
    block_first = uniform(min(min(s_first[0], s_first[1]), min(s_first[2], s_first[3])));
    all = w.end;
  } else {
    LaneGroup mine = {};
    if (a.n_groups > 0) mine = lane_group(a, 0);
    if (!find_tile(a, tile, kRowsP, w)) return;
    if (a.n_groups > 0) behind_prefix(w, prefix_of(a, w.seq, mine), a.max_prefix, a.max_kv, a.s.capacity, a.s.shift);
    r0 = (w.tiles - 1 - w.tile) * kRowsP;  // the last tiles see the most keys: first
    n_rows = min(w.lq, a.max_q) * a.group;
    const int rw = r0 + 32 * wave;
    x = lane_row(a, w, kv_head, rw + (lane & 31), n_rows);
    block_first = last_key(w, r0 / a.group);
    lim_first = last_key(w, min(rw, n_rows - 1) / a.group);
    lim_last = rw < n_rows ? last_key(w, min(rw + 31, n_rows - 1) / a.group) : -1;  // a wave without rows only loads
    all = max(last_key(w, (min(r0 + kRowsP, n_rows) - 1) / a.group) + 1 - w.own, 0);
  }
  const int chunk = prefix ? a.prefix_chunk : a.chunk;
  const int slot = prefix ? split : a.prefix_splits + split;
  auto empty = [&](int at) {
    if (x.valid && lane < 32) empty_share(a, at, x.q_row, x.head);
  };
  int splits = 1, entries = 0, kbeg = 0, kend;  // listed: kbeg and kend count the list's keys
  if (LISTED) {
    entries = uniform(build_list<256>(a, w, kv_head, r0, min(n_rows - r0, kRowsP), split, s_list,
                                      reinterpret_cast<uint32_t*>(&smem0[0][0])));
    kend = entries << a.s.shift;
    if (kend == 0 && a.slots > 1) return empty(slot);
  } else {
    splits = (all + chunk - 1) / chunk;  // that have keys to see
    if (!prefix && a.n_groups > 0 && split == 0 && w.own == 0)
      for (int i = 0; i < a.prefix_splits; ++i) empty(i);
    const SplitWork work = split_work(split, splits, a.slots, a.n_groups > 0);
    if (work == SplitWork::kEmpty) return empty(slot);
    if (work == SplitWork::kNothing) return;
    kbeg = w.own + split * chunk, kend = kbeg + min(all - split * chunk, chunk);
  }

  bf16x8 q[D / 16];
  load_q<D>(a, x, q);
  const int slot_mask = (1 << a.s.shift) - 1;
  ConstInts table = const_ints(a.s.table + w.seq * a.s.table_stride);
  // instruction i of a wave fills rows from (4 i + wave) * 512 / D on: one half each
  constexpr int kRowsOp = 512 / D;
  constexpr int kSame = D == 256 ? 2 : 1;  // instructions of a wave in a half
  const int in_half = D == 256 ? 0 : D == 128 ? wave : wave & 1;  // place of instruction 0 in its half
  int koff[kSame], voff[kSame];
#pragma unroll
  for (int i = 0; i < kSame; ++i) {
    koff[i] = half_offset<D, false>(D == 256 ? 4 * i + wave : in_half, static_cast<int>(a.k.row_stride) * 2);
    voff[i] = half_offset<D, true>(D == 256 ? 4 * i + wave : in_half, static_cast<int>(a.v.row_stride) * 2);
  }
  auto find = [&](int key) -> Found {
    return LISTED ? list_look_up<kSpan>(a, s_list, entries, key / kSpan, wave) : look_up(a, table, key);
  };
  auto find_all = [&](int key) {
    FoundAll<N> p;
#pragma unroll
    for (int i = 0; i < N; ++i) p.at[i] = find(key + kSpan * i);
    return p;
  };
  const int k16 = 32 * static_cast<int>(a.k.row_stride), v16 = 32 * static_cast<int>(a.v.row_stride);  // bytes of 16 rows
  auto issue = [&](uint8_t (&to)[2][kTile], const Spots<N>& p) {
    __amdgpu_buffer_rsrc_t kr, vr;
    if (N == 1) {
      kr = raw_buffer(spot_base(a.k, p.at[0], slot_mask, kv_head), 0x7fffffff);
      vr = raw_buffer(spot_base(a.v, p.at[0], slot_mask, kv_head), 0x7fffffff);
    }
#pragma unroll
    for (int i = 0; i < kOps; ++i) {
      // row (4 i + wave) * kRowsOp of the tile is in half `half`, for heads of 64 and the upper waves one on
      constexpr int kEach = 4 / N;  // halves of a spot
      const int half = 4 * i * kRowsOp / 16, more = D == 64 ? wave >> 1 : 0;
      if (N == 4 || (N == 2 && (i == 0 || half % kEach == 0))) {
        Spot y = p.at[half / kEach];
        if (N == 4 && more) y = p.at[half / kEach + 1];
        kr = raw_buffer(spot_base(a.k, y, slot_mask, kv_head), 0x7fffffff);
        vr = raw_buffer(spot_base(a.v, y, slot_mask, kv_head), 0x7fffffff);
      }
      dma16(kr, koff[i % kSame], N < 4 ? (half % kEach + more) * k16 : 0, &to[0][1024 * (4 * i + wave)]);
      dma16(vr, voff[i % kSame], N < 4 ? (half % kEach + more) * v16 : 0, &to[1][1024 * (4 * i + wave)]);
    }
  };

  RowState<D> st;
  st.clear();
  Spots<N> now, next;  // the tile in use, the one that is loaded
  FoundAll<N> after;   // the one behind it
  // Tile `key` has arrived in one stage and every wave is done with the other: refill that.
  auto turn = [&](uint8_t (&to)[2][kTile], int key) {
    wait_vmcnt<0>();
    stage_barrier();
    if (key + kKeysP < kend) {
      next = to_spots(a, after);
      issue(to, next);
      after = find_all(key + 2 * kKeysP);  // past the end: some page, unused
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto masked = [&](const uint8_t (&from)[2][kTile], int key, const Limits<kKeysP / 32>& lim, bool scan) {
    attend_halves<D, kKeysP / 32>(from[0], from[1], q, st, a.c, lim, scan, a.v.row_stride,
                                  [&](int i) {
                                    return spot_base(a.v, to_spot(a, find(key + 16 * i / kSpan * kSpan)), slot_mask, kv_head) +
                                           16 * i % kSpan * a.v.row_stride;
                                  });
  };
  int key = kbeg;
  auto start = [&] {
    if (key < kend) {
      now = to_spots(a, find_all(key));
      issue(smem0, now);
      after = find_all(key + kKeysP);
    }
  };
  start();
  if (LISTED) {
    const int tk = static_cast<int>(x.q_row) - w.q0 - (r0 + 32 * wave) / a.group;  // the lane's token of the wave's
    bool careful = false;  // see paged_token_kernel
    auto use = [&](const uint8_t (&from)[2][kTile], int key) {
      uint32_t any = 0;
      int last = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) any |= now.at[i].visible, last = max(last, now.at[i].key + kSpan - 1);
      if (any) masked(from, key, spot_limits<kKeysP / 32>(now, x.limit, tk), careful || last > lim_first);
      now = next;
    };
    for (;;) {
      if (kKeep<D>) {
        for (; key < kend; key += 2 * kKeysP) {
          turn(smem1, key);
          use(smem0, key);
          if (key + kKeysP >= kend) break;
          turn(smem0, key + kKeysP);
          use(smem1, key + kKeysP);
        }
      } else {  // one copy of the code: two need more registers than there are
        for (int stage = 0; key < kend; key += kKeysP, stage ^= 1) {
          turn(stage ? smem0 : smem1, key);
          use(stage ? smem1 : smem0, key);
        }
      }
      if (careful || !__syncthreads_or(not_finite(st))) break;
      careful = true;
      st.clear();
      key = kbeg;
      start();
    }
  } else {
    auto valid = [&](const Spots<N>& p) {
      uint32_t all = ~0u;
#pragma unroll
      for (int i = 0; i < N; ++i) all &= p.at[i].visible;
      return all != 0;
    };
    int stage = 0;
    // tiles that every row of the block sees whole, in pairs
    const int full = min(kend, block_first + 1);
    while (key + kKeysP <= full && valid(now)) {
      turn(smem1, key);
      if (lim_last >= 0) attend<D, kKeysP / 32, false, kKeep<D>>(smem0[0], smem0[1], q, st, a.c, 0, false);
      now = next;
      key += kKeysP;
      stage = 1;
      if (key + kKeysP > full || !valid(now)) break;
      turn(smem0, key);
      if (lim_last >= 0) attend<D, kKeysP / 32, false, kKeep<D>>(smem1[0], smem1[1], q, st, a.c, 0, false);
      now = next;
      key += kKeysP;
      stage = 0;
    }
    // the rest
    for (; key < kend; key += kKeysP, stage ^= 1) {
      uint8_t(&from)[2][kTile] = stage ? smem1 : smem0;
      turn(stage ? smem0 : smem1, key);
      if (key <= lim_last) masked(from, key, spot_limits<kKeysP / 32>(now, x.limit, 0), true);
      now = next;
    }
  }

  const float l = sum_halves(st.l);
  if (!x.valid) return;
  const int h = lane >> 5;
  const bool direct = a.every_slot() ? a.slots == 1 : splits <= 1;
  const int64_t row = part_row(a, slot, x.q_row, x.head);
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // register 4 j + e of o[i] is output 32 i + 8 j + 4 h + e
      const f32x4 o = {st.o[i][4 * j], st.o[i][4 * j + 1], st.o[i][4 * j + 2], st.o[i][4 * j + 3]};
      const int d = 32 * i + 8 * j + 4 * h;
      if (direct)
        store_quad(a, x.q_row, x.head, d, o, st.m, l);
      else
        *reinterpret_cast<f32x4*>(a.part_o + row * D + d) = o;
    }
  if (!direct && h == 0) a.part_ml[row] = make_float2(st.m, l);
}

// ---------------------------------------------------------------- the join of the shares
// A thread per four outputs of a row, kJoin shares at a time, so that their latencies
// overlap; with more than kJoinShared slots the block has one row, and its thread groups
// take turns over them and meet in LDS.  Either way in a fixed order.  (64 tokens of 32 heads in 18 slots, 19 MB: 9 us.)
constexpr int kJoin = 8, kJoinShared = 2 * kJoin;
template <int D>
__global__ __launch_bounds__(256) void paged_join_kernel(PagedArgs a) {
  constexpr int kGroups = 256 / (D / 4);
  __shared__ f32x4 s_o[kGroups][D / 4];
  __shared__ float2 s_ml[kGroups];
  const int grp = threadIdx.x / (D / 4), quad = threadIdx.x % (D / 4);
  const bool shared = a.join_rows == 1;
  const int64_t u = static_cast<int64_t>(blockIdx.x) * a.join_rows + (shared ? 0 : grp);
  int64_t q_row = u / a.q_heads;
  const int head = static_cast<int>(u - q_row * a.q_heads);
  int seq, pos;
  if (a.token) {  // u counts the rows below max_q of each sequence
    seq = static_cast<int>(q_row / a.max_q);
    if (seq >= a.s.n_seqs) return;
    pos = static_cast<int>(q_row - static_cast<int64_t>(seq) * a.max_q);
  } else {  // u counts q's rows: the sequence is the last one that begins at or before it
    if (q_row >= a.s.q_rows) return;
    int lo = min(static_cast<int>(q_row), a.s.n_seqs - 1), hi = a.s.n_seqs;
    if (a.s.cu_q[lo] > q_row || (lo + 1 < hi && a.s.cu_q[lo + 1] <= q_row)) lo = 0;  // not one row each
    else hi = lo + 1;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (a.s.cu_q[mid] <= q_row) lo = mid; else hi = mid;
    }
    seq = lo;
    pos = 0;
  }
  const PagedRange w = sequence(a, seq, 0);
  if (a.token)
    q_row = w.q0 + pos;
  else
    pos = static_cast<int>(q_row) - w.q0;
  if (pos < 0 || pos >= min(w.lq, a.max_q)) return;
  int splits = a.slots;
  if (!a.every_slot()) {
    // The tile kernels cut by what the tile's last row sees.
    const int last = min((pos * a.group + head % a.group) / a.tile_rows * a.tile_rows + a.tile_rows,
                         min(w.lq, a.max_q) * a.group) - 1;
    splits = (max(last_key(w, last / a.group) + 1, 0) + a.chunk - 1) / a.chunk;
    if (splits <= 1) return;  // written by its tile
  }
  float m = kNegInf, l = 0.f;
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  // a share (ml, p) with weight 2^((its maximum - m) c)
  auto rescale = [&](float to) {
    const float f = m == to ? 1.f : __builtin_amdgcn_exp2f((m - to) * a.c);
    m = to;
    l *= f;
    o *= f;
  };
  auto add = [&](float2 ml, f32x4 p) {
    const float f = __builtin_amdgcn_exp2f((ml.x - (m == kNegInf ? 0.f : m)) * a.c);
    l += f * ml.y;
    o += f * p;
  };
  const int step = shared ? kGroups : 1;
  for (int i = shared ? grp : 0; i < splits; i += kJoin * step) {
    float2 ml[kJoin];
    f32x4 part[kJoin];
#pragma unroll
    for (int j = 0; j < kJoin; ++j) {
      ml[j] = make_float2(kNegInf, 0.f);
      if (i + j * step < splits) ml[j] = a.part_ml[part_row(a, i + j * step, q_row, head)];
    }
#pragma unroll
    for (int j = 0; j < kJoin; ++j) {
      part[j] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (ml[j].y != 0.f)  // a slot without keys has no output
        part[j] = *reinterpret_cast<const f32x4*>(a.part_o + part_row(a, i + j * step, q_row, head) * D + 4 * quad);
    }
    float top = m;
#pragma unroll
    for (int j = 0; j < kJoin; ++j) top = fmaxf(top, ml[j].x);
    rescale(top);
#pragma unroll
    for (int j = 0; j < kJoin; ++j) add(ml[j], part[j]);
  }
  if (shared) {  // the whole block is here: it has one row
    s_o[grp][quad] = o;
    if (quad == 0) s_ml[grp] = make_float2(m, l);
    __syncthreads();
    if (grp != 0) return;
    float top = m;
#pragma unroll
    for (int g = 1; g < kGroups; ++g) top = fmaxf(top, s_ml[g].x);
    rescale(top);
#pragma unroll
    for (int g = 1; g < kGroups; ++g) add(s_ml[g], s_o[g][quad]);
  }
  store_quad(a, q_row, head, 4 * quad, o, m, l);
}

// ---------------------------------------------------------------- host
constexpr int kCus = 256;
constexpr int kRounds = 64;

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Plan {
  bool token;                   // the few-rows kernel: every sequence is one tile
  int waves;                    // of its blocks
  int64_t tiles, prefix_tiles;  // row tiles
  int chunk, splits;            // own keys of a split (listed blocks: the fewest); splits
  int prefix_chunk, prefix_splits;
  int slots() const { return splits + prefix_splits; }
  int64_t prefix_units() const { return prefix_tiles * prefix_splits; }
  int64_t units() const { return tiles * splits + prefix_units(); }
};

// Tokens that a tile may hold rows of.
int tile_tokens(int group, int max_q, bool token) {
  const int rows = token ? kRowsT : kRowsP;
  const int n = rows % group == 0 ? rows / group : group % rows == 0 ? 1 : (rows - 2) / group + 2;
  return std::min(n, max_q);
}

// Keys of a block for `tiles` tiles over `keys` keys: enough blocks to fill the card,
// pieces not so small that their join costs more than it gains.
int64_t pick_chunk(int64_t keys, int64_t tiles, int64_t unit, int64_t want, int64_t least, int64_t most) {
  int64_t chunk = ceil_div(keys, std::max<int64_t>(1, ceil_div(want, std::max<int64_t>(tiles, 1))));
  chunk = std::min(std::max(chunk, least), most);
  return ceil_div(ceil_div(keys, ceil_div(keys, chunk)), unit) * unit;  // equal pieces
}

// Tiles of kRowsP rows that `rows` rows in up to `parts` sequences or groups make.
int64_t tile_bound(int64_t rows, int64_t parts) { return (rows + (kRowsP - 1) * parts) / kRowsP; }

// Measured in us as a HIP graph, heads of 128 unless said; want, least and most are blocks, and keys of a block, in the
// terms of pick_chunk.
Plan make_plan(const moe_paged_attn& d) {
  Plan p = {};
  const moe_paged& s = d.p;
  const int64_t g = s.q_heads / s.kv_heads;
  const int64_t seqs = std::min<int64_t>(s.n_seqs, s.q_rows);
  const bool listed = d.n_blocks > 0, grouped = d.n_groups > 0;
  const bool few = d.max_q * g <= kRowsT;
  // One launch for prefixes and own keys, so that neither waits for the other's last blocks: the rows
  // kernel takes both, also for single tokens (64 tokens behind 16384 keys 114 in two launches, 105).
  p.token = few && !grouped;
  p.tiles = p.token ? s.n_seqs : tile_bound(s.q_rows * g, seqs);
  const int64_t tiles = std::max<int64_t>(p.tiles * s.kv_heads, 1);
  const int64_t rest = grouped ? s.page_size - 1 : 0;  // of the prefix's last page
  int64_t keys = std::max(d.max_kv, 1) + rest;
  if (listed)
    keys = std::max<int64_t>(1, std::min<int64_t>(static_cast<int64_t>(tile_tokens(g, d.max_q, p.token)) * d.n_blocks,
                                                  ceil_div(keys, s.page_size))) * s.page_size;
  // Two waves where there are many tiles: two blocks share a CU, and one loads while the other merges (64
  // tokens over up to 1024 keys 39 against 42 with four, over 8192 216 and 218); four where there are few (16
  // over 4096, heads of 64: 21 against 24).  Heads of 256 have LDS for two.
  p.waves = s.head_dim == 256 || tiles >= 2 * kCus ? 2 : 4;
  const int64_t unit = p.token ? kKeysT * p.waves : kKeysP;
  // As many blocks as the card holds at a time; half as many beside a prefix, whose own
  // fill the card too (three chunks of 200 behind 8192, heads of 256: 147 against 150; heads of 128 the same).  Listed
  // blocks of 509 tokens: half of them 54, twice 48, as they are 48.
  const int64_t want = (s.head_dim > (p.token ? 64 : 128) ? kCus : 2 * kCus) / (grouped ? 2 : 1);
  // Pieces of at least two or four tiles a wave (one listed token over 64 pages: 12.6 with one, 14 with two, 14.4 with
  // four, 18 with eight; 4 tokens behind a prefix 13.7, 12.9, 12.9), more in the rows kernel the more tiles
  // there are (listed blocks of 509 tokens: four 56, eight 47, sixteen 50).
  const int64_t least = p.token ? (keys <= 4 * unit ? 4 : 2) * unit
                                : std::min(std::max(tiles / 16, int64_t{4}), int64_t{16}) * unit;
  // Few rows over long caches of many lengths: at most 16 units a piece, so that a long one does not run on
  // alone, but no more than kRounds rounds of blocks.  8, 16, 32: 64 tokens over 8192 keys 221, 216, 223; behind a
  // prefix 24 over 8192 -, 110, 116, heads of 64, 64 over 4096 -, 75, 81.  What is left of the prefix's page
  // makes no piece of its own (64 over 2048 104 with it, 99; 24 over 8192 110, 103; 64 over 4096, heads of 256, 168, 178).
  const int64_t most = !few || listed ? INT32_MAX
                                      : std::max(16 * unit + rest, ceil_div(keys, std::max(kRounds * kCus / tiles, int64_t{1})));
  const int64_t chunk = pick_chunk(keys, tiles, unit, want, least, most);
  if (listed) {
    // How many blocks a tile's tokens list together is known to the kernel alone: as many as one
    // of them at least, and hardly more where they agree.
    const int64_t least_blocks = std::max<int64_t>(least / s.page_size, 1);
    const int64_t wanted = std::min(ceil_div(want, tiles), ceil_div(std::min<int64_t>(d.n_blocks, keys / s.page_size), least_blocks));
    p.chunk = static_cast<int>(least_blocks);
    p.splits = static_cast<int>(std::max(wanted, ceil_div(keys / s.page_size, kList)));
  } else {
    p.chunk = static_cast<int>(chunk);
    p.splits = static_cast<int>(ceil_div(keys, chunk));
  }
  if (grouped && d.max_prefix >= s.page_size) {
    p.prefix_tiles = tile_bound(s.q_rows * g, std::min<int64_t>(d.n_groups, s.q_rows));
    const int64_t blocks = p.prefix_tiles * s.kv_heads;
    // One block a CU, or two where that gains more than the shares of twice the splits cost: a second block on a CU
    // hides about a third of a tile's 400 ns.  256
    // blocks, 512: eight chunks of up to 256 behind 16384 432, 295; four of 64 behind 8192 44, 48; heads of 256, three of 200 164, 150.
    // Those have one block on a CU either way, so what they gain is smaller pieces at the end; the 800 is fitted to that case alone.
    const int64_t splits = std::max<int64_t>(kCus / std::max<int64_t>(blocks, 1), 1);
    const int64_t gain = blocks * ceil_div(d.max_prefix, kKeysP) / kCus * (s.head_dim == 256 ? 800 : s.head_dim);
    const int64_t cost = splits * 8 * s.q_rows * s.q_heads * s.head_dim / 5000;  // ns: stored and loaded once at 5 TB/s
    const int64_t piece = pick_chunk(d.max_prefix, blocks, kKeysP, gain > cost ? 2 * kCus : kCus,
                                     std::min(std::max(blocks / 16, int64_t{4}), int64_t{16}) * kKeysP, INT32_MAX);
    p.prefix_chunk = static_cast<int>(piece);
    p.prefix_splits = static_cast<int>(ceil_div(d.max_prefix, piece));
  }
  return p;
}

inline size_t align256(size_t v) { return (v + 255) & ~size_t{255}; }

size_t part_bytes(const moe_paged_attn& d, const Plan& p) {
  if (p.slots() <= 1) return 0;
  const size_t rows = static_cast<size_t>(p.slots()) * d.p.q_rows * d.p.q_heads;
  return align256(rows * d.p.head_dim * 4) + align256(rows * 8);
}

// Rows of a block of the join, and its blocks.
int join_rows(const moe_paged_attn& d, const Plan& p) { return p.slots() > kJoinShared ? 1 : 256 / (d.p.head_dim / 4); }
int64_t join_blocks(const moe_paged_attn& d, const Plan& p) {
  if (p.slots() <= 1) return 0;
  const int64_t rows = (p.token ? static_cast<int64_t>(d.p.n_seqs) * d.max_q : d.p.q_rows) * d.p.q_heads;
  return ceil_div(rows, join_rows(d, p));
}

// The shape fields, which the workspace depends on.
int check_shape(const moe_paged_attn* a) {
  if (!a) return MOE_EINVAL;
  const int st = check_paged_shape(a->p, false);
  if (st != MOE_OK) return st;
  const int64_t capacity = static_cast<int64_t>(a->p.table_pages) * a->p.page_size;
  if (a->max_q < 0 || a->max_q > a->p.q_rows || a->max_kv < 0 || a->max_kv > capacity) return MOE_EINVAL;
  if (a->max_prefix < 0 || a->max_prefix > capacity || a->n_groups < 0 || a->n_groups > a->p.n_seqs) return MOE_EINVAL;
  if (a->n_blocks < 0 || (a->n_blocks > 0 && a->n_groups > 0)) return MOE_EINVAL;
  if (a->n_blocks > 1024) return MOE_ESHAPE;
  if (a->n_blocks > 0 && a->max_kv > static_cast<int64_t>(32 * kWords) * a->p.page_size) return MOE_ESHAPE;
  const Plan p = make_plan(*a);
  // grid limits: 2^32 threads along x, 65535 blocks along y
  if (p.units() > 0xffffff / a->p.kv_heads || p.splits > 65535 || join_blocks(*a, p) > 0xffffff) return MOE_ESHAPE;
  if (static_cast<int64_t>(a->p.q_rows) * a->p.q_heads > 0x3fffffff) return MOE_ESHAPE;
  return MOE_OK;
}

template <int D, int NW, int N>
void launch_token(const PagedArgs& a, dim3 grid, hipStream_t s) {
  if (!a.n_blocks)
    paged_token_kernel<D, kTable, NW, N><<<grid, 64 * NW, 0, s>>>(a);
  else if (a.max_q == 1)
    paged_token_kernel<D, kListOne, NW, N><<<grid, 64 * NW, 0, s>>>(a);
  else
    paged_token_kernel<D, kListSeveral, NW, N><<<grid, 64 * NW, 0, s>>>(a);
}

template <int D, int N>
void launch_rows(const PagedArgs& a, unsigned blocks, hipStream_t s) {
  if (a.n_blocks)
    paged_rows_kernel<D, true, N><<<blocks, 256, 0, s>>>(a);
  else
    paged_rows_kernel<D, false, N><<<blocks, 256, 0, s>>>(a);
}

template <int D>
void launch(const PagedArgs& a, const Plan& p, int64_t joins, hipStream_t s) {
  if (p.token) {
    const dim3 grid(static_cast<unsigned>(p.tiles * a.kv_heads), static_cast<unsigned>(p.splits));
    const bool whole = 1 << a.s.shift >= kKeysT;
    if (p.waves == 2)
      whole ? launch_token<D, 2, 1>(a, grid, s) : launch_token<D, 2, 2>(a, grid, s);
    else if (D < 256)
      whole ? launch_token<D, D < 256 ? 4 : 2, 1>(a, grid, s) : launch_token<D, D < 256 ? 4 : 2, 2>(a, grid, s);
  } else {
    const unsigned blocks = static_cast<unsigned>(p.units() * a.kv_heads);
    switch (a.s.shift) {
      case 4: launch_rows<D, 4>(a, blocks, s); break;
      case 5: launch_rows<D, 2>(a, blocks, s); break;
      default: launch_rows<D, 1>(a, blocks, s); break;
    }
  }
  if (joins > 0) paged_join_kernel<D><<<static_cast<unsigned>(joins), 256, 0, s>>>(a);
}

}  // namespace
}  // namespace moe

extern "C" {

size_t moe_paged_attention_workspace_size(const moe_paged_attn* a) {
  if (moe::check_shape(a) != MOE_OK || a->p.n_seqs == 0 || a->p.q_rows == 0 || a->max_q == 0) return 0;
  return moe::part_bytes(*a, moe::make_plan(*a));
}

int moe_paged_attention(const moe_paged_attn* a, void* ws, size_t ws_bytes, void* stream) {
  int st = moe::check_shape(a);
  if (st != MOE_OK) return st;
  if (!(a->scale > 0.f && a->scale <= 0x1p127f)) return MOE_EINVAL;  // scale * log2(e) is finite
  const moe_paged& p = a->p;
  if (p.n_seqs == 0 || p.q_rows == 0 || a->max_q == 0) return MOE_OK;
  if ((st = moe::check_paged_arrays(p)) != MOE_OK) return st;
  if (a->n_groups > 0 && (!a->cu_group || !a->prefix_len)) return MOE_EINVAL;
  if (a->n_blocks > 0 && !a->blocks) return MOE_EINVAL;
  for (const moe_heads* h : {&a->q, &a->out})
    if ((st = moe::check_paged_heads(*h)) != MOE_OK) return st;
  if (p.n_pages > 0)
    for (const moe_pages* h : {&a->k, &a->v})
      if ((st = moe::check_pages(*h)) != MOE_OK) return st;
  const moe::Plan plan = moe::make_plan(*a);
  const size_t need = moe::part_bytes(*a, plan);
  if (need) {
    if (!ws) return MOE_EINVAL;
    if (reinterpret_cast<uintptr_t>(ws) & 255) return MOE_EALIGN;
    if (ws_bytes < need) return MOE_EWORKSPACE;
  }
  moe::PagedArgs k;
  k.s = moe::paged_seqs(p);
  k.q = a->q, k.out = a->out, k.k = a->k, k.v = a->v;
  k.cu_group = a->cu_group, k.prefix_len = a->prefix_len, k.blocks = a->blocks, k.lse = a->lse;
  k.part_o = static_cast<float*>(ws);
  const size_t rows = static_cast<size_t>(plan.slots()) * p.q_rows * p.q_heads;
  k.part_ml =
      need ? reinterpret_cast<float2*>(static_cast<char*>(ws) + moe::align256(rows * p.head_dim * 4)) : nullptr;
  k.q_heads = p.q_heads, k.kv_heads = p.kv_heads, k.group = p.q_heads / p.kv_heads;
  k.max_q = a->max_q, k.n_groups = a->n_groups, k.n_blocks = a->n_blocks;
  k.max_kv = std::min(a->max_kv, k.s.capacity), k.max_prefix = std::min(a->max_prefix, k.s.capacity);
  k.chunk = plan.chunk, k.splits = plan.splits, k.prefix_chunk = plan.prefix_chunk, k.prefix_splits = plan.prefix_splits;
  k.slots = plan.slots();
  k.tiles = static_cast<int>(plan.tiles), k.prefix_tiles = static_cast<int>(plan.prefix_tiles);
  k.units = static_cast<int>(plan.units()), k.prefix_units = static_cast<int>(plan.prefix_units());
  k.token = plan.token;
  k.tile_rows = plan.token ? moe::kRowsT : moe::kRowsP;
  k.join_rows = moe::join_rows(*a, plan);
  k.scale = a->scale;
  k.c = a->scale * 1.44269504088896340736f;  // log2(e)
  const int64_t joins = moe::join_blocks(*a, plan);
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  switch (p.head_dim) {
    case 64: moe::launch<64>(k, plan, joins, s); break;
    case 128: moe::launch<128>(k, plan, joins, s); break;
    default: moe::launch<256>(k, plan, joins, s); break;
  }
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_EHIP;
}

}  // extern "C"
