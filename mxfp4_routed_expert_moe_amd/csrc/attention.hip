// Packed softmax attention with grouped heads: prompts, chunks of a prompt and
// single tokens over a cache (include/moe_attention.h, moe_attention).
//
// Rows.  The G = q_heads / kv_heads query heads that share a key head are
// folded into the rows of one problem per (sequence, key head): row r is query
// r / G, head r % G of the group.  A tile of rows then reads every key and
// value once for the whole group, and a causal tile spans few key positions.
//
// One pass over the keys with a running maximum and sum; what a tile of keys does to
// a wave's rows stands in attention_core.h.
#include <math.h>

#include <algorithm>

#include "../../include/moe_attention.h"
#include "attention_core.h"
#include "attention_ranges.h"

namespace moe {

namespace {

// What the kernels take: the descriptor and what the host derived from it.
struct AttnArgs {
  moe_heads q, k, v, out;
  const int32_t *cu_q, *kv_start, *kv_len;
  float* lse;
  float* part_o;    // [splits, q_rows, q_heads, D]
  float2* part_ml;  // [splits, q_rows, q_heads]: maximum, sum
  int n_seqs, q_rows, kv_rows, q_heads, kv_heads, group, max_q, max_kv, causal;
  int chunk;        // keys of a split, a multiple of the tile
  int tile_rows;    // rows of a block
  int token;        // 1: the few-rows kernel
  int join_rows;    // rows of a block of the join
  float scale, c;   // c = scale * log2(e)
};

// ---------------------------------------------------------------- masked tiles
// A tile that some rows do not see all of.  v: its rows in memory, `rows` of
// them; lim as in attend.  Where the values are all finite, the weight 0 of a
// masked key is enough.  Otherwise the product is taken over the finite values
// alone, and each row adds the others that it sees: a weight above zero
// times such a value is that value.
template <int D, int NT>
__device__ __forceinline__ void attend_masked(const uint8_t* ks, const uint8_t* vs, const uint16_t* v,
                                              int64_t row_stride, int rows, const bf16x8 (&q)[D / 16],
                                              RowState<D>& st, float c, int lim) {
  const bool dirty = any_not_finite(vs, NT * 32 * 2 * D);
  attend<D, NT, true>(ks, vs, q, st, c, lim, dirty);
  if (!dirty) return;
  const int h = (threadIdx.x & 63) >> 5;
  for (int r = 0; r < min(rows, NT * 32); ++r) {
    if (r > lim) break;
    add_not_finite<D>(v + r * row_stride + 4 * h, st);
  }
}

// ---------------------------------------------------------------- work
// A tile of up to `rows` folded rows of one sequence.  All fields are uniform.
struct TileWork : SeqRange {
  int tile, tiles;
};

// Rows and keys of sequence b, cut to the tensors and to max_kv.  lq keeps the
// full length; only the rows below max_q are worked on.
__device__ __forceinline__ SeqRange sequence(const AttnArgs& a, int b) {
  return seq_range(a.cu_q, a.kv_start, a.kv_len, b, a.q_rows, a.kv_rows, a.max_kv);
}
__device__ __forceinline__ int row_tiles(const AttnArgs& a, int lq, int rows) {
  return (min(lq, a.max_q) * a.group + rows - 1) / rows;
}

// Tile t over all sequences (each sequence's tiles in a row): its sequence and
// its place there, by a prefix sum over 64 sequences at a time.
__device__ bool find_tile(const AttnArgs& a, int t, int rows, TileWork& w) {
  const int lane = threadIdx.x & 63;
  for (int base = 0; base < a.n_seqs; base += 64) {
    SeqRange s = {0, 0, 0, 0, 0};
    int nt = 0;
    if (base + lane < a.n_seqs) {
      s = sequence(a, base + lane);
      nt = row_tiles(a, s.lq, rows);
    }
    const int incl = wave_incl_scan(nt);
    const uint64_t past = __ballot(incl > t);
    if (past) {
      const int src = __ffsll(static_cast<unsigned long long>(past)) - 1;
      w.q0 = uniform(__shfl(s.q0, src, 64));
      w.lq = uniform(__shfl(s.lq, src, 64));
      w.k0 = uniform(__shfl(s.k0, src, 64));
      w.lk = uniform(__shfl(s.lk, src, 64));
      w.diag = uniform(__shfl(s.diag, src, 64));
      w.tiles = uniform(__shfl(nt, src, 64));
      w.tile = uniform(t - (__shfl(incl, src, 64) - w.tiles));
      return true;
    }
    t -= uniform(__shfl(incl, 63, 64));
  }
  return false;
}

__device__ __forceinline__ int last_key(const AttnArgs& a, const TileWork& w, int pos) {
  return last_key(static_cast<const SeqRange&>(w), a.causal, pos);
}

// A lane's row: the query row and head it reads and writes.
struct LaneRow {
  int64_t q_row;
  int head, limit;
  bool valid;
};
__device__ __forceinline__ LaneRow lane_row(const AttnArgs& a, const TileWork& w, int kv_head, int r, int n_rows) {
  LaneRow x;
  x.valid = r < n_rows;
  const int rc = min(r, n_rows - 1);
  const int pos = rc / a.group;
  x.q_row = w.q0 + pos;
  x.head = kv_head * a.group + rc - pos * a.group;
  x.limit = last_key(a, w, pos);
  return x;
}

template <int D>
__device__ __forceinline__ void load_q(const AttnArgs& a, const LaneRow& x, bf16x8 (&q)[D / 16]) {
  const uint16_t* p = a.q.base + x.q_row * a.q.row_stride + x.head * a.q.head_stride + 8 * ((threadIdx.x & 63) >> 5);
#pragma unroll
  for (int i = 0; i < D / 16; ++i) q[i] = __builtin_bit_cast(bf16x8, ld16(p + 16 * i));
}

// Outputs d .. d + 3 of a row from the sums o and l over the maximum m.  l is 0
// only where the row saw no score above -infinity: its largest weight is at least
// 2^-kLazy.  Such a row gives zeros; o may hold infinite values times 0.
__device__ __forceinline__ void store_quad(const AttnArgs& a, int64_t q_row, int head, int d, f32x4 o, float m,
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

// A split's share of a row: the unscaled output, the maximum and the sum.
__device__ __forceinline__ int64_t part_row(const AttnArgs& a, int split, int64_t q_row, int head) {
  return (static_cast<int64_t>(split) * a.q_rows + q_row) * a.q_heads + head;
}

// LDS-DMA of a tile's rows: every instruction fills 1 KiB, 512 / D rows; the lane
// that lands in slot s of row r loads the chunk whose slot that is (the XOR is
// its own inverse).  Rows past `rows` repeat the last one: they are masked.
template <int D, bool VALUE>
__device__ __forceinline__ int dma_offset(int i, int rows, int row_bytes) {
  constexpr int kChunks = D / 8;
  const int lane = threadIdx.x & 63;
  const int r = i * (64 / kChunks) + lane / kChunks, s = lane % kChunks;
  return min(r, rows - 1) * row_bytes + 16 * (VALUE ? v_slot<D>(r, s) : k_slot<D>(r, s));
}

// ---------------------------------------------------------------- many rows
// Each wave holds 32 rows, their queries and outputs in registers; the four waves
// share the key tiles, which come through LDS by DMA in two stages.  Bound by the
// matrix and vector pipes together: a causal prompt of 16384, 32 query heads of 128,
// runs in 1.95 to 2.1 ms = 1.05 to 1.13 PFLOP/s at 1.8 GHz, matrix pipes busy 57 %
// and vector pipes 46 % of the time, no LDS bank conflict, 96 % of the reads served
// by L2.  (A library product of 8192^3 in bf16 reaches 1.21 PFLOP/s on this card.)
// With heads of 64 there is half the matrix work per weight: 8192 tokens, 16 heads,
// 167 us = 0.82 PFLOP/s.  Blocks of one key head go to one XCD as long as the
// number of key heads is a multiple of eight, so that they share it in L2 (dealt
// round, 2.13 ms).
constexpr int kRowsP = 128;  // rows of a block: 4 waves x 32
constexpr int kKeysP = 64;   // keys of a tile

template <int D>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void attn_rows_kernel(AttnArgs a) {
  constexpr int kTile = kKeysP * 2 * D;
  constexpr int kOps = kTile / 4096;  // DMA instructions per wave and tile
  // The stages are variables of their own: the compiler then knows that the
  // DMA in flight into one does not write the other, and does not wait for it.
  __shared__ __attribute__((aligned(1024))) uint8_t smem0[2][kTile];
  __shared__ __attribute__((aligned(1024))) uint8_t smem1[2][kTile];
  const int kv_head = blockIdx.x % a.kv_heads;
  TileWork w;
  if (!find_tile(a, blockIdx.x / a.kv_heads, kRowsP, w)) return;
  const int split = blockIdx.y;
  // the last tiles of a causal sequence see the most keys: first
  const int r0 = (w.tiles - 1 - w.tile) * kRowsP;
  const int n_rows = min(w.lq, a.max_q) * a.group;
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int rw = r0 + 32 * wave;
  const LaneRow x = lane_row(a, w, kv_head, rw + (lane & 31), n_rows);
  const int lim_last = last_key(a, w, min(rw + 31, n_rows - 1) / a.group);
  const int block_first = last_key(a, w, r0 / a.group);
  const int all = max(last_key(a, w, (min(r0 + kRowsP, n_rows) - 1) / a.group) + 1, 0);
  const int splits = (all + a.chunk - 1) / a.chunk;  // that have keys to see
  if (split >= max(splits, 1)) return;
  const int kbeg = split * a.chunk, kend = min(all, kbeg + a.chunk);

  bf16x8 q[D / 16];
  load_q<D>(a, x, q);
  const int krow = static_cast<int>(a.k.row_stride) * 2, vrow = static_cast<int>(a.v.row_stride) * 2;
  const uint16_t* kb = a.k.base + w.k0 * a.k.row_stride + kv_head * a.k.head_stride;
  const uint16_t* vb = a.v.base + w.k0 * a.v.row_stride + kv_head * a.v.head_stride;
  int koff[kOps], voff[kOps];
#pragma unroll
  for (int i = 0; i < kOps; ++i) {
    koff[i] = dma_offset<D, false>(4 * i + wave, kKeysP, krow);
    voff[i] = dma_offset<D, true>(4 * i + wave, kKeysP, vrow);
  }
  auto issue = [&](uint8_t (&to)[2][kTile], int key) {
    const __amdgpu_buffer_rsrc_t kr = raw_buffer(kb + key * a.k.row_stride, 0x7fffffff);
    const __amdgpu_buffer_rsrc_t vr = raw_buffer(vb + key * a.v.row_stride, 0x7fffffff);
    if (key + kKeysP <= w.lk) {
#pragma unroll
      for (int i = 0; i < kOps; ++i)
        dma16(kr, koff[i], 0, &to[0][1024 * (4 * i + wave)]);
#pragma unroll
      for (int i = 0; i < kOps; ++i)
        dma16(vr, voff[i], 0, &to[1][1024 * (4 * i + wave)]);
    } else {
      for (int i = 0; i < kOps; ++i) {
        dma16(kr, dma_offset<D, false>(4 * i + wave, w.lk - key, krow), 0, &to[0][1024 * (4 * i + wave)]);
        dma16(vr, dma_offset<D, true>(4 * i + wave, w.lk - key, vrow), 0, &to[1][1024 * (4 * i + wave)]);
      }
    }
  };

  RowState<D> st;
  st.clear();
  // Tile `key` has arrived in one stage and every wave is done with the other: refill that.
  auto turn = [&](uint8_t (&next)[2][kTile], int key) {
    wait_vmcnt<0>();
    stage_barrier();
    if (key + kKeysP < kend) issue(next, key + kKeysP);
    __builtin_amdgcn_sched_barrier(0);
  };
  int key = kbeg;
  if (key < kend) issue(smem0, key);
  // tiles that every row of the block sees whole, in pairs
  const int whole = min(kend, block_first + 1);
  for (; key + 2 * kKeysP <= whole; key += 2 * kKeysP) {
    turn(smem1, key);
    attend<D, kKeysP / 32, false>(smem0[0], smem0[1], q, st, a.c, 0, false);
    turn(smem0, key + kKeysP);
    attend<D, kKeysP / 32, false>(smem1[0], smem1[1], q, st, a.c, 0, false);
  }
  // the rest
  for (int stage = 0; key < kend; key += kKeysP, stage ^= 1) {
    uint8_t(&now)[2][kTile] = stage ? smem1 : smem0;
    turn(stage ? smem0 : smem1, key);
    if (key <= lim_last)
      attend_masked<D, kKeysP / 32>(now[0], now[1], vb + key * a.v.row_stride, a.v.row_stride, w.lk - key, q, st, a.c,
                                    x.limit - key);
  }

  const float l = sum_halves(st.l);
  if (!x.valid) return;
  const int h = lane >> 5;
  const int64_t row = part_row(a, split, x.q_row, x.head);
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // register 4 j + e of o[i] is output 32 i + 8 j + 4 h + e
      const f32x4 o = {st.o[i][4 * j], st.o[i][4 * j + 1], st.o[i][4 * j + 2], st.o[i][4 * j + 3]};
      const int d = 32 * i + 8 * j + 4 * h;
      if (splits <= 1)
        store_quad(a, x.q_row, x.head, d, o, st.m, l);
      else
        *reinterpret_cast<f32x4*>(a.part_o + row * D + d) = o;
    }
  if (splits > 1 && h == 0) a.part_ml[row] = make_float2(st.m, l);
}

// ---------------------------------------------------------------- few rows
// At most 32 folded rows of a sequence (a single token of up to 32 grouped
// heads): one wave's worth, so the waves share the rows and split the keys, each
// with a ring of its own and no barrier in the loop; the kernel streams the
// cache.  At the end the waves' shares meet in LDS.  Bound by HBM on long caches (64
// sequences of up to 8192 keys, 8 key heads of 128: 1.3 GB in 235 us = 5.5 TB/s; a large
// copy moves 5.2 TB/s), by latency on short ones (4 x 1024 keys: 8 us, and 3 us for
// the join).  32 rows here against a block of the kernel above (us): 64 x 8 queries of 4
// heads over 4096 keys 140, 149; 16 x 8 over 4096 keys of 64 24.9, 29.1; 8 x 8 over 8192 43.9, 42.4.
constexpr int kRowsD = 32;
constexpr int kKeysD = 32;
template <int D>
constexpr int decode_waves() { return D == 256 ? 2 : 4; }

template <int D>
__global__ __launch_bounds__(64 * decode_waves<D>(), 1) void attn_token_kernel(AttnArgs a) {
  constexpr int NW = decode_waves<D>();
  constexpr int kTile = kKeysD * 2 * D;
  constexpr int kOps = kTile / 1024;
  constexpr int kStep = kKeysD * NW;
  // two variables: see attn_rows_kernel
  __shared__ __attribute__((aligned(1024))) uint8_t smem0[NW][2][kTile];
  __shared__ __attribute__((aligned(1024))) uint8_t smem1[NW][2][kTile];
  __shared__ float s_m[NW][32], s_l[NW][32];
  static_assert(NW * 32 * D * 4 == sizeof(smem0), "the merge uses a stage");
  const int seq = blockIdx.x / a.kv_heads, split = blockIdx.y;
  // Blocks are dealt to the 8 XCDs in turn; with eight key heads that would tie a
  // head to an XCD, and the rows of one head, a power of two apart, to a part of
  // the channels of its L2.  So the heads of each sequence and split begin
  // elsewhere (64 x up to 8192 keys: 237 us against 246).
  const int kv_head = (blockIdx.x + seq + split) % a.kv_heads;
  TileWork w;
  const SeqRange range = sequence(a, seq);
  w.q0 = uniform(range.q0), w.lq = uniform(range.lq), w.k0 = uniform(range.k0), w.lk = uniform(range.lk);
  w.diag = uniform(range.diag);
  const int n_rows = min(w.lq, a.max_q) * a.group;
  if (n_rows == 0) return;
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const LaneRow x = lane_row(a, w, kv_head, lane & 31, n_rows);
  const int lim_first = last_key(a, w, 0);
  const int all = max(last_key(a, w, (n_rows - 1) / a.group) + 1, 0);
  const int splits = (all + a.chunk - 1) / a.chunk;
  if (split >= max(splits, 1)) return;
  const int kbeg = split * a.chunk, kend = min(all, kbeg + a.chunk);

  bf16x8 q[D / 16];
  load_q<D>(a, x, q);
  const int krow = static_cast<int>(a.k.row_stride) * 2, vrow = static_cast<int>(a.v.row_stride) * 2;
  const uint16_t* kb = a.k.base + w.k0 * a.k.row_stride + kv_head * a.k.head_stride;
  const uint16_t* vb = a.v.base + w.k0 * a.v.row_stride + kv_head * a.v.head_stride;
  auto issue = [&](uint8_t (&to)[2][kTile], int key) {
    const __amdgpu_buffer_rsrc_t kr = raw_buffer(kb + key * a.k.row_stride, 0x7fffffff);
    const __amdgpu_buffer_rsrc_t vr = raw_buffer(vb + key * a.v.row_stride, 0x7fffffff);
#pragma unroll
    for (int i = 0; i < kOps; ++i)
      dma16(kr, dma_offset<D, false>(i, w.lk - key, krow), 0, &to[0][1024 * i]);
#pragma unroll
    for (int i = 0; i < kOps; ++i)
      dma16(vr, dma_offset<D, true>(i, w.lk - key, vrow), 0, &to[1][1024 * i]);
  };

  RowState<D> st;
  st.clear();
  // Tile `key` is in one stage; the reads of the other have returned: refill it.
  auto turn = [&](uint8_t (&next)[2][kTile], int key) {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0), other counters untouched
    if (key + kStep < kend) {
      issue(next, key + kStep);
      wait_vmcnt<2 * kOps>();
    } else {
      wait_vmcnt<0>();
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
    __builtin_amdgcn_sched_barrier(0);
  };
  int key = kbeg + kKeysD * wave;
  if (key < kend) issue(smem0[wave], key);
  const int whole = min(kend, lim_first + 1);  // keys that every row sees
  for (; key + kStep + kKeysD <= whole; key += 2 * kStep) {
    turn(smem1[wave], key);
    attend<D, 1, false>(smem0[wave][0], smem0[wave][1], q, st, a.c, 0, false);
    turn(smem0[wave], key + kStep);
    attend<D, 1, false>(smem1[wave][0], smem1[wave][1], q, st, a.c, 0, false);
  }
  for (int stage = 0; key < kend; key += kStep, stage ^= 1) {
    uint8_t(&now)[2][kTile] = stage ? smem1[wave] : smem0[wave];
    turn(stage ? smem0[wave] : smem1[wave], key);
    attend_masked<D, 1>(now[0], now[1], vb + key * a.v.row_stride, a.v.row_stride, w.lk - key, q, st, a.c,
                        x.limit - key);
  }
  __syncthreads();

  // the merge: quad d of row r of a wave is at slot d ^ (r mod 16), off the other rows' banks
  auto merge = [&](int wv, int r, int quad) {
    return reinterpret_cast<f32x4*>(&smem0[0][0][0]) + (wv * 32 + r) * (D / 4) + (quad ^ (r & 15));
  };
  const int n = lane & 31, h = lane >> 5;
  const float lsum = sum_halves(st.l);
  if (n < n_rows) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *merge(wave, n, 8 * i + 2 * j + h) =
            f32x4{st.o[i][4 * j], st.o[i][4 * j + 1], st.o[i][4 * j + 2], st.o[i][4 * j + 3]};
    if (h == 0) s_m[wave][n] = st.m, s_l[wave][n] = lsum;
  }
  __syncthreads();
  for (int u = threadIdx.x; u < n_rows * (D / 4); u += 64 * NW) {
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
    const int pos = r / a.group;
    const int64_t q_row = w.q0 + pos;
    const int head = kv_head * a.group + r - pos * a.group;
    if (splits <= 1) {
      store_quad(a, q_row, head, d, o, m, l);
    } else {
      const int64_t row = part_row(a, split, q_row, head);
      *reinterpret_cast<f32x4*>(a.part_o + row * D + d) = o;
      if (d == 0) a.part_ml[row] = make_float2(m, l);
    }
  }
}

// ---------------------------------------------------------------- the join of the splits
// A thread per four outputs of a row.  It reads kJoin shares at a time, so that
// their latencies overlap.  With few splits (a.join_rows = 256 / (D / 4) rows in
// a block) it takes them all; with more than kJoinShared the block has one row,
// and its thread groups take turns over the splits and meet in LDS.  Either way in
// a fixed order.  (Whole call, shared out or not: 128 queries over 8192 keys, 13
// splits, 39.8 against 35.7 us; one query over 65536 keys, 32 splits, 60.3 against
// 63.1; one over 16384 keys of 256, 128 splits, 17.0 against 27.5.)
constexpr int kJoin = 8, kJoinShared = 2 * kJoin;
template <int D>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a) {
  constexpr int kGroups = 256 / (D / 4);
  __shared__ f32x4 s_o[kGroups][D / 4];
  __shared__ float2 s_ml[kGroups];
  const int grp = threadIdx.x / (D / 4), quad = threadIdx.x % (D / 4);
  const bool shared = a.join_rows == 1;
  const int64_t u = static_cast<int64_t>(blockIdx.x) * a.join_rows + (shared ? 0 : grp);
  int64_t q_row = u / a.q_heads;
  const int head = static_cast<int>(u - q_row * a.q_heads);
  TileWork w;
  int pos;
  if (a.token) {  // u counts the rows below max_q of each sequence
    const int seq = static_cast<int>(q_row / a.max_q);
    if (seq >= a.n_seqs) return;
    static_cast<SeqRange&>(w) = sequence(a, seq);
    pos = static_cast<int>(q_row - static_cast<int64_t>(seq) * a.max_q);
    q_row = w.q0 + pos;
  } else {  // u counts q's rows: the sequence is the last one that begins at or before it
    if (q_row >= a.q_rows) return;
    int lo = 0, hi = a.n_seqs;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (a.cu_q[mid] <= q_row) lo = mid; else hi = mid;
    }
    static_cast<SeqRange&>(w) = sequence(a, lo);
    pos = static_cast<int>(q_row) - w.q0;
  }
  if (pos < 0 || pos >= min(w.lq, a.max_q)) return;
  // The tile kernels cut by what the tile's last row sees.
  const int last = min((pos * a.group + head % a.group) / a.tile_rows * a.tile_rows + a.tile_rows,
                       min(w.lq, a.max_q) * a.group) - 1;
  const int splits = (max(last_key(a, w, last / a.group) + 1, 0) + a.chunk - 1) / a.chunk;
  if (splits <= 1) return;  // written by its tile
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
      part[j] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (i + j * step < splits) {
        const int64_t row = part_row(a, i + j * step, q_row, head);
        ml[j] = a.part_ml[row];
        part[j] = *reinterpret_cast<const f32x4*>(a.part_o + row * D + 4 * quad);
      }
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

struct Plan {
  bool token;          // the few-rows kernel
  int64_t tiles;       // row tiles x key heads
  int splits, chunk;
};

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Which kernel, and how many keys a block takes.  Everything here follows
// from the shape fields, as the workspace does.  The keys are split where the
// tiles alone do not fill the card.  Few rows, 8 key heads unless said (us):
//   blocks wanted: one a CU where a block's LDS leaves no room for a second
//     (head_dim 128: 32 x 1024 keys 24.3, with two 28.5; 256: 4 x 2048 keys 19.4,
//     22.1), two where it does (64: 16 x 4096 keys 25.8, with one 29.1);
//   a sequence of up to 4 units in one piece, without a join (4 x 512 keys 8.5, in
//     halves 11.2); a longer one in pieces of at least 2 (4 x 1024 keys 12.0; one
//     unit each 12.3, four 12.8, whole 13.0);
//   no piece above 16 units, so that sequences of different lengths end together
//     (64 x up to 8192 keys, head_dim 128: 236; 8 units 243, 32 units 249, whole
//     263; head_dim 256, 32 x up to 4096: 123; 8 units 129, 32 units 141), until
//     kRounds blocks a CU, which are even enough, and bound the workspace.
// Many rows: blocks wanted as above (head_dim 128: 288 tiles, 4 x 256 queries after
//     4096 keys 51, with one 67; 256: 66 tiles, 512 queries over 16384 keys, 16 heads
//     over 2, in 4 pieces 174, with two 191, in turn; 168 to 197 between sessions);
//     pieces of at least tiles / 16 key tiles, 4 to 16, as a join costs more the more
//     rows there are (32 row tiles, 2 x 64 queries, 2048 keys, 4:
//     13.2, 8: 15.8, 16: 21.4; 144, a prompt of 1024, 4: 17.8, 8: 16.9, 16: 17.9;
//     264, a prompt of 1024, 8: 35.4, 16: 28.2).
constexpr int kRounds = 64;

Plan make_plan(const moe_attn& d) {
  Plan p;
  const int64_t g = d.q_heads / d.kv_heads;
  const int64_t seqs = std::min<int64_t>(d.n_seqs, d.q_rows);
  const int64_t keys = std::max(d.max_kv, 1);
  p.token = d.max_q * g <= kRowsD;
  p.tiles = (p.token ? d.n_seqs : seqs + d.q_rows * g / kRowsP) * d.kv_heads;
  const int64_t tiles = std::max<int64_t>(p.tiles, 1);
  const int64_t unit = p.token ? kKeysD * (d.head_dim == 256 ? 2 : 4) : kKeysP;
  const int64_t want = d.head_dim > (p.token ? 64 : 128) ? kCus : 2 * kCus;
  const int64_t least = p.token ? (keys <= 4 * unit ? 4 : 2) * unit
                                : std::min(std::max(tiles / 16, int64_t{4}), int64_t{16}) * unit;
  const int64_t most = !p.token ? INT32_MAX
                                : std::max(16 * unit, ceil_div(keys, std::max(kRounds * kCus / tiles, int64_t{1})));
  int64_t chunk = ceil_div(keys, std::max<int64_t>(1, ceil_div(want, tiles)));
  chunk = std::min(std::max(chunk, least), most);
  chunk = ceil_div(chunk, unit) * unit;
  const int64_t splits = ceil_div(keys, chunk);
  p.chunk = static_cast<int>(std::min<int64_t>(chunk, INT32_MAX - unit));
  p.splits = static_cast<int>(splits);
  return p;
}

inline size_t align256(size_t v) { return (v + 255) & ~size_t{255}; }

size_t part_bytes(const moe_attn& d, const Plan& p) {
  if (p.splits <= 1) return 0;
  const size_t rows = static_cast<size_t>(p.splits) * d.q_rows * d.q_heads;
  return align256(rows * d.head_dim * 4) + align256(rows * 8);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int check_heads(const moe_heads& h) {
  if (!h.base) return MOE_EINVAL;
  if (h.row_stride <= 0 || h.head_stride <= 0) return MOE_EINVAL;
  if (!aligned16(h.base) || h.row_stride % 8 != 0 || h.head_stride % 8 != 0) return MOE_EALIGN;
  return MOE_OK;
}

// The shape fields, which the workspace depends on.
int check_shape(const moe_attn* a) {
  if (!a) return MOE_EINVAL;
  if (a->abi_version != MOE_ABI_VERSION) return MOE_ELAYOUT;
  if (a->n_seqs < 0 || a->q_rows < 0 || a->kv_rows < 0 || a->max_q < 0 || a->max_kv < 0) return MOE_EINVAL;
  if (a->head_dim != 64 && a->head_dim != 128 && a->head_dim != 256) return MOE_ESHAPE;
  if (a->kv_heads < 1 || a->q_heads < 1 || a->q_heads > 1024 || a->q_heads % a->kv_heads != 0) return MOE_ESHAPE;
  if (a->n_seqs > 65536 || a->q_rows > MOE_MAX_TOKENS) return MOE_ESHAPE;
  if (a->max_q > a->q_rows || a->max_kv > a->kv_rows) return MOE_EINVAL;
  const Plan p = make_plan(*a);
  // grid limits: 2^32 threads along x, 65535 blocks along y
  if (p.tiles > 0xffffff || p.splits > 65535) return MOE_ESHAPE;
  if (static_cast<int64_t>(a->q_rows) * a->q_heads > 0x3fffffff) return MOE_ESHAPE;
  return MOE_OK;
}

template <int D>
void launch(const AttnArgs& a, const Plan& p, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(p.tiles), static_cast<unsigned>(p.splits));
  if (p.token)
    attn_token_kernel<D><<<grid, 64 * decode_waves<D>(), 0, s>>>(a);
  else
    attn_rows_kernel<D><<<grid, 256, 0, s>>>(a);
  if (p.splits > 1) {
    const int64_t rows = (p.token ? static_cast<int64_t>(a.n_seqs) * a.max_q : a.q_rows) * a.q_heads;
    attn_join_kernel<D><<<static_cast<unsigned>(ceil_div(rows, a.join_rows)), 256, 0, s>>>(a);
  }
}

}  // namespace
}  // namespace moe

extern "C" {

int moe_attn_init(moe_attn* a, const uint16_t* q, const uint16_t* k, const uint16_t* v, uint16_t* out,
                  const int32_t* cu_q, int32_t n_seqs, int32_t q_rows, int32_t kv_rows, int32_t q_heads,
                  int32_t kv_heads, int32_t head_dim) {
  if (!a || !q || !k || !v || !out || !cu_q) return MOE_EINVAL;
  *a = moe_attn{};
  a->abi_version = MOE_ABI_VERSION;
  a->head_dim = head_dim;
  a->q_heads = q_heads;
  a->kv_heads = kv_heads;
  a->n_seqs = n_seqs;
  a->q_rows = a->max_q = q_rows;
  a->kv_rows = a->max_kv = kv_rows;
  a->causal = 1;
  a->scale = head_dim > 0 ? 1.0f / sqrtf(static_cast<float>(head_dim)) : 0.f;
  const int64_t qs = static_cast<int64_t>(q_heads) * head_dim, ks = static_cast<int64_t>(kv_heads) * head_dim;
  a->q = moe_heads{const_cast<uint16_t*>(q), qs, head_dim};
  a->k = moe_heads{const_cast<uint16_t*>(k), ks, head_dim};
  a->v = moe_heads{const_cast<uint16_t*>(v), ks, head_dim};
  a->out = moe_heads{out, qs, head_dim};
  a->cu_q = cu_q;
  return MOE_OK;
}

size_t moe_attention_workspace_size(const moe_attn* a) {
  if (moe::check_shape(a) != MOE_OK || a->n_seqs == 0 || a->q_rows == 0 || a->max_q == 0) return 0;
  return moe::part_bytes(*a, moe::make_plan(*a));
}

int moe_attention(const moe_attn* a, void* ws, size_t ws_bytes, void* stream) {
  int st = moe::check_shape(a);
  if (st != MOE_OK) return st;
  if ((a->causal != 0 && a->causal != 1) || a->reserved != 0) return MOE_EINVAL;
  if (!(a->scale > 0.f && a->scale <= 0x1p127f)) return MOE_EINVAL;  // scale * log2(e) is finite
  if ((a->kv_start == nullptr) != (a->kv_len == nullptr)) return MOE_EINVAL;
  if (a->n_seqs == 0 || a->q_rows == 0 || a->max_q == 0) return MOE_OK;
  if (!a->cu_q) return MOE_EINVAL;
  for (const moe_heads* h : {&a->q, &a->out})
    if ((st = moe::check_heads(*h)) != MOE_OK) return st;
  if (a->kv_rows > 0)
    for (const moe_heads* h : {&a->k, &a->v}) {
      if ((st = moe::check_heads(*h)) != MOE_OK) return st;
      if (h->row_stride > (1 << 23)) return MOE_ESHAPE;
    }
  const moe::Plan p = moe::make_plan(*a);
  const size_t need = moe::part_bytes(*a, p);
  if (need) {
    if (!ws) return MOE_EINVAL;
    if (reinterpret_cast<uintptr_t>(ws) & 255) return MOE_EALIGN;
    if (ws_bytes < need) return MOE_EWORKSPACE;
  }
  moe::AttnArgs k;
  k.q = a->q, k.k = a->k, k.v = a->v, k.out = a->out;
  k.cu_q = a->cu_q, k.kv_start = a->kv_start, k.kv_len = a->kv_len;
  k.lse = a->lse;
  k.part_o = static_cast<float*>(ws);
  const size_t rows = static_cast<size_t>(p.splits) * a->q_rows * a->q_heads;
  k.part_ml =
      need ? reinterpret_cast<float2*>(static_cast<char*>(ws) + moe::align256(rows * a->head_dim * 4)) : nullptr;
  k.n_seqs = a->n_seqs, k.q_rows = a->q_rows, k.kv_rows = a->kv_rows;
  k.q_heads = a->q_heads, k.kv_heads = a->kv_heads, k.group = a->q_heads / a->kv_heads;
  k.max_q = a->max_q, k.max_kv = a->max_kv, k.causal = a->causal;
  k.chunk = p.chunk, k.tile_rows = p.token ? moe::kRowsD : moe::kRowsP;
  k.token = p.token;
  k.join_rows = p.splits > moe::kJoinShared ? 1 : 256 / (a->head_dim / 4);
  k.scale = a->scale;
  k.c = a->scale * 1.44269504088896340736f;  // log2(e)
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  switch (a->head_dim) {
    case 64: moe::launch<64>(k, p, s); break;
    case 128: moe::launch<128>(k, p, s); break;
    default: moe::launch<256>(k, p, s); break;
  }
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_EHIP;
}

}  // extern "C"
