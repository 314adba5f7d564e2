// Keys and values into the pages of a cache, with norm and rotation on the way
// (include/moe_paged.h, moe_paged_append).
//
// A block does one of two things.  The first blocks take runs: the rows that one
// sequence brings to one page, for one key head.  A group of L = D / 8 lanes holds a
// head of one row, eight elements a lane, so a block does 256 / L rows at a time; norm and
// rotation are those of a head alone (a sum of squares over the group, the rotation's
// partner from the lane that holds it).  The block that writes a page's rows also sees
// all that the call brings to the page, so the bounds need no atomics: every lane keeps the
// minimum and maximum of its columns, the groups meet in LDS, and what the bounds were joins
// unless the run begins the page.  The other blocks take heads of q, HP of a token
// per group.
//
// Bound by HBM for prompts: 16384 tokens of 32 query and 8 key heads of 128 are 412 MB in 82 us =
// 5.0 TB/s (a large copy moves 5.14); streaming stores for q 82 against 87, a second row in
// flight per group 86 against 87, four 95 (fewer waves).  By latency for single tokens: 4.4 us in
// a graph (5.6 with the page looked up before the first loads and every row's sequence searched for).
#include <algorithm>

#include "paged_internal.h"

namespace moe {

namespace {

struct AppendArgs {
  PagedSeqs s;
  moe_heads q, q_out, k, v;
  moe_pages kp, vp;
  uint16_t* bounds;
  const float *qw, *kw, *cs;
  const int32_t* pos;
  int q_heads, kv_heads, P, R, off, norm;
  unsigned run_blocks, chunks;  // blocks that take runs; chunks of q heads per token
  float eps;
};

constexpr float kInf = __builtin_huge_valf();

__device__ __forceinline__ void unpack8(u32x4 w, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return float_to_bf16_bits(a) | static_cast<uint32_t>(float_to_bf16_bits(b)) << 16;
}

// Eight values, or four of them twice each.
template <bool TWICE>
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p);
  if (TWICE) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = a[i / 2];
  } else {
    const f32x4 b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = a[i], f[4 + i] = b[i];
  }
}

// The sum over a group of L = 8, 16 or 32 lanes, in every lane of it.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 15, 15, true));
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
  v = dpp_add<0xb1>(v);   // quad_perm 1 0 3 2
  v = dpp_add<0x4e>(v);   // quad_perm 2 3 0 1
  v = dpp_add<0x141>(v);  // mirror within 8
  if (L >= 16) v = dpp_add<0x140>(v);  // mirror within 16
  if (L >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return v;
}

// What a lane's eight elements take of the rotation: c and s (with the sign that its
// product takes) for a token at rotary position p, and where their partners are.
template <int L, bool INTER>
struct Turn {
  float c[8], s[8];
  int step, mate;
  bool rot;
  __device__ __forceinline__ void place(const AppendArgs& a) {
    const int e0 = 8 * (threadIdx.x % L), r0 = e0 - a.off, half = a.R >> 1;
    rot = r0 >= 0 && r0 < a.R;
    step = INTER || !rot ? 0 : r0 < half ? half : -half;
    mate = 4 * (static_cast<int>(threadIdx.x & 63) + step / 8);
  }
  __device__ __forceinline__ void load(const AppendArgs& a, int p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = 1.f, s[i] = 0.f;
    if (!rot) return;
    const int r0 = 8 * static_cast<int>(threadIdx.x % L) - a.off, half = a.R >> 1;
    const bool first = r0 < half, ok = p >= 0 && p < a.P;
    if (ok) {
      const float* row = a.cs + static_cast<int64_t>(p) * a.R + (INTER ? r0 / 2 : first ? r0 : r0 - half);
      load8<INTER>(row, c);
      load8<INTER>(row + half, s);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (INTER ? i % 2 == 0 : first) s[i] = -s[i];
      if (!ok) c[i] = s[i] = __builtin_nanf("");
    }
  }
};

// The norm weights of a lane's elements and of their partners.
struct Weights {
  float own[8], mate[8];
};
template <bool INTER>
__device__ __forceinline__ Weights load_weights(const float* w, int e0, int step) {
  Weights r;
#pragma unroll
  for (int j = 0; j < 8; ++j) r.own[j] = r.mate[j] = 1.f;
  if (w) {
    load8<false>(w + e0, r.own);
    load8<false>(w + e0 + step, r.mate);
  }
  if (INTER) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const float v = r.mate[j];
      r.mate[j] = r.mate[j + 1], r.mate[j + 1] = v;
    }
  }
  return r;
}

// A head, eight elements a lane, normed and rotated, as bf16.
template <int L, bool INTER>
__device__ __forceinline__ u32x4 norm_turn(const AppendArgs& a, u32x4 raw, const Weights& w, const Turn<L, INTER>& t) {
  float x[8], y[8];
  unpack8(raw, x);
  float f = 1.f;
  if (a.norm) {
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(x[j], x[j], sum);
    f = rsqrtf(__builtin_fmaf(group_sum<L>(sum), 1.f / (8 * L), a.eps));
  }
  if (INTER) {
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = x[j ^ 1];
  } else {
    u32x4 other;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      other[j] = static_cast<unsigned>(__builtin_amdgcn_ds_bpermute(t.mate, static_cast<int>(raw[j])));
    unpack8(other, y);
  }
  u32x4 v;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float p[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = 2 * j + e;
      // an element that is not rotated must not meet another one's infinity, not even times 0
      const float turned = __builtin_fmaf(x[i], w.own[i] * t.c[i], y[i] * (w.mate[i] * t.s[i]));
      p[e] = f * (t.rot ? turned : x[i] * w.own[i]);
    }
    v[j] = pack2(p[0], p[1]);
  }
  return v;
}

// A run: rows row0 .. row0 + rows - 1 of k and v go to slots slot0 .. of a page.
struct Run {
  int row0, rows, pos0, seq;
};

// Run u over all sequences (each sequence's runs in a row), 64 sequences at a time.
__device__ bool find_run(const PagedSeqs& s, int u, Run& r) {
  const int lane = threadIdx.x & 63;
  for (int base = 0; base < s.n_seqs; base += 64) {
    int q0 = 0, lq = 0, first = 0, runs = 0;  // rows that have a position of the table, the first one's position
    if (base + lane < s.n_seqs) {
      const PagedRange x = paged_range(s.cu_q, s.kv_len, base + lane, s.q_rows, s.capacity, 0, 0, 0, s.shift);
      const int skip = min(max(-x.diag, 0), x.lq);
      q0 = x.q0 + skip, first = x.diag + skip;
      lq = min(x.lq - skip, max(s.capacity - first, 0));
      runs = lq > 0 ? ((first + lq - 1) >> s.shift) - (first >> s.shift) + 1 : 0;
    }
    const int incl = wave_prefix(runs);
    const uint64_t past = __ballot(incl > u);
    if (past) {
      const int src = __ffsll(static_cast<unsigned long long>(past)) - 1;
      q0 = lane_value(q0, src), lq = lane_value(lq, src), first = lane_value(first, src);
      const int i = u - (lane_value(incl, src) - lane_value(runs, src));
      // run i: positions of the sequence's i-th page
      const int begin = i == 0 ? first : ((first >> s.shift) + i) << s.shift;
      const int end = min(first + lq, ((first >> s.shift) + i + 1) << s.shift);
      r.seq = __builtin_amdgcn_readfirstlane(base + src);
      r.row0 = __builtin_amdgcn_readfirstlane(q0 + begin - first);
      r.rows = __builtin_amdgcn_readfirstlane(end - begin);
      r.pos0 = __builtin_amdgcn_readfirstlane(begin);
      return true;
    }
    u -= lane_value(incl, 63);
  }
  return false;
}

template <int L, bool INTER>
__device__ void append_run(const AppendArgs& a) {
  constexpr int kGroups = 256 / L, D = 8 * L;
  __shared__ float s_low[kGroups][D], s_high[kGroups][D];
  const int head = blockIdx.x % a.kv_heads;
  Run r;
  if (!find_run(a.s, blockIdx.x / a.kv_heads, r)) return;
  const int page = a.s.table[r.seq * a.s.table_stride + (r.pos0 >> a.s.shift)];
  const int slot0 = r.pos0 & ((1 << a.s.shift) - 1);
  const int grp = threadIdx.x / L, e0 = 8 * (threadIdx.x % L);
  const uint16_t* k = a.k.base + r.row0 * a.k.row_stride + head * a.k.head_stride + e0;
  const uint16_t* v = a.v.base + r.row0 * a.v.row_stride + head * a.v.head_stride + e0;
  // a group's first row is loaded before the page is known
  u32x4 raw, val;
  int pos = 0;
  auto load = [&](int i) {
    raw = ld16(k + i * a.k.row_stride);
    val = ld16(v + i * a.v.row_stride);
    pos = a.pos ? a.pos[r.row0 + i] : r.pos0 + i;
  };
  if (grp < r.rows) load(grp);
  Turn<L, INTER> t;
  t.place(a);
  const Weights w = load_weights<INTER>(a.kw, e0, t.step);
  if (page < 0 || page >= a.s.n_pages) return;
  uint16_t* ko = a.kp.base + page * a.kp.page_stride + slot0 * a.kp.row_stride + head * a.kp.head_stride + e0;
  uint16_t* vo = a.vp.base + page * a.vp.page_stride + slot0 * a.vp.row_stride + head * a.vp.head_stride + e0;
  uint16_t* const bound = a.bounds ? a.bounds + (static_cast<int64_t>(page) * 2 * a.kv_heads + head) * D : nullptr;
  const int64_t to_high = static_cast<int64_t>(a.kv_heads) * D;
  float low[8], high[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) low[j] = kInf, high[j] = -kInf;
  // Lanes exchange inside a group, and a group's lanes run the same rows.
  for (int i = grp; i < r.rows; i += kGroups) {
    if (i != grp) load(i);
    t.load(a, pos);
    const u32x4 out = norm_turn<L, INTER>(a, raw, w, t);
    *reinterpret_cast<u32x4*>(ko + i * a.kp.row_stride) = out;
    *reinterpret_cast<u32x4*>(vo + i * a.vp.row_stride) = val;
    float x[8];
    unpack8(out, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) low[e] = fminf(low[e], x[e]), high[e] = fmaxf(high[e], x[e]);
  }
  if (!bound) return;
  if (r.rows > 1) {  // the groups meet
#pragma unroll
    for (int j = 0; j < 8; ++j) s_low[grp][e0 + j] = low[j], s_high[grp][e0 + j] = high[j];
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * D; c += 256) {
      const bool is_high = c >= D;
      const int d = is_high ? c - D : c;
      float m = is_high ? s_high[0][d] : s_low[0][d];
      for (int g = 1; g < min(kGroups, r.rows); ++g) m = is_high ? fmaxf(m, s_high[g][d]) : fminf(m, s_low[g][d]);
      uint16_t* to = bound + (is_high ? to_high : 0) + d;
      if (slot0 > 0) {
        const float old = bf16_bits_to_float(*to);
        m = is_high ? fmaxf(m, old) : fminf(m, old);
      }
      *to = float_to_bf16_bits(m);
    }
  } else if (grp == 0) {
    u32x4* to_l = reinterpret_cast<u32x4*>(bound + e0);
    u32x4* to_h = reinterpret_cast<u32x4*>(bound + to_high + e0);
    if (slot0 > 0) {
      float x[8];
      unpack8(*to_l, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) low[j] = fminf(low[j], x[j]);
      unpack8(*to_h, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) high[j] = fmaxf(high[j], x[j]);
    }
    u32x4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = pack2(low[2 * j], low[2 * j + 1]);
    *to_l = o;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = pack2(high[2 * j], high[2 * j + 1]);
    *to_h = o;
  }
}

// The sequence of row t: the last one that begins at or before it (-1: none), and
// its position.
__device__ __forceinline__ bool find_row(const PagedSeqs& s, int t, int& pos) {
  int lo = min(t, s.n_seqs - 1), hi = s.n_seqs;  // often they have a row each
  PagedRange x = paged_range(s.cu_q, s.kv_len, lo, s.q_rows, s.capacity, 0, 0, 0, s.shift);
  if (t < x.q0 || (lo + 1 < hi && t >= x.q0 + x.lq)) {
    lo = 0;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (s.cu_q[mid] <= t) lo = mid; else hi = mid;
    }
    x = paged_range(s.cu_q, s.kv_len, lo, s.q_rows, s.capacity, 0, 0, 0, s.shift);
  }
  pos = t - x.q0 + x.diag;
  return t >= x.q0 && t < x.q0 + x.lq;
}

// Unit u = (row, chunk of HP heads) per group of L lanes.
template <int L, int HP, bool INTER>
__device__ void append_q(const AppendArgs& a) {
  const unsigned u = (blockIdx.x - a.run_blocks) * (256 / L) + threadIdx.x / L;
  const unsigned t = u / a.chunks;
  const int e0 = 8 * (threadIdx.x % L);
  if (t >= static_cast<unsigned>(a.s.q_rows)) return;
  const int h0 = static_cast<int>(u - t * a.chunks) * HP;
  u32x4 raw[HP];
#pragma unroll
  for (int i = 0; i < HP; ++i)
    if (h0 + i < a.q_heads) raw[i] = ld16(a.q.base + t * a.q.row_stride + (h0 + i) * a.q.head_stride + e0);
  int pos;
  if (!find_row(a.s, static_cast<int>(t), pos)) return;
  Turn<L, INTER> turn;
  turn.place(a);
  const Weights w = load_weights<INTER>(a.qw, e0, turn.step);
  turn.load(a, a.pos ? a.pos[t] : pos);
#pragma unroll
  for (int i = 0; i < HP; ++i) {
    if (h0 + i >= a.q_heads) break;
    const u32x4 v = norm_turn<L, INTER>(a, raw[i], w, turn);
    u32x4* to = reinterpret_cast<u32x4*>(a.q_out.base + t * a.q_out.row_stride + (h0 + i) * a.q_out.head_stride + e0);
    if (HP > 1)
      __builtin_nontemporal_store(v, to);
    else
      *to = v;
  }
}

template <int L, int HP, bool INTER>
__global__ __launch_bounds__(256) void append_kernel(AppendArgs a) {
  if (blockIdx.x < a.run_blocks)
    append_run<L, INTER>(a);
  else
    append_q<L, HP, INTER>(a);
}

// Lanes of work from which a group takes four heads of q: below, one head each spreads
// the work over more of the card (16384 tokens of 32 heads with one 159 us, with four 87).
constexpr int64_t kManyLanes = int64_t{1} << 19;

// Runs of a call: a sequence of n rows touches at most (n - 2) / page_size + 2 pages, and
// no more than n.
int64_t run_bound(int64_t rows, int64_t seqs, int shift) {
  return std::min(rows, (rows >> shift) + 2 * std::min(seqs, rows));
}
// Blocks that take q, with `per` heads to a group.
int64_t q_blocks(int64_t rows, int heads, int D, int per) {
  const int64_t groups = rows * ((heads + per - 1) / per), in_block = 2048 / D;
  return (groups + in_block - 1) / in_block;
}

template <int L, bool INTER>
void launch(AppendArgs a, hipStream_t s) {
  const int64_t T = a.s.q_rows;
  const bool many = T * a.q_heads * L >= kManyLanes;
  const int per = many ? 4 : 1;
  a.chunks = static_cast<unsigned>(std::max((a.q_heads + per - 1) / per, 1));
  a.run_blocks = static_cast<unsigned>(run_bound(T, a.s.n_seqs, a.s.shift) * a.kv_heads);
  const unsigned blocks = a.run_blocks + static_cast<unsigned>(q_blocks(T, a.q_heads, 8 * L, per));
  if (many)
    append_kernel<L, 4, INTER><<<blocks, 256, 0, s>>>(a);
  else
    append_kernel<L, 1, INTER><<<blocks, 256, 0, s>>>(a);
}

template <bool INTER>
void launch_for(const AppendArgs& a, int D, hipStream_t s) {
  if (D == 64)
    launch<8, INTER>(a, s);
  else if (D == 128)
    launch<16, INTER>(a, s);
  else
    launch<32, INTER>(a, s);
}

}  // namespace
}  // namespace moe

extern "C" int moe_paged_append(const moe_append* a, void* stream) {
  if (!a) return MOE_EINVAL;
  int st = moe::check_paged_shape(a->p, true);
  if (st != MOE_OK) return st;
  const moe_paged& p = a->p;
  const int shift = __builtin_ctz(static_cast<unsigned>(p.page_size));
  if (moe::run_bound(p.q_rows, p.n_seqs, shift) * p.kv_heads + moe::q_blocks(p.q_rows, p.q_heads, p.head_dim, 1) > 0xffffff)
    return MOE_ESHAPE;  // 2^32 threads
  if (a->rot_dim < 0 || a->rot_offset < 0 || a->n_positions < 0) return MOE_EINVAL;
  if (a->rot_dim % 16 != 0 || a->rot_offset % 8 != 0 || a->rot_dim > p.head_dim ||
      a->rot_offset > p.head_dim - a->rot_dim)
    return MOE_ESHAPE;
  if (!(a->eps >= 0.f) || (a->norm != 0 && a->norm != 1) || (a->interleaved != 0 && a->interleaved != 1))
    return MOE_EINVAL;
  if (!a->norm && (a->q_weight || a->k_weight)) return MOE_EINVAL;
  if (p.n_seqs == 0 || p.q_rows == 0) return MOE_OK;
  if ((st = moe::check_paged_arrays(p)) != MOE_OK) return st;
  for (const moe_heads* h : {&a->k, &a->v})
    if ((st = moe::check_paged_heads(*h)) != MOE_OK) return st;
  if (p.q_heads > 0)
    for (const moe_heads* h : {&a->q, &a->q_out})
      if ((st = moe::check_paged_heads(*h)) != MOE_OK) return st;
  if (p.n_pages > 0)
    for (const moe_pages* h : {&a->k_pages, &a->v_pages})
      if ((st = moe::check_pages(*h)) != MOE_OK) return st;
  if (a->rot_dim > 0 && !a->cos_sin) return MOE_EINVAL;
  if (!moe::paged_aligned16(a->cos_sin) || !moe::paged_aligned16(a->q_weight) || !moe::paged_aligned16(a->k_weight) ||
      !moe::paged_aligned16(a->bounds))
    return MOE_EALIGN;
  moe::AppendArgs k;
  k.s = moe::paged_seqs(p);
  k.q = a->q, k.q_out = a->q_out, k.k = a->k, k.v = a->v, k.kp = a->k_pages, k.vp = a->v_pages;
  k.bounds = a->bounds, k.qw = a->q_weight, k.kw = a->k_weight, k.cs = a->cos_sin, k.pos = a->positions;
  k.q_heads = p.q_heads, k.kv_heads = p.kv_heads;
  k.P = a->n_positions, k.R = a->rot_dim, k.off = a->rot_offset, k.norm = a->norm, k.eps = a->eps;
  k.run_blocks = k.chunks = 0;
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (a->interleaved)
    moe::launch_for<true>(k, p.head_dim, s);
  else
    moe::launch_for<false>(k, p.head_dim, s);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_EHIP;
}
