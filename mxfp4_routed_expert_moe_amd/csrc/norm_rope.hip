// RMS norm and rotary position of every query and key head, in one pass
// (include/moe_attention.h, moe_qk_norm_rope).
//
// A head of D elements is held by a group of L >= D / 8 lanes (L = 8 .. 64, a
// power of two), eight consecutive elements each: one 16-byte load, a sum of
// squares over the group by lane exchanges, one 16-byte store.  A rotated pair
// lies either inside a lane (interleaved) or in two lanes rot_dim / 16 apart,
// which exchange their inputs as stored (four words rather than eight floats).
// Norm weight, cosine and sine do not depend on the head, so with a lane's own
// inputs x and its partners' y an output is f (x A + y B), f = 1 / sqrt(mean(x^2) +
// eps), and A and B are built once for the HP heads of one token that a group
// takes: A = w c, B = -+ w' s.
//
// Bound by HBM: 16384 tokens of 40 heads of 128 are 344 MB in 79 us = 4.4 TB/s (a large
// copy moves 5.2 TB/s).  Four heads per group 79 us, two 83, eight 87; the stores past
// the caches 79 against 85, timed by the operator alone (with attention behind it,
// which reads q and k again, not compared).  A call of a few tokens is one launch,
// 2.5 us.
#include <math.h>

#include "../../include/moe_attention.h"
#include "moe_internal.h"

namespace moe {

namespace {

struct NormArgs {
  moe_heads q, k, q_out, k_out;
  const float *qw, *kw, *cs;
  const int32_t* pos;
  unsigned T, chunks;  // chunks of heads per token
  int q_heads, heads;  // heads = q_heads + k_heads
  int D, P, R, off;
  float eps, inv_d;
};

__device__ __forceinline__ void unpack8(u32x4 w, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
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

// The sum over a group of L lanes, in every lane of it.
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
  if (L >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return v;
}

// Unit u = (token, chunk of HP heads) per group of L lanes.
template <int L, int HP, bool INTER>
__global__ __launch_bounds__(256) void norm_rope_kernel(NormArgs a) {
  const unsigned u = blockIdx.x * (256 / L) + threadIdx.x / L;
  const unsigned token = u / a.chunks;
  const bool live = token < a.T;
  const unsigned t = live ? token : 0;
  const int h0 = static_cast<int>(u - token * a.chunks) * HP;
  const int l = threadIdx.x % L, e0 = 8 * l;
  const bool in = live && e0 < a.D;

  // all the loads of the heads first
  u32x4 raw[HP];
#pragma unroll
  for (int i = 0; i < HP; ++i) {
    const int h = h0 + i;
    raw[i] = u32x4{0, 0, 0, 0};
    if (in && h < a.heads) {
      const bool is_q = h < a.q_heads;
      const moe_heads& s = is_q ? a.q : a.k;
      raw[i] = ld16(s.base + t * s.row_stride + (is_q ? h : h - a.q_heads) * s.head_stride + e0);
    }
  }

  const int r0 = e0 - a.off;  // place in the rotated range
  const bool rot = in && r0 >= 0 && r0 < a.R;
  const int half = a.R >> 1;
  const bool first = r0 < half;  // of the two halves
  const int step = INTER ? 0 : rot ? (first ? half : -half) : 0;  // to the partners
  const int mate = 4 * (static_cast<int>(threadIdx.x & 63) + step / 8);
  // the angles of the lane's elements: cosine, and sine with the sign its product takes
  float c[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = 1.f, s[i] = 0.f;
  if (rot) {
    const int p = a.pos[t];
    const bool ok = p >= 0 && p < a.P;
    const float* row = a.cs + static_cast<int64_t>(ok ? p : 0) * a.R + (INTER ? r0 / 2 : first ? r0 : r0 - half);
    if (a.P > 0) {
      load8<INTER>(row, c);
      load8<INTER>(row + half, s);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (INTER ? i % 2 == 0 : first) s[i] = -s[i];
      if (!ok) c[i] = s[i] = __builtin_nanf("");
    }
  }

  float A[8], B[8];
#pragma unroll
  for (int i = 0; i < HP; ++i) {
    const int h = h0 + i;
    if (HP > 1 && !__any(h < a.heads)) break;
    const bool is_q = h < a.q_heads;
    if (i == 0 || h == a.q_heads) {
      const float* wp = is_q ? a.qw : a.kw;
#pragma unroll
      for (int j = 0; j < 8; ++j) A[j] = B[j] = 1.f;
      if (wp && in) {
        load8<false>(wp + e0, A);
        load8<false>(wp + e0 + step, B);
      }
      if (INTER) {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const float v = B[j];
          B[j] = B[j + 1], B[j + 1] = v;
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) A[j] *= c[j], B[j] *= s[j];
    }
    float x[8], y[8];
    unpack8(raw[i], x);
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(x[j], x[j], sum);
    const float f = rsqrtf(__builtin_fmaf(group_sum<L>(sum), a.inv_d, a.eps));
    if (INTER) {
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = x[j ^ 1];
      // An infinite norm: an element that is not rotated must not meet a neighbour's
      // infinity, not even times its B of 0.  (Chosen always, 2049 x 65 heads 18.6 us
      // against 14.1.)
      if (__any(f == 0.f)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = rot ? y[j] : x[j];
      }
    } else {
      u32x4 other;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        other[j] = static_cast<unsigned>(__builtin_amdgcn_ds_bpermute(mate, static_cast<int>(raw[i][j])));
      unpack8(other, y);
    }
    if (in && h < a.heads) {
      const moe_heads& o = is_q ? a.q_out : a.k_out;
      u32x4 v;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // an element that is not rotated has B = 0 and its own input as y
        const float p0 = f * __builtin_fmaf(x[2 * j], A[2 * j], y[2 * j] * B[2 * j]);
        const float p1 = f * __builtin_fmaf(x[2 * j + 1], A[2 * j + 1], y[2 * j + 1] * B[2 * j + 1]);
        v[j] = float_to_bf16_bits(p0) | static_cast<uint32_t>(float_to_bf16_bits(p1)) << 16;
      }
      u32x4* to = reinterpret_cast<u32x4*>(o.base + t * o.row_stride + (is_q ? h : h - a.q_heads) * o.head_stride + e0);
      if (HP > 1)
        __builtin_nontemporal_store(v, to);
      else
        *to = v;
    }
  }
}

// Lanes of work from which a group takes four heads: below, one head each
// spreads the work over more of the card (40 heads of 128: 512 tokens, 2^18.3
// lanes, 5.3 us against 6.3 with four; 1024 tokens, 2^19.3 lanes, 9.4 against 7.2).
constexpr int64_t kManyLanes = int64_t{1} << 19;

template <int L, bool INTER>
void launch(NormArgs a, hipStream_t s) {
  constexpr int kMany = 4;
  const bool many = static_cast<int64_t>(a.T) * a.heads * L >= kManyLanes;
  a.chunks = many ? (a.heads + kMany - 1) / kMany : a.heads;
  const unsigned blocks = (static_cast<unsigned>(a.T) * a.chunks + 256 / L - 1) / (256 / L);
  if (many)
    norm_rope_kernel<L, kMany, INTER><<<blocks, 256, 0, s>>>(a);
  else
    norm_rope_kernel<L, 1, INTER><<<blocks, 256, 0, s>>>(a);
}

template <bool INTER>
void launch_for(const NormArgs& a, hipStream_t s) {
  if (a.D <= 64)
    launch<8, INTER>(a, s);
  else if (a.D <= 128)
    launch<16, INTER>(a, s);
  else if (a.D <= 256)
    launch<32, INTER>(a, s);
  else
    launch<64, INTER>(a, s);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int check_heads(const moe_heads* h) {
  if (!h || !h->base || h->row_stride <= 0 || h->head_stride <= 0) return MOE_EINVAL;
  if (!aligned16(h->base) || h->row_stride % 8 != 0 || h->head_stride % 8 != 0) return MOE_EALIGN;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" int moe_qk_norm_rope(const moe_heads* q, int32_t q_heads, const moe_heads* k, int32_t k_heads, int32_t T,
                                int32_t head_dim, const float* q_weight, const float* k_weight, float eps,
                                const int32_t* positions, const float* cos_sin, int32_t n_positions, int32_t rot_dim,
                                int32_t rot_offset, int32_t interleaved, const moe_heads* q_out, const moe_heads* k_out,
                                void* stream) {
  if (T < 0 || q_heads < 0 || k_heads < 0 || rot_dim < 0 || rot_offset < 0 || n_positions < 0) return MOE_EINVAL;
  if (T > MOE_MAX_TOKENS || q_heads < 1 || q_heads > 1024 || k_heads > 1024 - q_heads) return MOE_ESHAPE;
  if (static_cast<int64_t>(T) * (q_heads + k_heads) >= (1 << 28)) return MOE_ESHAPE;  // 2^32 threads
  if (head_dim < 8 || head_dim > 512 || head_dim % 8 != 0) return MOE_ESHAPE;
  // heads wider than 256 take 64 lanes per four heads: again 2^32 threads
  if (head_dim > 256 && static_cast<int64_t>(T) * ((q_heads + k_heads + 3) / 4 * 4) >= (1 << 28)) return MOE_ESHAPE;
  if (rot_dim % 16 != 0 || rot_offset % 8 != 0 || rot_dim > head_dim || rot_offset > head_dim - rot_dim)
    return MOE_ESHAPE;
  if (!(eps >= 0.f) || (interleaved != 0 && interleaved != 1)) return MOE_EINVAL;
  if (T == 0) return MOE_OK;
  int st;
  if ((st = moe::check_heads(q)) != MOE_OK || (st = moe::check_heads(q_out)) != MOE_OK) return st;
  if (k_heads > 0 && ((st = moe::check_heads(k)) != MOE_OK || (st = moe::check_heads(k_out)) != MOE_OK)) return st;
  if (rot_dim > 0 && (!positions || !cos_sin)) return MOE_EINVAL;
  if (rot_dim > 0 && !moe::aligned16(cos_sin)) return MOE_EALIGN;
  if (!moe::aligned16(q_weight) || !moe::aligned16(k_weight)) return MOE_EALIGN;
  moe::NormArgs a;
  a.q = *q, a.q_out = *q_out;
  a.k = k_heads ? *k : moe_heads{}, a.k_out = k_heads ? *k_out : moe_heads{};
  a.qw = q_weight, a.kw = k_weight, a.cs = cos_sin, a.pos = positions;
  a.T = static_cast<unsigned>(T), a.chunks = 0;
  a.q_heads = q_heads, a.heads = q_heads + k_heads;
  a.D = head_dim, a.P = n_positions, a.R = rot_dim, a.off = rot_offset;
  a.eps = eps, a.inv_d = 1.f / static_cast<float>(head_dim);
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (interleaved)
    moe::launch_for<true>(a, s);
  else
    moe::launch_for<false>(a, s);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_EHIP;
}
