// RMS norm and rotary position of every query and key head, in one pass
// (include/moe_attention.h, moe_qk_norm_rope).
//
// A head of D elements is held by a group of L >= D / 8 lanes (L = 8 .. 64, a
// power of two), eight consecutive elements each: one 16-byte load, a sum of
// squares over the group by lane exchanges, one 16-byte store.  A rotated pair
// lies either inside a lane (interleaved) or in two lanes rot_dim / 16 apart,
// which exchange their inputs as stored (four words rather than eight floats: the
// partner's norm factor is the same, and its weights are loaded beside the own
// ones).  A block keeps to one token, so its cosines and sines are loaded
// once and serve all of the heads that a group takes in turn.
#include <math.h>

#include "../../include/moe_attention.h"
#include "moe_internal.h"

namespace moe {

namespace {

struct NormArgs {
  moe_heads q, k, q_out, k_out;
  const float *qw, *kw, *cs;
  const int32_t* pos;
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

__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = a[i], f[4 + i] = b[i];
}

// grid (T, chunks of 256 / L * HP heads); group g of a block takes heads g,
// g + 256 / L, ... of its chunk.
template <int L, int HP, bool INTER>
__global__ __launch_bounds__(256) void norm_rope_kernel(NormArgs a) {
  constexpr int kGroups = 256 / L;
  const int t = blockIdx.x;
  const int l = threadIdx.x % L, g = threadIdx.x / L;
  const int e0 = 8 * l;
  const bool in = e0 < a.D;
  const int h0 = blockIdx.y * (kGroups * HP) + g;

  // all the loads of the heads first
  u32x4 raw[HP];
#pragma unroll
  for (int i = 0; i < HP; ++i) {
    const int h = h0 + i * kGroups;
    raw[i] = u32x4{0, 0, 0, 0};
    if (in && h < a.heads) {
      const bool is_q = h < a.q_heads;
      const moe_heads& s = is_q ? a.q : a.k;
      raw[i] = ld16(s.base + t * s.row_stride + (is_q ? h : h - a.q_heads) * s.head_stride + e0);
    }
  }

  const int r0 = e0 - a.off;                          // place in the rotated range
  const bool rot = in && r0 >= 0 && r0 < a.R;
  const int half = a.R >> 1;
  const bool first = r0 < half;                       // of the two halves
  const int mate = INTER ? l : l + (first ? half : -half) / 8;  // lane in the group that holds the partners
  float c[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = 1.f, s[i] = 0.f;
  if (rot) {
    const int p = a.pos[t];
    if (p < 0 || p >= a.P) {
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = s[i] = __builtin_nanf("");
    } else {
      const float* row = a.cs + static_cast<int64_t>(p) * a.R;
      if (INTER) {
        const f32x4 cv = *reinterpret_cast<const f32x4*>(row + r0 / 2), sv = *reinterpret_cast<const f32x4*>(row + half + r0 / 2);
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = cv[i], s[i] = sv[i];
      } else {
        load8(row + (first ? r0 : r0 - half), c);
        load8(row + half + (first ? r0 : r0 - half), s);
        if (first) {
#pragma unroll
          for (int i = 0; i < 8; ++i) s[i] = -s[i];
        }
      }
    }
  }
  const int mate_e0 = rot ? 8 * mate : (in ? e0 : 0);

#pragma unroll
  for (int i = 0; i < HP; ++i) {
    const int h = h0 + i * kGroups;
    if (blockIdx.y * (kGroups * HP) + i * kGroups >= a.heads) break;  // the same for the whole block
    const bool is_q = h < a.q_heads;
    float x[8];
    unpack8(raw[i], x);
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = __builtin_fmaf(x[j], x[j], sum);
#pragma unroll
    for (int d = 1; d < L; d <<= 1) sum += __shfl_xor(sum, d, L);
    const float f = 1.f / sqrtf(__builtin_fmaf(sum, a.inv_d, a.eps));
    const float* wp = is_q ? a.qw : a.kw;
    float w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 1.f;
    if (wp && in) load8(wp + e0, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = x[j] * f * w[j];
    if (a.R) {
      if (INTER) {
        if (rot) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float u = x[2 * j], v = x[2 * j + 1];
            x[2 * j] = u * c[j] - v * s[j];
            x[2 * j + 1] = v * c[j] + u * s[j];
          }
        }
      } else {
        u32x4 other;
#pragma unroll
        for (int j = 0; j < 4; ++j) other[j] = __shfl(raw[i][j], rot ? mate : l, L);
        float y[8];
        unpack8(other, y);
        if (wp) load8(wp + mate_e0, w);
        if (rot) {
          // s is -sin in the first half, sin in the second
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = x[j] * c[j] + y[j] * f * w[j] * s[j];
        }
      }
    }
    if (in && h < a.heads) {
      const moe_heads& o = is_q ? a.q_out : a.k_out;
      u32x4 v;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] = float_to_bf16_bits(x[2 * j]) | static_cast<uint32_t>(float_to_bf16_bits(x[2 * j + 1])) << 16;
      *reinterpret_cast<u32x4*>(o.base + t * o.row_stride + (is_q ? h : h - a.q_heads) * o.head_stride + e0) = v;
    }
  }
}

template <int L, bool INTER>
void launch(const NormArgs& a, int T, hipStream_t s) {
  constexpr int kGroups = 256 / L;
  constexpr int kMany = 4;
  // few tokens: one head per group, so that the heads spread over the card
  if (a.heads <= kGroups || static_cast<int64_t>(T) * a.heads <= 1024 * kGroups)
    norm_rope_kernel<L, 1, INTER><<<dim3(T, (a.heads + kGroups - 1) / kGroups), 256, 0, s>>>(a);
  else
    norm_rope_kernel<L, kMany, INTER><<<dim3(T, (a.heads + kGroups * kMany - 1) / (kGroups * kMany)), 256, 0, s>>>(a);
}

template <bool INTER>
void launch_for(const NormArgs& a, int T, hipStream_t s) {
  if (a.D <= 64)
    launch<8, INTER>(a, T, s);
  else if (a.D <= 128)
    launch<16, INTER>(a, T, s);
  else if (a.D <= 256)
    launch<32, INTER>(a, T, s);
  else
    launch<64, INTER>(a, T, s);
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
  if (head_dim < 8 || head_dim > 512 || head_dim % 8 != 0) return MOE_ESHAPE;
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
  a.q_heads = q_heads, a.heads = q_heads + k_heads;
  a.D = head_dim, a.P = n_positions, a.R = rot_dim, a.off = rot_offset;
  a.eps = eps, a.inv_d = 1.f / static_cast<float>(head_dim);
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (interleaved)
    moe::launch_for<true>(a, T, s);
  else
    moe::launch_for<false>(a, T, s);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_EHIP;
}
