// One tile of keys against the rows of a wave, with the running maximum and sum of
// a softmax: what the attention kernels share.
//
// The scores are computed transposed,
// S^T = K Q^T, with the 32x32x16 bf16 MFMA: its result puts one query in each
// lane (column n = lane % 32; the two lanes n and n + 32 hold alternating groups
// of four keys), so the row maximum is a maximum over registers and one lane
// exchange, the running maximum m and sum l are one register each, and the
// rescale of the output by 2^(m_old - m_new) is a multiplication by a lane's
// own scalar.  The output is accumulated transposed too, O^T = V^T P^T: the
// registers of S^T, rounded to bf16 in pairs, already are the B operand (the
// order of the keys inside an MFMA is free as long as V's operand has the same
// order), and V^T comes from LDS through the transposing 8-byte reads.  P never
// leaves the registers.
//
// The output is only rescaled when some row's maximum has risen by more than
// 2^8 over the maximum in use: until then the weights are at most 2^8 too large,
// which float32 sums and bf16 weights (whose error is relative) hold as well.
//
// Keys that a row must not see are set to -infinity in S, so whatever K holds
// there is replaced; their weight is then exactly 0, but 0 times an infinite or
// NaN value would still reach the row.  So a wave looks through the values of a
// masked tile first and, where one is not finite, takes the product over the
// finite ones and adds the others only to the rows that see them.
#pragma once

#include "lds_dma.h"
#include "moe_internal.h"

namespace moe {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((__vector_size__(4 * sizeof(short)))) short s16x4;
typedef __attribute__((__vector_size__(8 * sizeof(short)))) short s16x8;

constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLazy = 8.0f;  // log2 of how far a row's maximum may rise before the output is rescaled
constexpr float kLargeScore = 0x1p16f;  // base-two score from which the maximum is subtracted before the scale

__device__ __forceinline__ f32x16 mfma32(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// The maximum and the sum of the values of lanes l and l ^ 32 (the swap gives
// both lanes the lower lane's value first, the upper one's second).
__device__ __forceinline__ float max_halves(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_halves(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// LDS slot of 16-byte chunk c of tile row r.  Key rows are read 16 bytes at a
// time by 32 lanes in 32 rows: the XOR spreads 16 consecutive rows over all
// banks.  Value rows are read by the transposing loads, 64 bytes of each of four
// consecutive rows at a time: the XOR puts those in four different 64-byte windows.
template <int D>
__device__ __forceinline__ int k_slot(int r, int c) {
  return D >= 128 ? c ^ (r & 15) : c ^ ((r >> 1) & 7);
}
template <int D>
__device__ __forceinline__ int v_slot(int r, int c) {
  return D >= 128 ? c ^ ((r & 3) << 2) : c ^ (((r >> 1) & 1) << 2);
}

// Four consecutive keys of one value column per lane: the transposing read.
__device__ __forceinline__ s16x4 ld_tr(const uint8_t* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(p));
}

// ---------------------------------------------------------------- one key tile
// What a lane carries for its query: the running maximum (of the unscaled
// scores), the sum of its own half of the weights, and 16 output rows per 32.
template <int D>
struct RowState {
  f32x16 o[D / 32];
  float m, l;
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] = 0.f;
    m = kNegInf;
    l = 0.f;
  }
};

// A value fragment with zeros for what is not finite.
__device__ __forceinline__ s16x8 clean(s16x8 v) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = (v[e] & 0x7f80) == 0x7f80 ? 0 : v[e];
  return v;
}

// The last key of each 16 that the lane's row sees, counted in the tile: an entry
// below its 16 keys hides them all.  (A tile may hold two pages or more, and a row
// may see one of them alone.)
template <int NT>
struct Limits {
  int at[2 * NT];
};

// The last visible key for the 16 keys i: one for all, or one each.
__device__ __forceinline__ int limit_of(int lim, int) { return lim; }
template <int NT>
__device__ __forceinline__ int limit_of(const Limits<NT>& lim, int i) { return lim.at[i]; }

// Attend to NT x 32 keys: ks and vs are the tile's rows in LDS, c = scale *
// log2(e), lim the last visible key of the lane's row, counted in the tile.
// dirty: values that are not finite count as zeros (masked tiles only).
// KEEP = false: the LDS addresses are not kept in registers from tile to tile (a lane number that the
// compiler takes for new has none), which a kernel does where it has no registers left.
template <int D, int NT, bool MASKED, bool KEEP = true, typename Lim>
__device__ __forceinline__ void attend(const uint8_t* ks, const uint8_t* vs, const bf16x8 (&q)[D / 16],
                                       RowState<D>& st, float c, Lim lim, bool dirty) {
  int lane = threadIdx.x & 63;
  if constexpr (!KEEP) asm volatile("" : "+v"(lane));
  const int n = lane & 31, h = lane >> 5;
  f32x16 s[NT];
  u32x4 kf[2][NT];  // the next step's operands are read while this one's are used
  auto read_k = [&](int i) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
      kf[i & 1][t] = ld16(ks + (32 * t + n) * (2 * D) + 16 * k_slot<D>(n, 2 * i + h));
  };
  read_k(0);
#pragma unroll
  for (int t = 0; t < NT; ++t) s[t] = 0.f;
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    if (i + 1 < D / 16) read_k(i + 1);
#pragma unroll
    for (int t = 0; t < NT; ++t) s[t] = mfma32(__builtin_bit_cast(bf16x8, kf[i & 1][t]), q[i], s[t]);
    __builtin_amdgcn_sched_barrier(0);
  }
  // lane (n, h), register i of s[t]: key 32 t + 8 (i / 4) + 4 h + i % 4
  if constexpr (MASKED) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        s[t][i] = 32 * t + 8 * (i / 4) + i % 4 <= limit_of(lim, 2 * t + i / 8) - 4 * h ? s[t][i] : kNegInf;
  }
  float mt = s[0][0];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 16; ++i) mt = fmaxf(mt, s[t][i]);
  mt = max_halves(mt);
  if (__any((mt - st.m) * c > kLazy)) {
    const float mn = fmaxf(st.m, mt);
    const float alpha = st.m == mn ? 1.f : __builtin_amdgcn_exp2f((st.m - mn) * c);
    st.m = mn;
    st.l *= alpha;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) st.o[i] *= alpha;
  }
  // A weight's exponent is one FMA, s c - m c, whose m c is rounded: off by 2^-24 of
  // it, no more than the rounding of s itself costs, and the same for all the weights
  // of the tile.  But where m c is large that is too much for an exponent (from
  // 2^31 on the weights would all be 0 or infinite), so there m is subtracted first.
  float mc = st.m == kNegInf ? 0.f : st.m * c;
  if (__any(fabsf(mc) > kLargeScore)) {
    const float m = st.m == kNegInf ? 0.f : st.m;
#pragma unroll
    for (int t = 0; t < NT; ++t) s[t] -= m;
    mc = 0.f;
  }
  // The weights are summed as rounded, so that their rounding leaves a row's
  // weights normalised: one dot product with ones per pair.
  const bf16x2 ones = {static_cast<__bf16>(1.f), static_cast<__bf16>(1.f)};
  bf16x8 p[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      bf16x2 e;
      e[0] = static_cast<__bf16>(__builtin_amdgcn_exp2f(__builtin_fmaf(s[t][i], c, -mc)));
      e[1] = static_cast<__bf16>(__builtin_amdgcn_exp2f(__builtin_fmaf(s[t][i + 1], c, -mc)));
      st.l = __builtin_amdgcn_fdot2_f32_bf16(e, ones, st.l, false);
      p[t][i / 8][i % 8] = e[0];
      p[t][i / 8][i % 8 + 1] = e[1];
    }

  // V^T operand: lane holds column d = lane % 32 of the 32-wide slice and the
  // keys 16 j + 4 h + {0..3, 8..11}, the order of p.  In each group of 16 lanes,
  // lane i reads 8 bytes of key row i / 4 and gets column i of the four rows.
  const int i16 = lane & 15, vr = 4 * h + (i16 >> 2);
  const uint8_t* vrow = vs + vr * (2 * D) + 8 * (i16 & 1);
  const int vc = 2 * ((lane >> 4) & 1) + ((i16 & 3) >> 1);
  s16x8 vf[2][NT][2];
  auto read_v = [&](int d) {
    const uint8_t* vp = vrow + 16 * v_slot<D>(vr, 4 * d + vc);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const s16x4 lo = ld_tr(vp + (32 * t + 16 * j) * (2 * D));
        const s16x4 hi = ld_tr(vp + (32 * t + 16 * j + 8) * (2 * D));
        vf[d & 1][t][j] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        if (MASKED && dirty) vf[d & 1][t][j] = clean(vf[d & 1][t][j]);
      }
  };
  read_v(0);
#pragma unroll
  for (int d = 0; d < D / 32; ++d) {
    if (d + 1 < D / 32) read_v(d + 1);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j) st.o[d] = mfma32(__builtin_bit_cast(bf16x8, vf[d & 1][t][j]), p[t][j], st.o[d]);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// ---------------------------------------------------------------- masked tiles
// Whether a value tile of `bytes` bytes holds anything that is not finite.
__device__ __forceinline__ bool any_not_finite(const uint8_t* vs, int bytes) {
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  u16x2 top = {0, 0};
#pragma unroll 4
  for (int i = 16 * (threadIdx.x & 63); i < bytes; i += 1024) {
    const u32x4 w = ld16(vs + i);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, w[e] & 0x7fff7fffu));
  }
  return __any(top[0] >= 0x7f80 || top[1] >= 0x7f80);
}

// What is not finite in a row of values, at p + 4 (lane / 32), added to the lane's outputs.
template <int D>
__device__ __forceinline__ void add_not_finite(const uint16_t* p, RowState<D>& st) {
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const u32x2 w = *reinterpret_cast<const u32x2*>(p + 32 * i + 8 * j);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t b = w[e / 2] >> (16 * (e % 2));
        st.o[i][4 * j + e] += (b & 0x7f80u) == 0x7f80u ? __uint_as_float(b << 16) : 0.f;
      }
      __builtin_amdgcn_sched_barrier(0);  // rare: keep it out of the registers of the common path
    }
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

}  // namespace moe
