// Matrix product in E4M3 with one scale per block of 128
// (include/moe_attention.h, moe_fp8_linear): y = x W^T, W as stored with a scale
// per 128 x 128 block, x quantised here with a scale per token and 128 columns.
//
// One v_mfma_scale_f32_16x16x128_f8f6f4 covers exactly one block of K, so a
// scale is constant inside it.  E8M0 scales go to the instruction, which applies
// them for nothing: the whole K is summed in one accumulator.  float32 scales
// cannot: each block's product starts from zero and is added as
// acc += (sx * sw) * product, four vector FMAs per MFMA, which run beside the
// matrix cores.  The weights are the A operand (result rows) and the tokens
// the B operand (result columns), so a lane's four results are four
// consecutive outputs of one token, and its token's scale is a lane's scalar.
//
// Past the end of K the quantised x is zero (its rows are padded to whole
// blocks), and W repeats its row's last 16 bytes: zero times a weight the row holds
// anyway.  Past the end of N and T the last row is repeated, or zeros are read, and
// nothing is stored.
#include <algorithm>

#include "../../include/moe_attention.h"
#include "lds_dma.h"
#include "moe_internal.h"

namespace moe {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr float kFp8Max = 448.f;
constexpr float kFloor = 0x1p-100f;  // least block maximum: keeps every scale and its inverse normal

// ---------------------------------------------------------------- quantisation
// The scale of a block from its largest magnitude, as the word the kernels
// take (the E8M0 byte, or the float32's bits), and the factor that x is
// multiplied by.
template <bool F32>
__device__ __forceinline__ uint32_t block_scale(float amax, float& inv) {
  amax = fmaxf(amax, kFloor);
  if (F32) {
    inv = kFp8Max / amax;
    return __float_as_uint(amax / kFp8Max);
  }
  // amax = 1.m * 2^(E - 127) and 448 = 1.75 * 2^8: the least e with amax <= 448 * 2^(e - 127)
  const uint32_t b = __float_as_uint(amax);
  const uint32_t e = (b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  inv = __uint_as_float((254 - e) << 23);
  return e;
}

__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Four consecutive values (two words of bf16 pairs) to four codes.
__device__ __forceinline__ uint32_t codes4(uint32_t w0, uint32_t w1, float inv) {
  int c = __builtin_amdgcn_cvt_pk_fp8_f32(lo_bf16(w0) * inv, hi_bf16(w0) * inv, 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(lo_bf16(w1) * inv, hi_bf16(w1) * inv, c, true));
}

__device__ __forceinline__ float max_abs(u32x4 w, float m) {
#pragma unroll
  for (int i = 0; i < 4; ++i) m = fmaxf(m, fmaxf(fabsf(lo_bf16(w[i])), fabsf(hi_bf16(w[i]))));
  return m;
}

// codes [kb, T, 128] (the last block padded with zeros), scales [kb, T].  Block by
// block, so that the rows a tile kernel reads at once are contiguous: rows K
// bytes apart would fall on few of the L2's channels.  16 lanes per block, 8
// values each.  Bound by HBM: 16384 x 4096 are 203 MB in 38 us = 5.3 TB/s (two, four or
// eight blocks per lane group the same).
template <bool F32>
__global__ __launch_bounds__(256) void fp8_quant_kernel(const uint16_t* __restrict__ x, int64_t x_stride, int T, int K,
                                                        int kb, uint8_t* __restrict__ codes,
                                                        uint32_t* __restrict__ scales) {
  const int64_t u = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4);
  if (u >= static_cast<int64_t>(T) * kb) return;
  const int64_t t = u / kb;
  const int b = static_cast<int>(u - t * kb), k = 128 * b + 8 * (threadIdx.x & 15);
  u32x4 w = {0, 0, 0, 0};
  if (k < K) w = ld16(x + t * x_stride + k);
  float m = max_abs(w, 0.f);
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) m = fmaxf(m, __shfl_xor(m, d, 16));
  float inv;
  const uint32_t s = block_scale<F32>(m, inv);
  const u32x2 c = {codes4(w[0], w[1], inv), codes4(w[2], w[3], inv)};
  *reinterpret_cast<u32x2*>(codes + (static_cast<int64_t>(b) * T + t) * 128 + 8 * (threadIdx.x & 15)) = c;
  if ((threadIdx.x & 15) == 0) scales[static_cast<int64_t>(b) * T + t] = s;
}

// ---------------------------------------------------------------- the product of one block
__device__ __forceinline__ i32x8 join(u32x4 a, u32x4 b) {
  return i32x8{static_cast<int>(a[0]), static_cast<int>(a[1]), static_cast<int>(a[2]), static_cast<int>(a[3]),
               static_cast<int>(b[0]), static_cast<int>(b[1]), static_cast<int>(b[2]), static_cast<int>(b[3])};
}

// acc += the scaled product of one 128-column block.  sw is W's scale word (the
// same in all lanes), sx the lane's token's; f32: their product, taken once per
// token tile.
template <bool F32>
__device__ __forceinline__ void block_mfma(i32x8 w, i32x8 x, f32x4& acc, int sw, int sx, float f32) {
  if (F32) {
    const f32x4 z = {0.f, 0.f, 0.f, 0.f};
    // scale operands of 127: 1.0
    const f32x4 p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, z, 0, 0, 0, 127, 0, 127);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(f32, p[i], acc[i]);
  } else {
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, acc, 0, 0, 0, sw, 0, sx);
  }
}

// W's scale of (128-row block nb, column block b), as a word.
template <bool F32>
__device__ __forceinline__ uint32_t weight_scale(const void* s, int64_t i) {
  return F32 ? static_cast<const uint32_t*>(s)[i] : static_cast<const uint8_t*>(s)[i];
}

// Four consecutive outputs n .. n + 3 of token t.
__device__ __forceinline__ void store4(uint16_t* y, int64_t y_stride, int64_t t, int n, int N, bool wide, f32x4 v) {
  uint16_t* p = y + t * y_stride + n;
  if (wide && n + 4 <= N) {
    const u32x2 w = {float_to_bf16_bits(v[0]) | static_cast<uint32_t>(float_to_bf16_bits(v[1])) << 16,
                     float_to_bf16_bits(v[2]) | static_cast<uint32_t>(float_to_bf16_bits(v[3])) << 16};
    *reinterpret_cast<u32x2*>(p) = w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < N) p[i] = float_to_bf16_bits(v[i]);
  }
}

struct LinearArgs {
  const uint16_t* x;
  int64_t x_stride, y_stride;
  const uint8_t* w;
  const void* w_scale;
  uint16_t* y;
  const uint8_t* codes;    // quantised x [kb, T, 128]
  const uint32_t* scales;  // [kb, T]
  int T, N, K, kb;         // kb: blocks of K
  int n_tiles, t_tiles;
  int splits, chunk;       // of K: a split takes chunk blocks
  f32x4* part;             // [splits, tiles, BN BT / 4]: the splits' sums
  bool wide;               // rows of y take 8-byte stores
};

// ---------------------------------------------------------------- few tokens
// A block holds 16 NI rows of W and 16 MT tokens; its NW waves take the blocks of
// K in turn, straight from memory, and meet in LDS.  W is read once per token
// block: the kernel streams it.  QUANT: the block quantises x itself, into LDS,
// while its first loads of W are on their way.  Bound by latency (1 x 6144 x 4096: 7.9
// us, 3.2 TB/s, of which 3.8 us are left with W in the cache) and, with more tokens, by x,
// which every block reads whole from its L2 (16 x 6144 x 4096: 13.1 us).
constexpr int kNW = 8;
// Codes of x that the block quantises itself (8 x 2048 x 2048, 16 KB, 5.1 us, by a
// kernel of its own 5.8; 8 x 6144 x 4096, 32 KB, 13.1 against 11.6).
constexpr int kFusedBytes = 16 << 10;

template <int MT, int NI, bool F32, bool QUANT>
__global__ __launch_bounds__(64 * kNW) void fp8_few_kernel(LinearArgs a) {
  static_assert(MT * NI <= kNW, "a wave per tile at the end");
  constexpr int kU = MT <= 2 ? 4 : 2;  // blocks of K in flight per wave
  __shared__ f32x4 part[kNW][MT * NI][64];
  __shared__ __attribute__((aligned(16))) uint8_t q_codes[QUANT ? kFusedBytes : 16];
  __shared__ uint32_t q_scales[QUANT ? kFusedBytes / 128 : 1];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int r = lane & 15, g = lane >> 4;
  const int n0 = 16 * NI * blockIdx.x, t0 = 16 * MT * blockIdx.y;
  const uint8_t* wp[NI];
  int64_t srow[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    wp[i] = a.w + static_cast<int64_t>(min(n0 + 16 * i + r, a.N - 1)) * a.K;
    srow[i] = static_cast<int64_t>(min(n0 + 16 * i, a.N - 1) >> 7) * a.kb;
  }
  const int last = a.K - 16;

  f32x4 acc[NI][MT];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[i][m] = f32x4{0.f, 0.f, 0.f, 0.f};

  u32x4 wv[kU][NI][2];
  uint32_t sw[kU][NI];
  auto load_w = [&](int b0) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int b = b0 + u * kNW, k = 128 * b + 32 * g;
      if (b >= a.kb) break;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        wv[u][i][0] = ld16(wp[i] + min(k, last));
        wv[u][i][1] = ld16(wp[i] + min(k + 16, last));
        sw[u][i] = weight_scale<F32>(a.w_scale, srow[i] + b);
      }
    }
  };
  load_w(wave);
  if (QUANT) {
    __builtin_amdgcn_sched_barrier(0);
    // 16 lanes per token and block of K, 8 values each; all the loads first
    constexpr int kPer = kFusedBytes / 8 / (64 * kNW);
    const int cols = a.kb * 16, all = a.T * cols;
    u32x4 w[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int u = threadIdx.x + 64 * kNW * i, t = u / cols, c = u - t * cols;
      w[i] = u32x4{0, 0, 0, 0};
      if (u < all && 8 * c < a.K) w[i] = ld16(a.x + t * a.x_stride + 8 * c);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int u = threadIdx.x + 64 * kNW * i;
      if (u >= all) break;
      float m = max_abs(w[i], 0.f), inv;
#pragma unroll
      for (int d = 1; d < 16; d <<= 1) m = fmaxf(m, __shfl_xor(m, d, 16));
      const uint32_t s = block_scale<F32>(m, inv);
      *reinterpret_cast<u32x2*>(&q_codes[8 * u]) = u32x2{codes4(w[i][0], w[i][1], inv), codes4(w[i][2], w[i][3], inv)};
      if ((u & 15) == 0) q_scales[u >> 4] = s;
    }
    stage_barrier();  // leaves the loads of W in flight
  }

  for (int b0 = wave; b0 < a.kb; b0 += kNW * kU) {
    u32x4 xv[kU][MT][2];
    uint32_t sx[kU][MT];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int b = b0 + u * kNW;
      if (b >= a.kb) break;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int t = min(t0 + 16 * m + r, a.T - 1);
        const uint8_t* p = QUANT ? &q_codes[128 * (t * a.kb + b) + 32 * g]
                                 : a.codes + (static_cast<int64_t>(b) * a.T + t) * 128 + 32 * g;
        xv[u][m][0] = ld16(p);
        xv[u][m][1] = ld16(p + 16);
        sx[u][m] = QUANT ? q_scales[t * a.kb + b] : a.scales[static_cast<int64_t>(b) * a.T + t];
      }
    }
    __builtin_amdgcn_sched_barrier(0);  // all of them are on their way before the first is used
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (b0 + u * kNW >= a.kb) break;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const i32x8 wf = join(wv[u][i][0], wv[u][i][1]);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const float f = F32 ? __uint_as_float(sw[u][i]) * __uint_as_float(sx[u][m]) : 0.f;
          block_mfma<F32>(wf, join(xv[u][m][0], xv[u][m][1]), acc[i][m], static_cast<int>(sw[u][i]),
                          static_cast<int>(sx[u][m]), f);
        }
      }
    }
    if (b0 + kNW * kU < a.kb) load_w(b0 + kNW * kU);
  }

#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int m = 0; m < MT; ++m) part[wave][i * MT + m][lane] = acc[i][m];
  __syncthreads();
  if (wave >= MT * NI) return;
  f32x4 v = part[0][wave][lane];
#pragma unroll
  for (int i = 1; i < kNW; ++i) v += part[i][wave][lane];
  const int t = t0 + 16 * (wave % MT) + r;
  if (t < a.T) store4(a.y, a.y_stride, t, n0 + 16 * (wave / MT) + 4 * g, a.N, a.wide, v);
}

// ---------------------------------------------------------------- many tokens
// A block of eight waves holds BN rows of W and BT tokens: group 0 (waves 0 to 3)
// the first half of the rows, group 1 the second, each wave a quarter of the
// tokens.  Both operands come through LDS by DMA, in two stages of one block of K.
//
// Two waves share a SIMD, one of each group.  Were both to read their fragments
// after the same barrier and multiply after that, the matrix cores would wait for
// the LDS in every step; so the groups run half a step apart: while one reads the
// fragments of a block of K into its registers, the other multiplies, and a
// barrier swaps them.
//
//   phase 2 b       group 0 reads block b        group 1 multiplies block b - 1
//   phase 2 b + 1   group 0 multiplies block b   group 1 reads block b
//
// Each part of a stage is refilled as soon as its readers are done, so that
// loads are in flight at all times: the tokens X (read in both phases) and group
// 1's rows of block b + 1 are issued in phase 2 b, group 0's rows of block b + 2 in
// phase 2 b + 1.  The loads return in order, so a wait names how many of the
// latest may still be out.
//
// With 256 x 256 tiles a phase takes about 1.7 times its products: 16384 x 6144 x 4096 in 386
// to 397 us with its 40 of quantisation, 2.3 to 2.4 PFLOP/s for the product (a library
// product of quantised operands with one scale each: 344 us); without the copies'
// traffic, on zeros, the call would take 350.  4096^3 with float32 scales 80 to 82 with
// its 14, 2.05 PFLOP/s (library: 54).  128 x 64 tiles with K split are bound by the
// latency of a step, about 0.6 us.
//
// Layout: rows of 128 bytes, 16-byte chunk c of row r in slot c ^ ((r / 2) mod 8),
// which spreads the 16 rows of a fragment read over all banks.  An operand's lane
// (r, g) holds chunks g and 4 + g of row r.  Every part is a variable of its own:
// the compiler then knows that a DMA in flight does not write what is read.
__device__ __forceinline__ int slot(int r, int c) { return c ^ ((r >> 1) & 7); }

// Consecutive tiles cover kBand token tiles before the next rows of W, so that
// the blocks an XCD runs at once share both operands in its L2.
template <int BN, int BT>
__device__ __forceinline__ void tile_place(const LinearArgs& a, int tile, int& n0, int& t0) {
  constexpr int kBand = 4;
  const int band = tile / (kBand * a.n_tiles), in_band = tile - band * kBand * a.n_tiles;
  const int wide = min(kBand, a.t_tiles - kBand * band);
  t0 = __builtin_amdgcn_readfirstlane((kBand * band + in_band % wide) * BT);
  n0 = __builtin_amdgcn_readfirstlane((in_band / wide) * BN);
}

template <int BN, int BT, bool F32>
__global__ __launch_bounds__(512, 2) void fp8_tile_kernel(LinearArgs a) {
  constexpr int kN = BN / 32, kT = BT / 64;        // 16 x 16 tiles of a wave
  constexpr int kWOps = BN / 128, kXOps = BT / 64;  // DMA instructions of a wave: a group's rows; the tokens
  struct Tokens {
    uint8_t x[BT * 128];
    uint32_t s[BT];
  };
  __shared__ __attribute__((aligned(1024))) Tokens x0;
  __shared__ __attribute__((aligned(1024))) Tokens x1;
  __shared__ __attribute__((aligned(1024))) uint8_t wa0[BN * 64];
  __shared__ __attribute__((aligned(1024))) uint8_t wa1[BN * 64];
  __shared__ __attribute__((aligned(1024))) uint8_t wb0[BN * 64];
  __shared__ __attribute__((aligned(1024))) uint8_t wb1[BN * 64];
  __shared__ uint32_t w_scale[2][MOE_MAX_DIM / 128];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int group = wave >> 2, wt = wave & 3;
  const int r = lane & 15, g = lane >> 4;

  // Blocks are dealt to the 8 XCDs in turn: each XCD gets a run of consecutive
  // units, the tiles of one split of K after those of another.
  const int tiles = a.n_tiles * a.t_tiles, total = tiles * a.splits, per = (total + 7) >> 3;
  const int unit = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if ((blockIdx.x >> 3) >= per || unit >= total) return;
  const int split = unit / tiles;
  const int begin = split * a.chunk, end = min(a.kb, begin + a.chunk);  // of the blocks of K
  int n0, t0;
  tile_place<BN, BT>(a, unit - split * tiles, n0, t0);

  // W's scales of the two groups' rows
  for (int i = threadIdx.x; i < 2 * a.kb; i += 512) {
    const int h = i >= a.kb, b = i - (h ? a.kb : 0);
    w_scale[h][b] = weight_scale<F32>(a.w_scale, static_cast<int64_t>(min(n0 + h * (BN / 2), a.N - 1) >> 7) * a.kb + b);
  }

  // Sources: one 32-bit lane offset per operand from the part's first row (the
  // instructions of a wave are 64 rows apart).  Rows past the end of W or x lie
  // past the end of the resource, which reads as zeros; they are not stored.
  // So do the blocks past the last one, which the loop asks for: their resource
  // is empty, and no memory is read.
  const int w_bytes[2] = {__builtin_amdgcn_readfirstlane(min(BN / 2, a.N - n0) * a.K),
                          __builtin_amdgcn_readfirstlane(max(min(BN / 2, a.N - n0 - BN / 2), 0) * a.K)};
  const int x_rows = __builtin_amdgcn_readfirstlane(min(BT, a.T - t0));
  const int row0 = 8 * wave + (lane >> 3);
  // Instruction i of the rows of group h, of block b.
  auto issue_w = [&](int h, uint8_t* to, int b, int i) __attribute__((always_inline)) {
    int row = row0;
    asm volatile("" : "+v"(row));  // derived offsets are not kept in registers from step to step
    const __amdgpu_buffer_rsrc_t src =
        raw_buffer(a.w + static_cast<int64_t>(n0 + h * (BN / 2)) * a.K, b < end ? w_bytes[h] : 0);
    const int k = row * a.K + min(128 * b + 16 * slot(row, lane & 7), a.K - 16);
    dma16(src, k + 64 * i * a.K, 0, to + 1024 * (8 * i + wave));
  };
  // Instruction i of the tokens of block b; the last one takes their scales.
  const int spart = wave % (BT / 64);
  auto issue_x = [&](Tokens& to, int b, int i) __attribute__((always_inline)) {
    const int64_t first = static_cast<int64_t>(b) * a.T + t0;
    const int rows = b < end ? x_rows : 0;
    if (i == kXOps) {
      dma4(raw_buffer(a.scales + first, 4 * rows), 4 * (64 * spart + lane), &to.s[64 * spart]);
      return;
    }
    int row = row0;
    asm volatile("" : "+v"(row));
    dma16(raw_buffer(a.codes + 128 * first, 128 * rows), 128 * row + 16 * slot(row, lane & 7) + 8192 * i, 0,
          &to.x[1024 * (8 * i + wave)]);
  };
  // What an even phase issues for block b, and an odd one.
  constexpr int kEven = kXOps + 1 + kWOps, kOdd = kWOps;
  // Where they go out (us, first choice against the other): large tiles after the
  // fragments are read (4096^3, float32 scales, 80.5 against 85.8; 768 x 6144 x 4096 38.8, 40.9) and
  // between the products (16384 x 6144 x 4096 386 to 393, all at the start of them 405);
  // 64 tokens, bound by latency, first of all (64 x 8192 x 8192 25.5, 26.9).
  constexpr bool kLate = BT > 64, kSpread = BN == 256;
  auto even_op = [&](Tokens& x, uint8_t* wb, int b, int i) __attribute__((always_inline)) {
    if (i <= kXOps) issue_x(x, b, i); else issue_w(1, wb, b, i - kXOps - 1);
  };

  f32x4 acc[kN][kT];
#pragma unroll
  for (int i = 0; i < kN; ++i)
#pragma unroll
    for (int j = 0; j < kT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  i32x8 wf[kN], xf[kT];
  uint32_t sx[kT], sw;
  const int operand = 128 * r + 16 * slot(r, g);  // chunk 4 + g is at ^ 64
  auto read = [&](const Tokens& x, const uint8_t* w, int b) __attribute__((always_inline)) {
    __builtin_amdgcn_sched_barrier(0);
    int c = operand;
    asm volatile("" : "+v"(c));
    const uint8_t* xp = &x.x[128 * (BT / 4) * wt];
#pragma unroll
    for (int j = 0; j < kT; ++j) {
      xf[j] = join(ld16(xp + 2048 * j + c), ld16(xp + 2048 * j + (c ^ 64)));
      sx[j] = x.s[(BT / 4) * wt + 16 * j + (c >> 7)];
    }
    sw = w_scale[group][b];
#pragma unroll
    for (int i = 0; i < kN; ++i) wf[i] = join(ld16(w + 2048 * i + c), ld16(w + 2048 * i + (c ^ 64)));
    __builtin_amdgcn_sched_barrier(0);
  };
  // The loads that go out in this phase can be spread over the products: a wave issues
  // in order, and would wait for the queue of the loads before its first product.
  auto multiply = [&](int ops, auto&& op) __attribute__((always_inline)) {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(1);
    float f[kT];
    if (F32) {
#pragma unroll
      for (int j = 0; j < kT; ++j) f[j] = __uint_as_float(sx[j]) * __uint_as_float(sw);
    }
    // float32 scales: product u is added kLag products later, when it is there
    // (4096 x 4096 x 4096: 82 us; 2 later 84, 1 later 86, at once 106)
    constexpr int kLag = 3;
    f32x4 p[kLag + 1];
    auto add = [&](int u) __attribute__((always_inline)) {
      const int i = u / kT, j = u % kT;
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(f[j], p[u % (kLag + 1)][e], acc[i][j][e]);
    };
#pragma unroll
    for (int u = 0; u < kN * kT; ++u) {
      const int i = u / kT, j = u % kT;
      if (F32) {
        const f32x4 z = {0.f, 0.f, 0.f, 0.f};
        p[u % (kLag + 1)] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf[i], xf[j], z, 0, 0, 0, 127, 0, 127);
        __builtin_amdgcn_sched_barrier(0);  // the additions stay behind this product
        if (u >= kLag) add(u - kLag);
      } else {
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf[i], xf[j], acc[i][j], 0, 0, 0,
                                                                     static_cast<int>(sw), 0, static_cast<int>(sx[j]));
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int k = 0; k < ops; ++k)
        if ((kSpread ? k * kN * kT / ops : 0) == u) op(k);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (F32) {
#pragma unroll
      for (int u = kN * kT - kLag; u < kN * kT; ++u) add(u);
    }
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
  };
  // The end of an even phase: group 1's rows of the block have arrived; rows of
  // group 0, tokens and rows of group 1 were issued since.
  auto end_even = [&]() __attribute__((always_inline)) {
    wait_vmcnt<2 * kWOps + kXOps + 1>();
    stage_barrier();
  };
  // The end of an odd phase: the next block's tokens and rows of group 0 have
  // arrived; rows of group 1 and of group 0 were issued since.
  auto end_odd = [&]() __attribute__((always_inline)) {
    wait_vmcnt<2 * kWOps>();
    stage_barrier();
  };

#pragma unroll
  for (int i = 0; i < kOdd; ++i) issue_w(0, wa0, begin, i), issue_w(0, wa1, begin + 1, i);
#pragma unroll
  for (int i = 0; i < kEven; ++i) even_op(x0, wb0, begin, i);
  wait_vmcnt<0>();
  stage_barrier();
  int b = begin;
  if (group == 0) {
    auto step = [&](const Tokens& x, uint8_t* wa, Tokens& xn, uint8_t* wbn) __attribute__((always_inline)) {
      if (kLate) read(x, wa, b);
#pragma unroll
      for (int i = 0; i < kEven; ++i) even_op(xn, wbn, b + 1, i);
      if (!kLate) read(x, wa, b);
      end_even();
      multiply(kOdd, [&](int i) __attribute__((always_inline)) { issue_w(0, wa, b + 2, i); });
      end_odd();
      ++b;
    };
    while (b + 1 < end) {
      step(x0, wa0, x1, wb1);
      step(x1, wa1, x0, wb0);
    }
    if (b < end) step(x0, wa0, x1, wb1);
  } else {
    auto odd = [&](const Tokens& x, const uint8_t* wb, uint8_t* wa) __attribute__((always_inline)) {
      end_even();
      if (kLate) read(x, wb, b);
#pragma unroll
      for (int i = 0; i < kOdd; ++i) issue_w(0, wa, b + 2, i);
      if (!kLate) read(x, wb, b);
      end_odd();
      ++b;
    };
    auto step = [&](const Tokens& x, const uint8_t* wb, uint8_t* wa, Tokens& xn,
                    uint8_t* wbn) __attribute__((always_inline)) {
      multiply(kEven, [&](int i) __attribute__((always_inline)) { even_op(xn, wbn, b + 1, i); });
      odd(x, wb, wa);
    };
#pragma unroll
    for (int i = 0; i < kEven; ++i) even_op(x1, wb1, b + 1, i);
    odd(x0, wb0, wa0);
    while (b + 1 < end) {
      step(x1, wb1, wa1, x0, wb0);
      step(x0, wb0, wa0, x1, wb1);
    }
    if (b < end) step(x1, wb1, wa1, x0, wb0);
    multiply(0, [](int) {});
  }
  wait_vmcnt<0>();  // no DMA is left for the LDS of the next block

  if (BT == 64 && a.splits > 1) {
    f32x4* p = a.part + static_cast<int64_t>(unit) * (BN * BT / 4) + wave * (64 * kN * kT) + lane;
#pragma unroll
    for (int i = 0; i < kN; ++i)
#pragma unroll
      for (int j = 0; j < kT; ++j) p[64 * (i * kT + j)] = acc[i][j];
    return;
  }
#pragma unroll
  for (int j = 0; j < kT; ++j) {
    const int t = t0 + (BT / 4) * wt + 16 * j + r;
    if (t >= a.T) continue;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int n = n0 + group * (BN / 2) + 16 * i + 4 * g;
      store4(a.y, a.y_stride, t, n, a.N, a.wide, acc[i][j]);
    }
  }
}

// The sum of the splits, in order.  A block takes the tiles of one wave of one tile
// of the kernel above, and finds their places as that does.
template <int BN, int BT>
__global__ __launch_bounds__(256) void fp8_join_kernel(LinearArgs a) {
  constexpr int kN = BN / 32, kT = BT / 64;
  static_assert(kN * kT % 4 == 0, "four waves share the tiles");
  const int tiles = a.n_tiles * a.t_tiles, tile = blockIdx.x >> 3, wave = blockIdx.x & 7;
  int n0, t0;
  tile_place<BN, BT>(a, tile, n0, t0);
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
#pragma unroll
  for (int u = threadIdx.x >> 6; u < kN * kT; u += 4) {
    const f32x4* p = a.part + static_cast<int64_t>(tile) * (BN * BT / 4) + wave * (64 * kN * kT) + 64 * u + lane;
    f32x4 v = p[0];
    for (int i = 1; i < a.splits; ++i) v += p[static_cast<int64_t>(i) * tiles * (BN * BT / 4)];
    const int t = t0 + (BT / 4) * (wave & 3) + 16 * (u % kT) + r;
    const int n = n0 + (wave >> 2) * (BN / 2) + 16 * (u / kT) + 4 * g;
    if (t < a.T) store4(a.y, a.y_stride, t, n, a.N, a.wide, v);
  }
}

// ---------------------------------------------------------------- host
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t align256(size_t v) { return (v + 255) & ~size_t{255}; }
inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool shape_ok(int32_t T, int32_t N, int32_t K) {
  return T >= 0 && T <= MOE_MAX_TOKENS && N > 0 && N <= MOE_MAX_DIM && K > 0 && K <= MOE_MAX_DIM && K % 16 == 0;
}

// Which kernel (microseconds of a call with E8M0 scales, quantisation and join
// included, T x N x K).
//   Up to 16 tokens: the few-token kernel (16 x 6144 x 4096 13.1, 128 x 64 tiles 16.6;
//   16 x 4096 x 16384 24.1, 25.5).  Beyond, where its blocks are on the card at once and K
//   is short enough for a block of it: 17 to 32 tokens up to 48 blocks of K (32 x 4096 x 4096
//   10.7, tiles 14.0; 32 x 1024 x 8192 15.5, 13.5; 512 blocks, 32 x 8192 x 8192, 31.6, 25.3),
//   more tokens up to 24 (512 x 1024 x 2064 10.3, tiles 13.3; 128 x 4096 x 4096 16.9, 15.7;
//   512 blocks, 512 x 2048 x 2048, 17.7, 15.3).
//   128 x 64 tiles, K split over the card, below kTiles128 tiles of 128 x 128 (96 of
//   them, 768 x 2048 x 2048, 14.4, with 128 x 128 18.9; 160, 640 x 4096 x 4096, 32.4,
//   31.6; 256, 1024 x 4096 x 4096, 35.9, 33.1).
//   256 x 256 tiles from kTiles256 of them (128 tiles, 2048 x 4096 x 4096, 61.6, with
//   128 x 128 51.0; 160, 1280 x 8192 x 4096, 61.8, 65.9).
constexpr int64_t kCus = 256, kTiles128 = 160, kTiles256 = 160;

bool few_tokens(int64_t T, int64_t N, int64_t kb) {
  if (T <= 16) return true;
  if (T <= 32) return ceil_div(N, 16) <= kCus && kb <= 48;
  return ceil_div(N, 32) * ceil_div(T, 64) <= kCus && kb <= 24;
}

// Splits of K for 128 x 64 tiles: one block per CU, of at least 4 blocks of K (64 x
// 2048 x 2048 10.4; of at least 8 11.6; 64 x 8192 x 4096 18.4, two blocks per CU 20.7).
int splits_of(int64_t tiles, int64_t kb) {
  return static_cast<int>(std::max<int64_t>(1, std::min(kCus / tiles, kb / 4)));
}

// Room for the splits' sums of any call with up to T tokens, N rows and kb blocks of K.
size_t part_bytes(int64_t T, int64_t N, int64_t kb) {
  if (T <= 16) return 0;
  const int64_t tiles = ceil_div(N, 128) * ceil_div(T, 64);
  return static_cast<size_t>(std::min(kCus, tiles * std::max<int64_t>(kb / 4, 1))) * (128 * 64 * 4);
}

template <bool F32>
void launch(LinearArgs& a, hipStream_t s) {
  if (a.T <= 16 && a.T * a.kb * 128 <= kFusedBytes) {
    fp8_few_kernel<1, 1, F32, true><<<dim3(ceil_div(a.N, 16), 1), 64 * kNW, 0, s>>>(a);
    return;
  }
  fp8_quant_kernel<F32><<<static_cast<unsigned>(ceil_div(static_cast<int64_t>(a.T) * a.kb, 16)), 256, 0, s>>>(
      a.x, a.x_stride, a.T, a.K, a.kb, const_cast<uint8_t*>(a.codes), const_cast<uint32_t*>(a.scales));
  if (few_tokens(a.T, a.N, a.kb)) {
    if (a.T <= 16)
      fp8_few_kernel<1, 1, F32, false><<<dim3(ceil_div(a.N, 16), 1), 64 * kNW, 0, s>>>(a);
    else if (a.T <= 32)
      fp8_few_kernel<2, 1, F32, false><<<dim3(ceil_div(a.N, 16), 1), 64 * kNW, 0, s>>>(a);
    else
      fp8_few_kernel<4, 2, F32, false><<<dim3(ceil_div(a.N, 32), ceil_div(a.T, 64)), 64 * kNW, 0, s>>>(a);
    return;
  }
  auto tiles = [&](int bn, int bt, int splits) {
    a.n_tiles = static_cast<int>(ceil_div(a.N, bn));
    a.t_tiles = static_cast<int>(ceil_div(a.T, bt));
    a.chunk = static_cast<int>(ceil_div(a.kb, splits));
    a.splits = static_cast<int>(ceil_div(a.kb, a.chunk));
    return static_cast<unsigned>(ceil_div(static_cast<int64_t>(a.n_tiles) * a.t_tiles * a.splits, 8) * 8);
  };
  if (ceil_div(a.N, 256) * ceil_div(a.T, 256) >= kTiles256) {
    const unsigned grid = tiles(256, 256, 1);
    fp8_tile_kernel<256, 256, F32><<<grid, 512, 0, s>>>(a);
  } else if (ceil_div(a.N, 128) * ceil_div(a.T, 128) >= kTiles128) {
    const unsigned grid = tiles(128, 128, 1);
    fp8_tile_kernel<128, 128, F32><<<grid, 512, 0, s>>>(a);
  } else {
    const unsigned grid = tiles(128, 64, splits_of(ceil_div(a.N, 128) * ceil_div(a.T, 64), a.kb));
    fp8_tile_kernel<128, 64, F32><<<grid, 512, 0, s>>>(a);
    if (a.splits > 1)
      fp8_join_kernel<128, 64><<<static_cast<unsigned>(a.n_tiles * a.t_tiles) * 8, 256, 0, s>>>(a);
  }
}

}  // namespace
}  // namespace moe

extern "C" {

size_t moe_fp8_linear_workspace_size(int32_t T, int32_t N, int32_t K) {
  if (!moe::shape_ok(T, N, K) || T <= 0) return 0;
  const size_t kb = moe::ceil_div(K, 128);
  return moe::align256(static_cast<size_t>(T) * kb * 128) + moe::align256(static_cast<size_t>(T) * kb * 4) +
         moe::part_bytes(T, N, kb);
}

int moe_fp8_linear(const uint16_t* x, int64_t x_stride, int32_t T, int32_t K, const uint8_t* w, const void* w_scale,
                   int32_t scale_type, int32_t N, uint16_t* y, int64_t y_stride, void* ws, size_t ws_bytes,
                   void* stream) {
  if (T < 0) return MOE_EINVAL;
  if (!moe::shape_ok(T, N, K)) return MOE_ESHAPE;
  if (scale_type != MOE_SCALE_E8M0 && scale_type != MOE_SCALE_F32) return MOE_EINVAL;
  if (T == 0) return MOE_OK;
  if (!x || !w || !w_scale || !y || !ws) return MOE_EINVAL;
  if (x_stride < K || y_stride < N) return MOE_EINVAL;
  if (!moe::aligned(x, 16) || x_stride % 8 != 0 || !moe::aligned(w, 16) || !moe::aligned(y, 2) ||
      !moe::aligned(ws, 256) || (scale_type == MOE_SCALE_F32 && !moe::aligned(w_scale, 4)))
    return MOE_EALIGN;
  if (ws_bytes < moe_fp8_linear_workspace_size(T, N, K)) return MOE_EWORKSPACE;
  moe::LinearArgs a;
  a.x = x, a.x_stride = x_stride, a.y = y, a.y_stride = y_stride;
  a.w = w, a.w_scale = w_scale;
  a.T = T, a.N = N, a.K = K, a.kb = static_cast<int>(moe::ceil_div(K, 128));
  a.codes = static_cast<const uint8_t*>(ws);
  a.scales = reinterpret_cast<const uint32_t*>(a.codes + moe::align256(static_cast<size_t>(T) * a.kb * 128));
  a.part = reinterpret_cast<moe::f32x4*>(static_cast<char*>(ws) + moe::align256(static_cast<size_t>(T) * a.kb * 128) +
                                    moe::align256(static_cast<size_t>(T) * a.kb * 4));
  a.n_tiles = a.t_tiles = 0;
  a.splits = 1, a.chunk = a.kb;
  a.wide = y_stride % 4 == 0 && moe::aligned(y, 8);
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (scale_type == MOE_SCALE_F32)
    moe::launch<true>(a, s);
  else
    moe::launch<false>(a, s);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_EHIP;
}

}  // extern "C"
