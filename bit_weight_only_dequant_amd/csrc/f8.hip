// f8.hip - 8-bit floating point (E4M3) with an fp32 scale for blocks of 128:
// quantising, the product y = x . W^T, the two projections of a gated
// feed-forward block with its activation, and that block's backward pass.
// The format and the entry points are described in include/qgemm.h.
//
// Kernels (times in replayed graphs of 12 passes with the operands in the
// on-die cache)
//   f8_quantize_rows, f8_quantize_tiles, f8_dequantize
//                   bound by HBM: 8192 x 8192 fp32 in blocks of 128 x 128 67 us
//                   (5.0 TB/s; a large copy reaches 5.16), bf16 in blocks of 1
//                   42 us (4.8), turned over 49 us (4.1); read back to fp32 67.
//   f8_rows         few rows.  W goes from memory straight to registers, x
//                   through LDS; waves split K.  1 x 6144 x 2048 with fp16 x 6.3
//                   us, 8 x 2048 x 8192 with bf16 x and a residual 9.1, gate and
//                   up projection of 8192 features of one row 9.5 (of 60 passes,
//                   without the residual: 5.7, 8.2 and 8.7).
//   f8_tile         more rows.  x and W through a ring of LDS stages by direct
//                   loads; a stage of 128 k is one block of the scales.  8-bit
//                   x to bf16: 4096 x 8192 x 8192 256 to 265 us (2.1 PFLOP/s;
//                   the library's product with one scale reaches 2.7 to 2.8);
//                   bf16 x: 4096 x 2048 x 16384 240 us (1.15 PFLOP/s; the
//                   library's bf16 product reaches 1.33 to 1.40).
//   f8_no_k         a product without a k.
// A block's products are summed by the matrix cores and join the fp32 sum times
// the two scales, four multiply-adds and one product for 16 x 16 outputs and
// 128 k, under which the next products run.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <climits>
#include <type_traits>

#include "../../include/qgemm.h"
#include "device.h"
#include "internal.h"

namespace qg {
namespace {

typedef uint32_t u2 __attribute__((ext_vector_type(2)));

constexpr int F8 = QG_F8_E4M3;
constexpr float F8_TOP = 448.f;                 // the largest code
constexpr float F8_LOWEST = 0x1p-100f;          // a block's largest magnitude counts as at least this

// ---------------------------------------------------------------------------
// quantise
// ---------------------------------------------------------------------------
// Bound by HBM.  A code is the nearest to q = 448 v / A, A the block's largest
// magnitude, ties to the even one.  Quotients midway between two codes are
// common, so q has to be exact there.  v and A are taken times the power of two
// that makes A 1..2, so that nothing overflows; t is q rounded to 24 bits by
// one step of division (a product with 448 / A, then its remainder times 1 / A).
// Middles have at most 5 significant bits.  With 16-bit v the numerator 448 v
// is exact in fp32, and a quotient that is not a middle is further from any
// than t's rounding, so t decides.  With fp32 v the numerator takes two parts,
// and where t is a middle the sign of what is left tells the side.
struct F8Block { float inv, rcp, top; int shift; bool finite; };   // 448 / A, 1 / A, A, all at A's scale

__device__ __forceinline__ F8Block f8_block(uint32_t top_bits) {   // the bits of A
  F8Block b;
  b.finite = top_bits < 0x7f800000u;
  const uint32_t t = max(top_bits, f32_bits(F8_LOWEST));
  b.shift = 127 - (int)(t >> 23);
  b.top = bits_f32((t & 0x7fffffu) | 0x3f800000u);
  b.inv = F8_TOP / b.top;
  b.rcp = b.inv * (1.f / F8_TOP);
  return b;
}
__device__ __forceinline__ float f8_scale(uint32_t top_bits) {
  return top_bits < 0x7f800000u ? fmaxf(bits_f32(top_bits), F8_LOWEST) / F8_TOP : bits_f32(0x7fc00000u);
}

template <int T> __device__ __forceinline__ float f8_quotient(float v, const F8Block& b) {
  const float x = ldexpf(v, b.shift);
  const float h = F8_TOP * x;
  float t = x * b.inv;
  if constexpr (T != F32) return copysignf(fmaf(fmaf(-t, b.top, h), b.rcp, t), v);   // a zero keeps its sign
  const float l = fmaf(F8_TOP, x, -h);
  t = fmaf(fmaf(-t, b.top, h) + l, b.rcp, t);
  const float rest = fmaf(-t, b.top, h) + l;
  const uint32_t bits = f32_bits(t);
  if ((bits & 0x7ffffu) == 0 && rest != 0.f && t != 0.f) t = bits_f32((rest > 0.f) == (t > 0.f) ? bits + 1 : bits - 1);
  return copysignf(t, v);
}

// 4 codes, the first in the lowest byte
__device__ __forceinline__ uint32_t f8_codes(float a, float b, float c, float d) {
  int w = 0;
  w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, w, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// Largest of the 16 lanes of a row (quads, then the quads of a half, then the halves).
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  v = quad_max(v);
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xf, 0xf, true));          // row_half_mirror
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xf, 0xf, true));       // row_mirror
}

template <int T> __device__ __forceinline__ void load8_or_zero(const typename Elem<T>::type* p, bool have, float v[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.f;
  if (have) load8<T>(p, v);
}

// i / per, for i below n: in 32 bits where they hold it (a 64-bit division takes as long as a block's conversion).
__device__ __forceinline__ int64_t row_of(int64_t i, uint32_t per, int64_t n) {
  return n <= (int64_t)UINT32_MAX ? (int64_t)((uint32_t)i / per) : i / per;
}

// Blocks of 128 along a row: a lane takes 8 elements, 16 lanes a block (the
// last block of a row may have idle ones), so a wave's codes are 512 contiguous
// bytes.  n: 16-lane groups, kb of them a row.
template <int T>
__global__ __launch_bounds__(EW_THREADS) void f8_quantize_rows_kernel(const typename Elem<T>::type* __restrict__ x,
                                                                      int64_t ldx, int K, int kb, int64_t n,
                                                                      uint8_t* __restrict__ codes,
                                                                      float* __restrict__ scales) {
  const int64_t step = (int64_t)gridDim.x * (EW_THREADS / 16);
  const int lane = threadIdx.x & 15;
  for (int64_t i = (int64_t)blockIdx.x * (EW_THREADS / 16) + (threadIdx.x >> 4); i < n; i += step) {
    const int64_t r = row_of(i, kb, n);
    const int k = (int)(i - r * kb) * 128 + lane * 8;
    float v[8];
    load8_or_zero<T>(x + r * ldx + k, k < K, v);
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, f32_bits(v[j]) & 0x7fffffffu);
    top = row_max(top);
    const F8Block b = f8_block(top);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = f8_quotient<T>(v[j], b);
    const u2 c = {f8_codes(v[0], v[1], v[2], v[3]), f8_codes(v[4], v[5], v[6], v[7])};
    if (k < K) *reinterpret_cast<u2*>(codes + r * K + k) = b.finite ? c : u2{0, 0};
    if (lane == 0) scales[i] = f8_scale(top);
  }
}

// Reading back, 16 bytes of y a lane (4 codes for fp32, 8 for 16 bits): each value rounded once.  n: such groups,
// per of them a row; shift 0 or 7: rows of a block.  Bound by HBM.
template <int T>
__global__ __launch_bounds__(EW_THREADS) void f8_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                                   const float* __restrict__ scales, int shift, int kb,
                                                                   uint32_t per, int64_t n,
                                                                   typename Elem<T>::type* __restrict__ y, int64_t ldy) {
  typedef typename Elem<T>::type E;
  constexpr int C = 16 / sizeof(E);
  typedef E Out __attribute__((ext_vector_type(C)));
  const int64_t step = (int64_t)gridDim.x * EW_THREADS;
  for (int64_t i = (int64_t)blockIdx.x * EW_THREADS + threadIdx.x; i < n; i += step) {
    const int64_t r = row_of(i, per, n);
    const uint32_t k = (uint32_t)(i - r * per) * C;
    const float s = scales[(r >> shift) * kb + (k >> 7)];
    const uint32_t* from = reinterpret_cast<const uint32_t*>(codes) + i * (C / 4);
    Out v;
#pragma unroll
    for (int j = 0; j < C / 4; ++j) {
      const uint32_t w = from[j];
      const f2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
      v[4 * j] = (E)(a.x * s);
      v[4 * j + 1] = (E)(a.y * s);
      v[4 * j + 2] = (E)(b.x * s);
      v[4 * j + 3] = (E)(b.y * s);
    }
    *reinterpret_cast<Out*>(y + r * ldy + k) = v;
  }
}

// Tiles of 128 x 128: those whose block spans rows, and those that are turned
// over (8192 x 8192 bf16 47 to 49 us with blocks of 1, 46 with blocks of 128 x
// 128: the stores go out in pieces of 128 bytes).  A lane takes 8 columns of 4
// consecutive rows, so that 4 codes of a column are a word.  Largest magnitudes
// go from lane to lane over a wave's 16 rows and through LDS over the waves;
// turned codes go through LDS in rows of 33 words, and are stored 32 bytes a
// lane.  A wave's writes touch 32 of the 64 banks twice (the columns of lanes c8
// and c8 + 8 are 64 rows apart, a multiple of 64 words for any pitch), its reads
// 40 of them up to twice.  M rows of x; `wide` is the pitch of the turned codes,
// M rounded up to 16, zeros past M.
template <int T, bool BLOCK, bool TURN>
__global__ __launch_bounds__(512) void f8_quantize_tiles_kernel(const typename Elem<T>::type* __restrict__ x,
                                                                int64_t ldx, int M, int K, int wide,
                                                                uint8_t* __restrict__ codes,
                                                                float* __restrict__ scales) {
  constexpr int PITCH = 33;
  __shared__ uint32_t turned[TURN ? 128 * PITCH : 1];
  __shared__ uint32_t tops[8 * 128];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int c8 = tid & 15, r4 = tid >> 4;                     // columns 8 c8.., rows 4 r4..
  const int mb = blockIdx.y, kblk = blockIdx.x;
  const int k = kblk * 128 + c8 * 8, m = mb * 128 + r4 * 4;
  float v[4][8];
  uint32_t top[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) load8_or_zero<T>(x + (int64_t)(m + i) * ldx + k, k < K && m + i < M, v[i]);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    top[j] = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) top[j] = max(top[j], f32_bits(v[i][j]) & 0x7fffffffu);
  }
  uint32_t one = 0;
  if constexpr (BLOCK) {
#pragma unroll
    for (int j = 0; j < 8; ++j) one = max(one, top[j]);
    one = row_max(one);
    one = max(one, (uint32_t)__shfl_xor((int)one, 16));
    one = max(one, (uint32_t)__shfl_xor((int)one, 32));
    if (lane == 0) tops[wave] = one;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) one = max(one, tops[w]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      top[j] = max(top[j], (uint32_t)__shfl_xor((int)top[j], 16));
      top[j] = max(top[j], (uint32_t)__shfl_xor((int)top[j], 32));
      if (lane < 16) tops[wave * 128 + c8 * 8 + j] = top[j];
    }
    __syncthreads();
    if (tid < 128) {
      uint32_t t = tops[tid];
#pragma unroll
      for (int w = 1; w < 8; ++w) t = max(t, tops[w * 128 + tid]);
      tops[tid] = t;     // this lane alone reads and writes the column's first word here
    }
    __syncthreads();
  }
  F8Block b;
  if constexpr (BLOCK) b = f8_block(one);
  uint32_t word[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if constexpr (!BLOCK) b = f8_block(tops[c8 * 8 + j]);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i][j] = f8_quotient<T>(v[i][j], b);
    if constexpr (TURN) {
      word[j] = b.finite ? f8_codes(v[0][j], v[1][j], v[2][j], v[3][j]) : 0u;
      turned[(c8 * 8 + j) * PITCH + r4] = word[j];
    }
  }
  const int kbs = (K + 127) >> 7, mbs = (M + 127) >> 7;
  if constexpr (BLOCK) {
    if (tid == 0) scales[TURN ? (int64_t)kblk * mbs + mb : (int64_t)mb * kbs + kblk] = f8_scale(one);
  } else {
    if (tid < 128 && kblk * 128 + tid < K) scales[(int64_t)(kblk * 128 + tid) * mbs + mb] = f8_scale(tops[tid]);
  }
  if constexpr (!TURN) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const u2 c = {f8_codes(v[i][0], v[i][1], v[i][2], v[i][3]), f8_codes(v[i][4], v[i][5], v[i][6], v[i][7])};
      if (k < K && m + i < M) *reinterpret_cast<u2*>(codes + (int64_t)(m + i) * K + k) = b.finite ? c : u2{0, 0};
    }
  } else {
    __syncthreads();
    const int col = tid >> 2, part = tid & 3;
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = turned[col * PITCH + part * 8 + i];
    uint8_t* to = codes + (int64_t)(kblk * 128 + col) * wide + mb * 128 + part * 32;
    if (kblk * 128 + col < K) {
      if (mb * 128 + part * 32 < wide) *reinterpret_cast<u4*>(to) = u4{w[0], w[1], w[2], w[3]};
      if (mb * 128 + part * 32 + 16 < wide) *reinterpret_cast<u4*>(to + 16) = u4{w[4], w[5], w[6], w[7]};
    }
  }
}

// ---------------------------------------------------------------------------
// products
// ---------------------------------------------------------------------------
// What is done with the products: stored (with the residual), gated, or turned
// into the gradients of the two gated projections.
constexpr int PRODUCT = 0, GATED = 1, GRAD = 2;

struct F8Args {
  const char* x; const float* xs; const uint8_t* w; const float* ws;
  const char* resid; char* y;
  const char* dh;                   // GRAD: [M, F]
  int64_t ldx_bytes, ldr, ldy, ldd; // x row pitch in bytes, the others in elements
  int M, N, K, F;                   // N: columns of y; F: features of the gated forms
  int w_rows, kb;                   // rows of W, blocks of 128 along K
  int y_type, act;
};

// The gate's value g s(t) and its slope s + g s (1 - s) t', with the logistic
// function s and t = g (silu) or 2 sqrt(2 / pi) (g + 0.044715 g^3) (gelu in its
// tanh form: (1 + tanh z) / 2 is s(2 z)).  e = exp(-|t|) <= 1 gives s and 1 - s
// without overflow or cancellation.  Past |g| = 200 s (1 - s) is 0, and g is
// held there so that it does not meet an infinite factor.
struct Gate { float value, slope; };
__device__ __forceinline__ Gate gate(float g, int act) {
  constexpr float C = 1.5957691216057308f, D = 0.044715f;     // 2 sqrt(2 / pi)
  const float t = act == QG_ACT_SILU ? g : C * (g + D * g * g * g);
  const float e = __builtin_amdgcn_exp2f(-fabsf(t) * 1.4426950408889634f);
  const float r = __builtin_amdgcn_rcpf(1.f + e);
  const float s = t >= 0.f ? r : e * r, s1 = t >= 0.f ? e * r : r;
  const float h = fminf(fmaxf(g, -200.f), 200.f);
  const float dt = act == QG_ACT_SILU ? 1.f : C * (1.f + 3.f * D * h * h);
  return {g * s, s + h * (s * s1) * dt};
}

// C consecutive outputs at y, `have` of them (C or more: all), rounded once.
template <typename E, int C> __device__ __forceinline__ void put_rounded(E* y, int have, const float (&v)[C]) {
  E q[C];
#pragma unroll
  for (int i = 0; i < C; ++i) q[i] = (E)v[i];
  if (have >= C) put(y, q);
  else for (int i = 0; i < C; ++i) if (i < have) y[i] = q[i];
}

// What an output needs beside its sums, C columns (of a gated form: features) from n on of row m: the residual, or
// dh.  Zeros without one.
template <int MODE, int YT, int C>
__device__ __forceinline__ void load_beside(const F8Args& a, int m, int n, typename Elem<YT>::type (&e)[C]) {
  typedef typename Elem<YT>::type E;
#pragma unroll
  for (int i = 0; i < C; ++i) e[i] = (E)0.f;
  if (m >= a.M) return;
  if constexpr (MODE == GRAD) {
    if (n < a.F) get(reinterpret_cast<const E*>(a.dh) + (int64_t)m * a.ldd + n, e);
  } else if constexpr (MODE == PRODUCT) {
    if (!a.resid || n >= a.N) return;
    const E* p = reinterpret_cast<const E*>(a.resid) + (int64_t)m * a.ldr + n;
    if (n + C <= a.N) get(p, e);
    else for (int i = 0; i < C; ++i) if (i < a.N - n) e[i] = p[i];
  }
}

// Stores them: v the sums (of a gated form the gate's, u the other projection's), e what load_beside() gave.
template <int MODE, int YT, int C>
__device__ __forceinline__ void store_outputs(const F8Args& a, int m, int n, float (&v)[C], float (&u)[C],
                                              const typename Elem<YT>::type (&e)[C]) {
  typedef typename Elem<YT>::type E;
  E* const y = reinterpret_cast<E*>(a.y) + (int64_t)m * a.ldy + n;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    if constexpr (MODE == PRODUCT) {
      if (a.resid) v[i] += to_f32(e[i]);
    } else {
      const Gate g = gate(v[i], a.act);
      if constexpr (MODE == GATED) {
        v[i] = g.value * u[i];
      } else {
        const float dh = to_f32(e[i]);
        v[i] = dh * u[i] * g.slope;
        u[i] = dh * g.value;
      }
    }
  }
  put_rounded(y, MODE == PRODUCT ? a.N - n : C, v);
  if constexpr (MODE == GRAD) put_rounded(y + a.F, C, u);
}

template <int MODE, int YT>
__device__ __forceinline__ void store_four_as(const F8Args& a, int m, int n, float (&v)[4], float (&u)[4]) {
  typename Elem<YT>::type e[4];
  load_beside<MODE, YT, 4>(a, m, n, e);
  store_outputs<MODE, YT, 4>(a, m, n, v, u, e);
}
template <int MODE> __device__ __forceinline__ void store_four(const F8Args& a, int m, int n, float (&v)[4], float (&u)[4]) {
  if (a.y_type == F32) store_four_as<MODE, F32>(a, m, n, v, u);
  else if (a.y_type == F16) store_four_as<MODE, F16>(a, m, n, v, u);
  else store_four_as<MODE, BF16>(a, m, n, v, u);
}

// 8 codes -> 8 exact 16-bit values (E4M3 lies within fp16's and bf16's numbers)
__device__ __forceinline__ b8 f8_to_bf16(uint32_t lo, uint32_t hi) {
  const b2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false);
  const b2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true);
  const b2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false);
  const b2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true);
  return b8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}
__device__ __forceinline__ h8 f8_to_f16(uint32_t lo, uint32_t hi) {
  const h2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, false);
  const h2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, true);
  const h2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, false);
  const h2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, true);
  return h8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// 8 codes as 16-bit operands for x of type XT (codes: fp16).
template <int XT> __device__ __forceinline__ u4 f8_to_16(uint32_t lo, uint32_t hi) {
  if constexpr (XT == BF16) return __builtin_bit_cast(u4, f8_to_bf16(lo, hi));
  else return __builtin_bit_cast(u4, f8_to_f16(lo, hi));
}
// 16 x 16 outputs, 32 of k, 8 16-bit elements a lane.  Converted codes and
// their products are exact in fp32.
template <int XT> __device__ __forceinline__ f4 mfma_16(u4 w, u4 x, f4 c) {
  if constexpr (XT == BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, w), __builtin_bit_cast(b8, x), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, w), __builtin_bit_cast(h8, x), c, 0, 0, 0);
}

// LDS of a wave for a chunk of 512 k of x: whole direct loads of a kilobyte
// (two rows of codes, one 16-bit row)
template <int XT> __host__ __device__ constexpr int f8_x_bytes(int M) {
  const int rows = M < 16 ? M : 16;
  return 1024 * (XT == F8 ? (rows + 1) / 2 : rows);
}

// Few rows: bound by the weights' bytes.  A workgroup owns a block of 16 columns
// of y (rows of W; of a gated form 16 of the gate's and the same 16 of the
// other projection) and up to 16 rows of it; its NW waves take K's chunks of
// 512 in turn and are summed through LDS in wave order.  Lane l = 16 g + r of a
// wave loads the eight 16-byte pieces 4 u + g of a chunk of row r of W straight
// to registers and converts them there.  x goes straight to the wave's own LDS; row r keeps
// its piece c at place c ^ r, so 16 rows' reads touch the 64 banks once.  Each
// block of 128 has its own sum, which joins the others times its scales.  W is
// the first operand, so a lane ends with four consecutive outputs of one row.
// MULTI: a workgroup goes through several column blocks, or its waves through
// several chunks, the next weights on their way meanwhile.
template <int XT, int MODE, int NW, bool MULTI, bool ROWS>
__global__ __launch_bounds__(NW * 64) void f8_rows_kernel(F8Args a) {
  constexpr int NT = MODE == PRODUCT ? 1 : 2;
  constexpr int XC = XT == F8 ? 512 : 1024;       // bytes of an x row a chunk
  extern __shared__ __align__(1024) uint8_t rows_lds[];
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int np = a.K >> 4;                        // 16-byte pieces of a row of codes
  const int chunks = (np + 31) >> 5, turns = (chunks + NW - 1) / NW;   // (at least one) a wave's chunks: wave, wave + NW, ..
  const int blocks = MODE == PRODUCT ? (a.N + 15) >> 4 : a.F >> 4;
  const int m0 = blockIdx.y * 16, rows = min(a.M - m0, 16), rr = min(r, rows - 1);
  const int xbytes = f8_x_bytes<XT>(a.M);
  uint8_t* const xl = rows_lds + wave * xbytes;
  auto w_row = [&](int nb, int j) { return (MODE == PRODUCT ? 0 : j * a.F) + nb * 16; };   // a block's first row of W

  struct W { u4 c[NT][8]; };
  auto load_w = [&](int nb, int c, W& w) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const uint8_t* wp = a.w + (int64_t)min(w_row(nb, j) + r, a.w_rows - 1) * a.K;
#pragma unroll
      for (int u = 0; u < 8; ++u) w.c[j][u] = *reinterpret_cast<const u4*>(wp + (int64_t)min(c * 32 + 4 * u + g, np - 1) * 16);
    }
  };
  auto dma = [](const char* from, uint8_t* to) { __builtin_amdgcn_global_load_lds((gptr)from, (lptr)to, 16, 0, 0); };
  // x: a whole chunk of the rows there are (past K: a row's last piece again)
  auto load_x = [&](int c) {
    if constexpr (XT == F8) {
      for (int i = 0; i < rows; i += 2) {
        const int row = i + (lane >> 5);
        dma(a.x + (int64_t)(m0 + min(row, rows - 1)) * a.ldx_bytes + (int64_t)min(c * 32 + ((lane & 31) ^ row), np - 1) * 16,
            xl + i * XC);
      }
    } else {
      for (int i = 0; i < rows; ++i)
        dma(a.x + (int64_t)(m0 + i) * a.ldx_bytes + (int64_t)min(c * 64 + (lane ^ i), np * 2 - 1) * 16, xl + i * XC);
    }
  };
  // the scales of a chunk's four blocks: this lane's row of x, and the rows of
  // W behind its four outputs (one for all of them where a block has 128 rows)
  constexpr int SR = ROWS ? 4 : 1;
  struct S { float x[4], w[NT][SR][4]; };
  auto load_scales = [&](int nb, int c, S& s) {
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int kb = min(c * 4 + b, a.kb - 1);
      s.x[b] = XT == F8 ? a.xs[(int64_t)(m0 + rr) * a.kb + kb] : 1.f;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < SR; ++i) {
          const int64_t row = ROWS ? min(w_row(nb, j) + 4 * g + i, a.w_rows - 1) : w_row(nb, j) >> 7;
          s.w[j][i][b] = a.ws[row * a.kb + kb];
        }
    }
  };

  W w0, w1;
  S s;
  f4 acc[NT];
  int nb = blockIdx.x, turn = 0, buf = 0;
  // The first loads go out before anything that follows is begun (mixed with it: 1 x 6144 x 2048 5.75 us instead of 5.65).
  __builtin_amdgcn_sched_barrier(0);
  if (turns == 1 && wave < chunks) load_x(wave);
  load_w(nb, min(wave, chunks - 1), w0);
  __builtin_amdgcn_sched_barrier(0);
  // one chunk of one block: its products, and after a block's last chunk the sums
  auto item = [&](auto MORE, W& w, W& next) {   // MORE: another item follows
    const int c = wave + turn * NW;
    const bool last = turn + 1 >= turns;
    if (c < chunks) {
      load_scales(nb, c, s);
      if (turns > 1) load_x(c);
    }
    // The next item's weights (a wave without a chunk loads some).  All other loads are waited for: those stay on their way.
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (decltype(MORE)::value) {
      load_w(last ? nb + (int)gridDim.x : nb, min(last ? wave : c + NW, chunks - 1), next);
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      wait_loads<NT * 8>();
    } else {
      wait_loads<0>();
    }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    if (turn == 0) {
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[j] = f4{0.f, 0.f, 0.f, 0.f};
    }
    if (c < chunks) {
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        if (c * 32 + 8 * b >= np) break;
        u4 xv[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int p = 8 * b + 4 * h + g;
          const bool past = c * 32 + p >= np;   // zero operands
          if constexpr (XT == F8) {
            u4 v = *reinterpret_cast<const u4*>(xl + rr * XC + ((p ^ rr) * 16));
            if (past) v = u4{0, 0, 0, 0};
            xv[2 * h] = f8_to_16<XT>(v.x, v.y);
            xv[2 * h + 1] = f8_to_16<XT>(v.z, v.w);
          } else {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              xv[2 * h + q] = *reinterpret_cast<const u4*>(xl + rr * XC + (((2 * p + q) ^ rr) * 16));
              if (past) xv[2 * h + q] = u4{0, 0, 0, 0};
            }
          }
#pragma unroll
          for (int j = 0; j < NT; ++j)
            if (past) w.c[j][2 * b + h] = u4{0, 0, 0, 0};
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          f4 part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int q = 0; q < 4; ++q)
            part = mfma_16<XT>(f8_to_16<XT>(w.c[j][2 * b + q / 2][2 * (q & 1)], w.c[j][2 * b + q / 2][2 * (q & 1) + 1]), xv[q], part);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[j][i] = fmaf(part[i], s.x[b] * s.w[j][ROWS ? i : 0][b], acc[j][i]);
        }
      }
    }
    if (!last) {
      wait_lds();   // x has been read, its place may be sent for again
      asm volatile("" ::: "memory");
      ++turn;
      return;
    }
    // the waves' sums; two buffers, so one barrier a block does
    f4* part = reinterpret_cast<f4*>(rows_lds + NW * xbytes) + buf * (NW * NT * 64);
#pragma unroll
    for (int j = 0; j < NT; ++j) part[(wave * NT + j) * 64 + lane] = acc[j];
    lds_barrier();
    if (wave == buf % NW) {
      f4 v[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        v[j] = part[j * 64 + lane];
#pragma unroll
        for (int k = 1; k < NW; ++k) v[j] += part[(k * NT + j) * 64 + lane];
      }
      const int n = nb * 16 + 4 * g;
      if (r < rows && n < (MODE == PRODUCT ? a.N : a.F)) {
        float o[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
        float u[4] = {v[NT - 1].x, v[NT - 1].y, v[NT - 1].z, v[NT - 1].w};
        store_four<MODE>(a, m0 + r, n, o, u);
      }
    }
    buf ^= 1;
    turn = 0;
    nb += gridDim.x;
  };
  int left = nb < blocks ? ((blocks - 1 - nb) / (int)gridDim.x + 1) * turns : 0;
  if constexpr (MULTI) {
    for (; left > 2; left -= 2) {
      item(std::true_type{}, w0, w1);
      item(std::true_type{}, w1, w0);
    }
    if (left == 2) {
      item(std::true_type{}, w0, w1);
      item(std::false_type{}, w1, w0);
      left = 0;
    }
  }
  if (left == 1) item(std::false_type{}, w0, w1);
}

// ---------------------------------------------------------------------------
// more rows
// ---------------------------------------------------------------------------
// 16 x 16 outputs, 128 of k: both operands 32 codes a lane.  Any order of k is
// right as long as both follow it.  The matrix cores add the products of 8
// codes of a lane on a grid of 2^(e - 13), e the largest sum of two exponents
// among them, and cut what is finer (measured; whatever the instruction's
// shape): seven products of up to 2^(e - 13) each at most.  The rest of the sum
// is as exact as fp32.
__device__ __forceinline__ f4 mfma_f8(u4 a0, u4 a1, u4 b0, u4 b1) {
  const i8v a = {(int)a0.x, (int)a0.y, (int)a0.z, (int)a0.w, (int)a1.x, (int)a1.y, (int)a1.z, (int)a1.w};
  const i8v b = {(int)b0.x, (int)b0.y, (int)b0.z, (int)b0.w, (int)b1.x, (int)b1.y, (int)b1.z, (int)b1.w};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

// Which tile a workgroup has: numbered row tile fastest within blocks of 8 row
// tiles, a range of numbers to an XCD (workgroup b runs on XCD b % 8), so that
// tiles whose operands an XCD's L2 holds run together.
__device__ __forceinline__ bool f8_tile(int tiles_m, int tiles_n, int& tm, int& tn) {
  const int64_t total = (int64_t)tiles_m * tiles_n;
  const int xcd = blockIdx.x & 7;
  const int64_t id = total * xcd / 8 + (blockIdx.x >> 3);
  if (id >= total * (xcd + 1) / 8) return false;
  const int64_t per = (int64_t)8 * tiles_n;
  const int blk = (int)(id / per), in = (int)(id - blk * per);
  const int bm = min(8, tiles_m - blk * 8);
  tm = blk * 8 + in % bm;
  tn = in / bm;
  return true;
}

// Stores a wave's MI x NI blocks of 16 x 16 (lane 16 g + r: columns 4 g .. 4 g +
// 3 of row r) at row m0 and column (gated forms: feature) n0.  Each strip of 16 rows
// passes through LDS (the wave's own `strip`, rows padded by 16 bytes), so that
// a lane stores 8 consecutive outputs.  Gated forms have gate and other
// projection in turn, 16 features each.
// The residual's (or dh's) pieces of a strip are sent for two strips ahead.
template <int MODE, int YT, int MI, int NI>
__device__ __forceinline__ void f8_store_as(const F8Args& a, uint8_t* strip, int m0, int n0, const f4 (&acc)[MI][NI]) {
  typedef typename Elem<YT>::type E;
  constexpr int PITCH = 16 * NI + 4, PARTS = MODE == PRODUCT ? 1 : 2;
  constexpr int LANES = 2 * NI / PARTS, ROWS = 64 / LANES;   // lanes a row, rows at a time
  constexpr int PASSES = (16 + ROWS - 1) / ROWS;
  const int lane = threadIdx.x & 63, c = lane % LANES, n = n0 + c * 8;
  float* s = reinterpret_cast<float*>(strip);
  const float* from = s + (MODE == PRODUCT ? c * 8 : (c >> 1) * 32 + (c & 1) * 8);
  E beside[2][PASSES][8];
  auto load = [&](int i) {
#pragma unroll
    for (int p = 0; p < PASSES; ++p) load_beside<MODE, YT, 8>(a, m0 + i * 16 + p * ROWS + lane / LANES, n, beside[i & 1][p]);
  };
  load(0);
  load(1);
#pragma unroll
  for (int i = 0; i < MI; ++i) {
#pragma unroll
    for (int j = 0; j < NI; ++j) *reinterpret_cast<f4*>(s + (lane & 15) * PITCH + 16 * j + 4 * (lane >> 4)) = acc[i][j];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int r = p * ROWS + lane / LANES, m = m0 + i * 16 + r;
      if (r < 16 && m < a.M && n < (MODE == PRODUCT ? a.N : a.F)) {
        float v[8], u[8];
        __builtin_memcpy(v, from + r * PITCH, sizeof(v));
        __builtin_memcpy(u, from + r * PITCH + (MODE == PRODUCT ? 0 : 16), sizeof(u));
        store_outputs<MODE, YT, 8>(a, m, n, v, u, beside[i & 1][p]);
      }
    }
    if (i + 2 < MI) load(i + 2);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
}

// A buffer of `bytes` (below 2^31) from `base` on: loads past its end give zeros.
typedef __amdgpu_buffer_rsrc_t Buffer;
__device__ __forceinline__ Buffer f8_buffer(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00020000);
}
constexpr uint32_t PAST = 0x80000000u;   // an offset past every buffer's end

// x and W stream through a ring of RING LDS stages of 128 k: a workgroup of WM
// x WN waves, each MI x NI blocks of 16 x 16 outputs.  The loads go straight to
// LDS, RING stages ahead; a stage is one block of the scales, which come with
// it.  A row's 16-byte pieces change places by the row's number, so that the
// fragment reads touch the 64 banks evenly: rows of codes are 128 bytes (piece c
// at c ^ (row / 2 % 8)), 16-bit rows 256 (c ^ (row % 16)).  Pieces past K and
// rows past the last are zeros.  The one barrier a stage, before its last row of
// blocks, says both that everyone's loads of the next stage have arrived and
// that this one has been read: the next fragments of W and the first of x are
// read, and the loads of stage it + RING sent for, while that row is multiplied.
// FAST: 8-bit matrix instructions; else the codes are converted to 16 bits.
// KG: so many groups of WM x WN waves share a tile, group g taking every KG-th
// stage from the gth on in a ring of its own; their sums are added through LDS in
// the groups' order.  (A stage of a small tile is a chain of waits that a single
// group of waves cannot fill.)
// W is the first operand: a lane's outputs run along a row of y.
template <int XT, bool ROWS, int MI, int NI, int WM, int WN, int RING, int KG> constexpr int f8_tile_lds() {
  constexpr int TM = 16 * MI * WM, TN = 16 * NI * WN;
  return KG * RING * (TM * (XT == F8 ? 128 : 256) + TN * 128 + ((XT == F8 ? TM : 0) + (ROWS ? TN : 0)) * 4);
}
template <int XT, bool FAST, int MODE, bool ROWS, int MI, int NI, int WM, int WN, int RING, int KG>
__global__ __launch_bounds__(WM * WN * KG * 64) __attribute__((amdgpu_waves_per_eu(2))) void f8_tile_kernel(F8Args a, int tiles_m, int tiles_n) {
  constexpr int NW = WM * WN, TM = 16 * MI * WM, TN = 16 * NI * WN, TF = MODE == PRODUCT ? TN : TN / 2;
  constexpr bool C8 = XT == F8;
  constexpr int XB = C8 ? 128 : 256, XR = 1024 / XB;         // bytes of an x row a stage, rows a direct load brings
  constexpr int QA = TM / XR / NW, QB = TN / 8 / NW, QD = QA + QB;   // direct loads of 1 KiB a wave and stage
  static_assert(QA * XR * NW == TM && QB * 8 * NW == TN, "rows split evenly over the waves");
  // rows whose scales come with a stage: x's, and W's where each of its rows has its own (else they are the same for a
  // wave's 16 columns, and come by scalar loads a stage ahead)
  constexpr int SROWS = (C8 ? TM : 0) + (ROWS ? TN : 0), SOFF = C8 ? TM : 0;
  static_assert(SROWS % 64 == 0 && SOFF % 64 == 0, "a load brings the scales of 64 rows, of x or of W");
  constexpr int SL = SROWS / 64 > 0 ? SROWS / 64 : 1, QS = (SROWS / 64 + NW - 1) / NW, QALL = QD + QS;   // such loads, and a wave's
  constexpr bool WHOLE = MI * NI <= (FAST ? 16 : 8);   // a stage's fragments are read during the one before (below)
  constexpr int PIECES = TM * XB + TN * 128, STAGE = PIECES + SROWS * 4;
  static_assert(KG * RING * STAGE == f8_tile_lds<XT, ROWS, MI, NI, WM, WN, RING, KG>() && KG * RING * STAGE <= 160 * 1024, "LDS");
  static_assert(NW * 16 * (16 * NI + 4) * 4 <= RING * STAGE && (KG == 1 || 16 * (16 * NI + 4) <= MI * NI * 256),
                "the strips of f8_store_as: a wave's lies within its own part of the sums");
  // One array: with two, the compiler waits for every direct load before each read.  Its size is the launch's: where
  // the compiler sees that one workgroup fills a CU, it gives its waves accumulation registers too, and moves the
  // products out of them one by one.
  extern __shared__ __align__(1024) uint8_t smem[];
  int tm, tn;
  if (!f8_tile(tiles_m, tiles_n, tm, tn)) return;
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
  const int kg = KG == 1 ? 0 : __builtin_amdgcn_readfirstlane(tid >> 6) / NW;   // the wave's group, and its number there
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6) - kg * NW;
  const int wm = wave / WN, wn = wave % WN;
  const int m0 = tm * TM, n0 = tn * TF;                       // n0: first column, or feature
  const int stages = (a.kb + KG - 1) / KG;                    // of a group; stage `it` of it is block KG it + kg of K
  const uint32_t xpitch = (uint32_t)a.ldx_bytes, wpitch = (uint32_t)a.K;

  // The tile's rows as buffers (the host sees to it that a tile's rows stay below 2^31 bytes).  Row p of the
  // tile's W: of the gated forms 16 features of the gate, the same of the other projection, and so on; the two
  // have a buffer each.
  const int wrows = MODE == PRODUCT ? min(a.w_rows - n0, TN) : min(a.F - n0, TF);
  const Buffer xb = f8_buffer(a.x + (int64_t)m0 * a.ldx_bytes, (int64_t)min(a.M - m0, TM) * a.ldx_bytes);
  const uint8_t* const wbase = a.w + (int64_t)n0 * a.K;
  // Direct load q of a wave brings eight rows of codes (or four 16-bit rows), lane l a piece of the (l / 8)th.  The
  // piece's number depends on q by its parity only (16-bit rows: by q % 4), so offsets within a load are few and
  // the rest is the same for all lanes.
  constexpr int XV = C8 ? 2 : 4;
  int xpiece[XV], wpiece[2];
#pragma unroll
  for (int v = 0; v < XV; ++v)
    xpiece[v] = C8 ? (lane & 7) ^ ((v * 4 + (lane >> 4)) & 7) : (lane & 15) ^ ((v * 4 + (lane >> 4)) & 15);
#pragma unroll
  for (int v = 0; v < 2; ++v) wpiece[v] = (lane & 7) ^ ((v * 4 + (lane >> 4)) & 7);
  const uint32_t xlane = (lane / (64 / XR)) * xpitch, wlane = (lane >> 3) * wpitch;
  // scales: rows 64 n .. of the tile's x, then of its W (waves to spare bring the same rows again)
  const Buffer xsb = f8_buffer(C8 ? a.xs + (int64_t)m0 * a.kb : nullptr, C8 ? (int64_t)min(a.M - m0, TM) * a.kb * 4 : 0);
  const Buffer wsb = f8_buffer(ROWS ? a.ws + (int64_t)n0 * a.kb : nullptr, ROWS ? (int64_t)wrows * a.kb * 4 : 0);
  uint32_t soff[QS > 0 ? QS : 1];
#pragma unroll
  for (int q = 0; q < QS; ++q) {
    const int p = (wave * QS + q) % SL * 64 + lane;
    soff[q] = (uint32_t)(C8 && p < TM ? p : p - SOFF) * (uint32_t)a.kb * 4;
  }
  typedef const float __attribute__((address_space(4)))* Scalars;
  Scalars wsp[NI];
#pragma unroll
  for (int j = 0; j < NI; ++j) {
    const int q = wn * NI + j;
    const int row = MODE == PRODUCT ? min(n0 + q * 16, a.w_rows - 1) : (q & 1) * a.F + min(n0 + (q >> 1) * 16, a.F - 1);
    wsp[j] = (Scalars)(a.ws + (int64_t)(row >> 7) * a.kb);
  }
  // Load q of stage `it` into place `to`; past K zeros.  The rows are in the lanes' offsets and the scalar one lies within
  // a row, so that no row past the last makes it larger than the buffer.
  auto issue = [&](int it, uint8_t* to, int q) {
    it = it * KG + kg;
    const int left = a.K - it * 128;       // of K, for the pieces that lie past it
    const int along = left > 0 ? it : 0;
    if (q < QA) {
      const int n = wave * QA + q, v = (QA % XV == 0 ? q : n) % XV;
      const uint32_t at = xpiece[v] * (C8 ? 16 : 8) < left ? xlane + xpiece[v] * 16 + n * XR * xpitch : PAST;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(xb, (lptr)(to + n * 1024), 16, (int)at, along * XB, 0, 0);
    } else if (q < QD) {
      const int n = wave * QB + q - QA, v = (QB % 2 == 0 ? q - QA : n) % 2;
      const int half = MODE == PRODUCT ? 0 : n >> 1 & 1, row = MODE == PRODUCT ? n * 8 : (n >> 2) * 16 + (n & 1) * 8;
      const uint32_t at = wpiece[v] * 16 < left ? wlane + wpiece[v] * 16 + row * wpitch : PAST;
      const Buffer wb = f8_buffer(half ? wbase + (int64_t)a.F * a.K : wbase, (int64_t)wrows * a.K);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(wb, (lptr)(to + TM * XB + n * 1024), 16, (int)at, along * 128, 0, 0);
    } else {
      const int n = (wave * QS + q - QD) % SL;
      const uint32_t at = left > 0 ? soff[q - QD] : PAST;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(C8 && n * 64 < TM ? xsb : wsb, (lptr)(to + PIECES + n * 256), 4, (int)at, along * 4, 0, 0);
    }
  };
  auto barrier = [] {
    asm volatile("" ::: "memory");   // no LDS access moves across it
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  // fragments: lane 16 g + r reads pieces g and 4 + g of row r of codes, the same k of 16-bit rows.  (Next to each other
  // for next g: the 16 lanes whose reads go together are of two g, rows 0 .. 3 and 12 .. 15 of one and 4 .. 11 of the
  // other or the reverse, and with pieces 2 g and 2 g + 1 they met in half of the banks.)
  int foff[2], xoff[4];
#pragma unroll
  for (int h = 0; h < 2; ++h) foff[h] = r * 128 + (((4 * h + g) ^ (r >> 1 & 7)) * 16);
  const int xrow = wm * MI * 16 * XB, wrow = TM * XB + wn * NI * 2048;   // the wave's first rows in a stage
#pragma unroll
  for (int q = 0; q < 4; ++q) xoff[q] = r * 256 + (((8 * (q >> 1) + 2 * g + (q & 1)) ^ r) * 16);
  typedef std::conditional_t<ROWS, f4, float> F;
  // Two ways to have the fragments in time.  WHOLE: a stage's are all read while the one before is multiplied, where
  // registers hold two stages' of them.  Else x is read one row of blocks ahead, and the last row goes through its
  // blocks from HALF on and around: the fragments of the others, which it needs last, have a second place (`other`),
  // the later ones are read again as soon as it has used them.
  constexpr int HALF = NI / 2;
  auto block = [](int i, int s) { return !WHOLE && i == MI - 1 ? (s + HALF) % NI : s; };   // the block in turn s of row i
  u4 first[HALF][2], late[HALF][2], other[HALF][2];
  F ws[NI], ws_next[NI];   // W's scales (the first blocks join nothing, times these)
#pragma unroll
  for (int j = 0; j < NI; ++j) ws[j] = ws_next[j] = F{};
  // `at`: a stage's place in smem.  It is kept from the compiler where one lies (opaque()): it would hold every
  // fragment's address in a register of its own.
  auto opaque = [](int at) {
    asm volatile("" : "+s"(at));
    return at;
  };
  auto read_w = [&](int at, int j, u4 (&to)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) to[h] = *reinterpret_cast<const u4*>(smem + (at + wrow + foff[h]) + j * 2048);
  };
  auto read_ws = [&](int at, int it, F (&to)[NI]) {
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      if constexpr (ROWS) to[j] = *reinterpret_cast<const f4*>(smem + (at + PIECES + (SOFF + wn * NI * 16 + 4 * g) * 4) + j * 64);
      else to[j] = wsp[j][min(it * KG + kg, a.kb - 1)];
      if constexpr (!ROWS && KG > 1) to[j] = it * KG + kg < a.kb ? to[j] : 0.f;   // a stage past K adds nothing, whatever the last scale
    }
  };
  u4 x[2][C8 ? 2 : 4];
  float sx[2] = {1.f, 1.f};
  auto read_x = [&](int at, int i) {
#pragma unroll
    for (int h = 0; h < (C8 ? 2 : 4); ++h)
      x[i & 1][h] = *reinterpret_cast<const u4*>(smem + (at + xrow + (C8 ? foff[h & 1] : xoff[h])) + i * (16 * XB));
    if constexpr (C8) sx[i & 1] = *reinterpret_cast<const float*>(smem + (at + PIECES + (wm * MI * 16 + r) * 4) + i * 64);
  };
  f4 acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j) acc[i][j] = f4{0.f, 0.f, 0.f, 0.f};
  // A block's products join its sum LAG blocks later: the matrix cores' results take their time to come.  part, f:
  // the outstanding blocks' products and factors.
  constexpr int LAG = FAST ? 3 : NI, KEPT = FAST ? 4 : NI;
  static_assert(MI * NI % KEPT == 0, "the next stage's first block takes place 0 again");
  // LATE: W's row scales would take four registers a block with x's already in them; they are multiplied in when the
  // block joins, from the stage's own scales `s`.
  constexpr bool LATE = ROWS && !WHOLE;
  typedef std::conditional_t<LATE, float, F> Factor;
  f4 part[KEPT];
  Factor f[KEPT];
#pragma unroll
  for (int t = 0; t < KEPT; ++t) {
    part[t] = f4{0.f, 0.f, 0.f, 0.f};
    f[t] = Factor{};
  }
  auto join = [&](int t, const F (&s)[NI]) {   // block t (counted along the rows of blocks), t < 0: of the stage before
    const int at = (t + MI * NI) % (MI * NI), p = at % KEPT, i = at / NI, j = block(i, at % NI);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (LATE) acc[i][j][k] = fmaf(part[p][k], f[p] * s[j][k], acc[i][j][k]);
      else if constexpr (ROWS) acc[i][j][k] = fmaf(part[p][k], f[p][k], acc[i][j][k]);
      else acc[i][j][k] = fmaf(part[p][k], f[p], acc[i][j][k]);
    }
  };

  // Of a stage's loads the first EARLY are sent for in the last row of blocks, the others along the next stage's first
  // rows (where all is read ahead: all along the stage).  All in the last row make its waves wait to send: in turn on one
  // machine, warm from such runs (which take 255 to 265 us from rest), 4096 x 8192 x 8192 303 us instead of 290, gradients
  // of 4096 x 2048 -> 8192 196 instead of 188; with 16-bit x no difference (4096 x 2048 x 16384 238 to 245 either way).
  constexpr int EARLY = WHOLE ? QALL : C8 ? 4 : 6;
  static_assert(WHOLE || (EARLY <= QALL && (QALL - EARLY - 1) * 2 + 1 < (MI - 1) * NI), "the others are sent for in time");
#pragma unroll
  for (int it = 0; it < RING; ++it)
#pragma unroll
    for (int q = 0; q < (it < RING - 1 ? QALL : EARLY); ++q) issue(it, smem + kg * (RING * STAGE) + it * STAGE, q);
  wait_loads<(RING - 2) * QALL + EARLY>();
  barrier();
  const int ring = kg * (RING * STAGE);
  int cur = opaque(ring);   // the place of the stage at hand
  if constexpr (WHOLE) {
    constexpr int XP = C8 ? 2 : 4, READS = MI * XP + NI * 2;
    struct Frags { u4 x[MI][XP], w[NI][2]; float sx[MI]; F s[NI]; };
    auto read = [&](int at, Frags& f, int n) {   // read n of a stage's fragments
      if (n < NI * 2) {
        const int j = n / 2, h = n % 2;
        f.w[j][h] = *reinterpret_cast<const u4*>(smem + (at + wrow + foff[h]) + j * 2048);
      } else {
        const int i = (n - NI * 2) / XP, h = (n - NI * 2) % XP;
        f.x[i][h] = *reinterpret_cast<const u4*>(smem + (at + xrow + (C8 ? foff[h & 1] : xoff[h])) + i * (16 * XB));
        if (h == 0) f.sx[i] = C8 ? *reinterpret_cast<const float*>(smem + (at + PIECES + (wm * MI * 16 + r) * 4) + i * 64) : 1.f;
      }
    };
    auto stage = [&](int it, const Frags& c, Frags& next) {
      const int nxt = opaque(cur == ring + (RING - 1) * STAGE ? ring : cur + STAGE);
      wait_loads<(RING - 2) * QALL>();
      barrier();
      __builtin_amdgcn_sched_barrier(0);
      read_ws(nxt, it + 1, next.s);
      u4 half[FAST ? 1 : NI][4];
      if constexpr (!FAST) {
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) half[j][q] = f8_to_16<XT>(c.w[j][q >> 1][2 * (q & 1)], c.w[j][q >> 1][2 * (q & 1) + 1]);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        u4 xh[4];
        if constexpr (!FAST) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            xh[q] = C8 ? f8_to_16<XT>(c.x[i][q >> 1 & 1][2 * (q & 1)], c.x[i][q >> 1 & 1][2 * (q & 1) + 1]) : c.x[i][C8 ? 0 : q];
        }
        constexpr int Q = FAST ? 1 : 4;
#pragma unroll
        for (int q = 0; q < Q; ++q)
#pragma unroll
          for (int j = 0; j < NI; ++j) {
            const int t = i * NI + j, p = t % KEPT;
            if constexpr (FAST) {
              part[p] = mfma_f8(c.w[j][0], c.w[j][1], c.x[i][0], c.x[i][1]);
              join(t - LAG, c.s);
            } else {
              if (q == 0) join(t - LAG, c.s);
              part[p] = mfma_16<XT>(half[j][q], xh[q], q ? part[p] : f4{0.f, 0.f, 0.f, 0.f});
            }
            if (q == 0) f[p] = c.sx[i] * c.s[j];
            // the next stage's reads spread over the first half of the products, the loads over all of them: issued at
            // once they hold the wave up
            constexpr int SLOTS = MI * NI * Q;
            const int slot = (i * Q + q) * NI + j;
#pragma unroll
            for (int n = 0; n < READS; ++n)
              if (n * (SLOTS / 2) / READS == slot) read(nxt, next, n);
#pragma unroll
            for (int l = 0; l < QALL; ++l)
              if (l * SLOTS / QALL == slot) issue(it + RING, smem + cur, l);
            __builtin_amdgcn_sched_barrier(0);
          }
      }
      cur = nxt;
    };
    Frags f0, f1;
#pragma unroll
    for (int n = 0; n < READS; ++n) read(cur, f0, n);
    read_ws(cur, 0, f0.s);
    int it = 0;
#pragma unroll 1
    for (; it + 1 < stages; it += 2) {
      stage(it, f0, f1);
      stage(it + 1, f1, f0);
    }
    if (it < stages) stage(it, f0, f1);
  } else {
  read_x(cur, 0);
#pragma unroll
  for (int j = 0; j < NI; ++j) read_w(cur, j, j < HALF ? first[j] : late[j - HALF]);
  read_ws(cur, 0, ws);
  int before = ring + (RING - 1) * STAGE;   // and of the one before
  // early: the fragments of the first HALF blocks, late: those of the others; next: where the next stage's first ones go
  auto stage = [&](int it, u4 (&early)[HALF][2], u4 (&late)[HALF][2], u4 (&next)[HALF][2], F (&s)[NI], F (&s_next)[NI]) {
    const int nxt = opaque(cur == ring + (RING - 1) * STAGE ? ring : cur + STAGE);
    auto w = [&](int j) -> u4 (&)[2] { return j < HALF ? early[j] : late[j - HALF]; };
    u4 half[FAST ? 1 : NI][4];
    if constexpr (!FAST) {
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) half[j][q] = f8_to_16<XT>(w(j)[q >> 1][2 * (q & 1)], w(j)[q >> 1][2 * (q & 1) + 1]);
    }
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      if (i + 1 < MI) {
        read_x(cur, i + 1);
      } else {
        wait_loads<(RING - 2) * QALL>();
        barrier();
        __builtin_amdgcn_sched_barrier(0);
        read_x(nxt, 0);
#pragma unroll
        for (int j = 0; j < HALF; ++j) read_w(nxt, j, next[j]);
        read_ws(nxt, it + 1, s_next);
      }
      u4 xh[4];
      if constexpr (!FAST) {
#pragma unroll
        for (int q = 0; q < 4; ++q) xh[q] = C8 ? f8_to_16<XT>(x[i & 1][q >> 1 & 1][2 * (q & 1)], x[i & 1][q >> 1 & 1][2 * (q & 1) + 1]) : x[i & 1][C8 ? 0 : q];
      }
      constexpr int Q = FAST ? 1 : 4;
#pragma unroll
      for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int n = 0; n < NI; ++n) {
          const int t = i * NI + n, p = t % KEPT, j = block(i, n);
          if constexpr (FAST) {
            part[p] = mfma_f8(w(j)[0], w(j)[1], x[i & 1][0], x[i & 1][1]);
            join(t - LAG, t < LAG ? s_next : s);
          } else {
            if (q == 0) join(t - LAG, t < LAG ? s_next : s);   // (the stage before's scales are still in s_next)
            part[p] = mfma_16<XT>(half[j][q], xh[q], q ? part[p] : f4{0.f, 0.f, 0.f, 0.f});
          }
          if (q == 0) {
            if constexpr (LATE) f[p] = sx[i & 1];
            else f[p] = sx[i & 1] * s[j];
          }
          if (i < MI - 1 && q == 0) {
#pragma unroll
            for (int l = EARLY; l < QALL; ++l)
              if ((l - EARLY) * 2 + 1 == t) issue(it - 1 + RING, smem + before, l);
          }
          if (i == MI - 1 && q == Q - 1) {   // the loads spread over the row
#pragma unroll
            for (int l = 0; l < QALL; ++l)
              if (l < EARLY && l * NI / EARLY == n) issue(it + RING, smem + cur, l);
            if (j >= HALF) read_w(nxt, j, late[j - HALF]);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
    }
    before = cur;
    cur = nxt;
  };
  int it = 0;
#pragma unroll 1
  for (; it + 1 < stages; it += 2) {
    stage(it, first, late, other, ws, ws_next);
    stage(it + 1, other, late, first, ws_next, ws);
  }
  if (it < stages) stage(it, first, late, other, ws, ws_next);
  }
#pragma unroll
  for (int t = MI * NI - LAG; t < MI * NI; ++t) join(t - MI * NI, stages & 1 ? ws : ws_next);
  wait_loads<0>();   // nothing is on its way to LDS any more
  barrier();
  if constexpr (KG > 1) {
    static_assert((KG - 1) * TM * TN * 4 <= KG * RING * STAGE, "the other groups' sums");
    f4* const sums = reinterpret_cast<f4*>(smem) + wave * (MI * NI * 64) + lane;
    if (kg > 0) {
#pragma unroll
      for (int t = 0; t < MI * NI; ++t) sums[(kg - 1) * (TM * TN / 4) + t * 64] = acc[t / NI][t % NI];
    }
    wait_lds();
    barrier();
    if (kg > 0) return;
#pragma unroll
    for (int k = 0; k < KG - 1; ++k)
#pragma unroll
      for (int t = 0; t < MI * NI; ++t) acc[t / NI][t % NI] += sums[k * (TM * TN / 4) + t * 64];
  }
  // (of several groups the first one's waves alone are left: a wave reads its own sums before its strip takes their place)
  uint8_t* const strip = smem + wave * (KG > 1 ? MI * NI * 1024 : 16 * (16 * NI + 4) * 4);
  const int m = m0 + wm * MI * 16, n = n0 + wn * NI * (MODE == PRODUCT ? 16 : 8);
  if constexpr (FAST) {
    f8_store_as<MODE, BF16, MI, NI>(a, strip, m, n, acc);
  } else {
    if (a.y_type == F32) f8_store_as<MODE, F32, MI, NI>(a, strip, m, n, acc);
    else if (a.y_type == F16) f8_store_as<MODE, F16, MI, NI>(a, strip, m, n, acc);
    else f8_store_as<MODE, BF16, MI, NI>(a, strip, m, n, acc);
  }
}

// A product without a k, one output a lane (of the gated forms a feature): the residual, or what sums of zero give.
template <int MODE, int YT> __global__ __launch_bounds__(EW_THREADS) void f8_no_k_kernel(F8Args a) {
  typedef typename Elem<YT>::type E;
  const int cols = MODE == PRODUCT ? a.N : a.F;
  const int64_t step = (int64_t)gridDim.x * EW_THREADS, n = (int64_t)a.M * cols;
  for (int64_t i = (int64_t)blockIdx.x * EW_THREADS + threadIdx.x; i < n; i += step) {
    const int64_t row = i / cols, col = i - row * cols;
    E* const y = reinterpret_cast<E*>(a.y) + row * a.ldy + col;
    float v = 0.f;
    if (MODE == PRODUCT && a.resid) v += to_f32(reinterpret_cast<const E*>(a.resid)[row * a.ldr + col]);
    if (MODE == GRAD) y[a.F] = (E)(v = 0.f * to_f32(reinterpret_cast<const E*>(a.dh)[row * a.ldd + col]));
    y[0] = (E)v;
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// Which kernel takes a product.  tile 0: f8_rows_kernel with nw waves a workgroup (without a k f8_no_k_kernel); 1..5:
// f8_tile_kernel on F8_TILES.  QF8_TILE=0..5 in the environment forces one where there is a choice, with a k and rows
// of x of up to 4 MiB (tests, tuning).  fits: whether a grid holds it.
struct F8Plan { int tile, nw; int64_t workgroups; bool fits; };

// What the tiles multiply with: 16-bit x, 8-bit x on converted codes, 8-bit x as it is.
enum { KIND_16 = 0, KIND_EXACT = 1, KIND_FAST = 2 };

// The rule is a model of the time in nanoseconds, fitted to what the kernels took in replayed graphs (40 random shapes of
// 1..4096 rows and 8 chosen ones, plain and gated, of each kind; on 40 other random ones what it picks is 0.4 to 1.4 %
// behind the best).  A tile's stage of 128 k takes `alone` when its CU runs one tile and `shared` for each of the CU's
// tiles when the chip is full; `start` is a tile's first loads and stores, of which the share `more` shows again for every
// further tile of the CU.  The rows kernel takes 1.3 to 1.9 for a block of 16 x 16 outputs and chunk of 512 k, over the
// whole chip.  For instance 8-bit x to bf16: 383 x 2048 x 4128 on 64 x 64 tiles 15.9 us, on 128 x 128 27; 4096 x 8192 x
// 8192 on 256 x 256 255 to 265, on 128 x 128 403 to 420.  The last tile is the first with two groups of waves: 128 x 2048
// x 8192 with bf16 x 24.5 us, with one group 33 to 34; where there are several tiles for a CU they only cost.  Tiles of
// 64 x 128 and 128 x 128 with two groups were built too and never paid.
struct F8Tile { int rows, cols, groups, waves; double alone, shared, start, more; };   // waves: of a group
constexpr F8Tile F8_TILES[3][5] = {
    {{64, 64, 1, 4, 475, 364, 3760, 0.39}, {64, 128, 1, 4, 900, 582, 3560, 0.54}, {128, 128, 1, 8, 848, 844, 4800, 1.31},
     {128, 256, 1, 8, 1455, 1455, 5810, 1.92}, {64, 64, 2, 4, 499, 695, 4550, 0.70}},
    {{64, 64, 1, 4, 468, 382, 3800, 0.35}, {64, 128, 1, 4, 676, 480, 4110, 0.49}, {128, 128, 1, 8, 988, 988, 5200, 1.42},
     {128, 256, 1, 8, 1940, 1580, 6010, 2.68}, {64, 64, 2, 4, 507, 703, 4490, 0.77}},
    {{64, 64, 1, 4, 276, 276, 3650, 0.28}, {64, 128, 1, 4, 388, 388, 3490, 0.37}, {128, 128, 1, 4, 639, 729, 5200, 0.84},
     {256, 256, 1, 8, 1406, 1406, 7650, 0.27}, {64, 64, 2, 4, 327, 527, 4050, 0.72}}};

int64_t f8_pieces(int64_t M, int64_t w_rows, const F8Tile& t) {
  return (M + t.rows - 1) / t.rows * ((w_rows + t.cols - 1) / t.cols);
}
int64_t f8_grid(int64_t M, int64_t w_rows, const F8Tile& t) { return (f8_pieces(M, w_rows, t) + 7) / 8 * 8; }

// N: columns of y, or features of a gated form.  pitch: bytes from one row of x to the next.
F8Plan plan_f8(int mode, int M, int N, int K, int64_t pitch, int kind) {
  F8Plan p = {0, 1, 0, true};
  if (M == 0 || N == 0) return p;
  const int64_t chunks = ((int64_t)K + 511) / 512, stages = ((int64_t)K + 127) / 128;
  const int64_t w_rows = mode == PRODUCT ? N : 2 * (int64_t)N, row_tiles = ((int64_t)M + 15) / 16;
  // The tiles' buffers hold 256 rows of codes, or 128 of 16-bit x, in less than 2^31 bytes.  A larger pitch is the rows kernel's.
  if (K > 0 && pitch <= (1 << 22)) {
    double best = 3200 + (1.25 + 0.04 * std::min(M, 16)) * (double)(row_tiles * ((w_rows + 15) / 16) * chunks) + 120 * (double)chunks;
    if (row_tiles > 65535) best = 1e300;   // the rows kernel's grid
    for (int i = 0; i < 5; ++i) {
      const F8Tile& t = F8_TILES[kind][i];
      const double turns = (double)((f8_pieces(M, w_rows, t) + 255) / 256);
      const double cost = (double)((stages + t.groups - 1) / t.groups) * std::max(t.alone, t.shared * turns) +
                          t.start * (1 + t.more * (turns - 1));
      if (cost < best) best = cost, p.tile = i + 1;
    }
    const int forced = env_int("QF8_TILE", -1);
    if (forced >= 0 && forced <= 5) p.tile = forced;
  }
  if (p.tile) {
    const F8Tile& t = F8_TILES[kind][p.tile - 1];
    p.nw = 0;
    p.workgroups = f8_pieces(M, w_rows, t);
    p.fits = f8_grid(M, w_rows, t) * t.waves * t.groups * 64 <= (int64_t)UINT32_MAX;
    return p;
  }
  // a wave for every chunk, as far as LDS holds x and the sums for them
  p.nw = chunks <= 1 ? 1 : chunks <= 2 ? 2 : chunks <= 4 ? 4 : chunks <= 8 ? 8 : 16;
  const int rows = std::min(M, 16), nt = mode == PRODUCT ? 1 : 2;
  while (p.nw * ((kind != KIND_16 ? (rows + 1) / 2 : rows) + 2 * nt) > 160) p.nw /= 2;
  p.workgroups = row_tiles * (((int64_t)N + 15) / 16);
  // 16 waves have 128 registers each: enough for one chunk a wave and one block a workgroup, not for the next ones' weights
  if (p.nw == 16 && (chunks > 16 || p.workgroups > 256 * 2)) p.nw = 8;
  p.fits = K == 0 || row_tiles <= 65535;   // without a k an elementwise kernel takes it
  return p;
}

template <int XT, int MODE, int NW, bool ROWS> void launch_rows(const F8Args& a, hipStream_t s) {
  constexpr int NT = MODE == PRODUCT ? 1 : 2;
  const int64_t gy = ((int64_t)a.M + 15) / 16;
  const size_t lds = (size_t)NW * f8_x_bytes<XT>(a.M) + 2 * NW * NT * 1024;
  // column blocks a workgroup takes: no more workgroups than keep 32 waves on every CU
  const int64_t blocks = MODE == PRODUCT ? ((int64_t)a.N + 15) / 16 : a.F / 16;
  const int64_t slots = 256 * 32 / NW, share = (blocks * gy + slots - 1) / slots;
  const dim3 grid((unsigned)((blocks + share - 1) / share), (unsigned)gy);
  if constexpr (NW <= 8) {
    if (share > 1 || a.K > 512 * NW) {
      hipLaunchKernelGGL((f8_rows_kernel<XT, MODE, NW, true, ROWS>), grid, dim3(NW * 64), lds, s, a);
      return;
    }
  }
  hipLaunchKernelGGL((f8_rows_kernel<XT, MODE, NW, false, ROWS>), grid, dim3(NW * 64), lds, s, a);
}

template <int XT, bool FAST, int MODE, bool ROWS, int TILE, int MI, int NI, int WM, int WN, int RING>
void launch_tiles(const F8Args& a, hipStream_t s) {
  constexpr F8Tile t = F8_TILES[FAST ? KIND_FAST : XT == F8 ? KIND_EXACT : KIND_16][TILE - 1];
  static_assert(t.rows == 16 * MI * WM && t.cols == 16 * NI * WN && t.waves == WM * WN, "as planned");
  constexpr size_t lds = f8_tile_lds<XT, ROWS, MI, NI, WM, WN, RING, t.groups>();
  const dim3 grid((unsigned)f8_grid(a.M, a.w_rows, t));
  hipLaunchKernelGGL((f8_tile_kernel<XT, FAST, MODE, ROWS, MI, NI, WM, WN, RING, t.groups>), grid, dim3(t.waves * t.groups * 64),
                     lds, s, a, (a.M + t.rows - 1) / t.rows, (int)(((int64_t)a.w_rows + t.cols - 1) / t.cols));
}

template <int XT, bool FAST, int MODE, bool ROWS> void launch_f8(const F8Args& a, const F8Plan& p, hipStream_t s) {
  if (p.tile == 1) return launch_tiles<XT, FAST, MODE, ROWS, 1, 2, 2, 2, 2, XT == F8 ? 4 : 3>(a, s);
  if (p.tile == 2) return launch_tiles<XT, FAST, MODE, ROWS, 2, 2, 4, 2, 2, XT == F8 ? 3 : 2>(a, s);
  if (p.tile == 5) return launch_tiles<XT, FAST, MODE, ROWS, 5, 2, 2, 2, 2, XT == F8 ? 4 : 3>(a, s);
  if constexpr (FAST) {
    if (p.tile == 3) return launch_tiles<XT, FAST, MODE, ROWS, 3, 4, 4, 2, 2, 4>(a, s);
    if (p.tile == 4) return launch_tiles<XT, FAST, MODE, ROWS, 4, 8, 4, 2, 4, 2>(a, s);
  } else {
    if (p.tile == 3) return launch_tiles<XT, FAST, MODE, ROWS, 3, 4, 2, 2, 4, XT == F8 ? 4 : 3>(a, s);
    if (p.tile == 4) return launch_tiles<XT, FAST, MODE, ROWS, 4, 4, 4, 2, 4, XT == F8 ? 3 : 2>(a, s);
  }
  if constexpr (!FAST) {
    if (p.nw == 1) return launch_rows<XT, MODE, 1, ROWS>(a, s);
    if (p.nw == 2) return launch_rows<XT, MODE, 2, ROWS>(a, s);
    if (p.nw == 4) return launch_rows<XT, MODE, 4, ROWS>(a, s);
    if (p.nw == 8) return launch_rows<XT, MODE, 8, ROWS>(a, s);
    return launch_rows<XT, MODE, 16, ROWS>(a, s);
  }
}

// The 8-bit matrix instructions cut a sum of 8 products (see mfma_f8) by up to 7 * 2^-13 of the largest: less than half
// a step of bf16 (2^-8) of that product, and about a tenth of a result's rounding with random operands, though not
// where large products cancel.  So bf16 results alone take them: 4096 x 8192 x 8192 takes 265 us with them and 486 with
// converted codes.  fp16 and fp32 results, and products of blocks of 1 (weights' gradients), take converted codes, whose
// sums are as exact as fp32.
int f8_kind(int x_type, int y_type, int w_block) {
  return x_type != F8 ? KIND_16 : y_type == BF16 && w_block == 128 ? KIND_FAST : KIND_EXACT;
}

template <int MODE> int run_f8(const F8Args& a, int x_type, int w_block, void* stream) {
  const int kind = f8_kind(x_type, a.y_type, w_block);
  const F8Plan p = plan_f8(MODE, a.M, MODE == PRODUCT ? a.N : a.F, a.K, a.ldx_bytes, kind);
  if (!p.fits) return QG_E_UNSUPPORTED;
  int st = device_present();
  if (st != QG_OK) return st;
  const void* ptrs[7] = {a.x, a.xs, a.w, a.ws, a.resid, a.dh, a.y};
  st = check_device_pointers(ptrs, 7);
  if (st != QG_OK) return st;
  clear_pending_error();
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (a.K == 0) {
    const dim3 grid = ew_grid(1, (int64_t)a.M * (MODE == PRODUCT ? a.N : a.F)), block(EW_THREADS);
    if (a.y_type == F32) hipLaunchKernelGGL((f8_no_k_kernel<MODE, F32>), grid, block, 0, s, a);
    else if (a.y_type == F16) hipLaunchKernelGGL((f8_no_k_kernel<MODE, F16>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((f8_no_k_kernel<MODE, BF16>), grid, block, 0, s, a);
    return launch_status();
  }
  if constexpr (MODE == PRODUCT) {
    if (w_block == 1) {
      launch_f8<F8, false, MODE, true>(a, p, s);
      return launch_status();
    }
  }
  if (x_type == BF16) launch_f8<BF16, false, MODE, false>(a, p, s);
  else if (x_type == F16) launch_f8<F16, false, MODE, false>(a, p, s);
  else if (kind == KIND_FAST && p.tile) launch_f8<F8, true, MODE, false>(a, p, s);
  else launch_f8<F8, false, MODE, false>(a, p, s);
  return launch_status();
}

// Checks shared by the three products; fills the fields that all use.  N: the
// columns of y, w_rows: the rows of W.
int setup_f8(const void* x, int ldx, int x_type, const float* xs, const uint8_t* w, const float* ws, int w_block, int M,
             int N, int w_rows, int K, void* y, int ldy, int y_type, F8Args* a) {
  if (x_type != F16 && x_type != BF16 && x_type != F8) return QG_E_ARG;
  if (!float_type(y_type) || M < 0 || N < 0 || K < 0 || K % 16) return QG_E_ARG;
  if ((w_block != 1 && w_block != 128) || (w_block == 1 && x_type != F8)) return QG_E_ARG;
  if (M == 0 || N == 0) return QG_OK;
  if (M > INT_MAX - 512 || w_rows > INT_MAX - 512 || K > INT_MAX - 512) return QG_E_UNSUPPORTED;   // the kernels round them up in 32 bits
  if (!y || ldy < N) return QG_E_ARG;
  if (K > 0) {
    if (!x || !w || !ws || (x_type == F8) != (xs != nullptr)) return QG_E_ARG;
    if (x_type == F8 ? ldx != K : ldx < K) return QG_E_ARG;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(ws, 4) || !aligned(xs, 4) || ldx % 8) return QG_E_ALIGN;
  }
  if (!aligned(y, 16)) return QG_E_ALIGN;
  *a = F8Args{};
  a->x = reinterpret_cast<const char*>(x);
  a->xs = xs; a->w = w; a->ws = ws;
  a->ldx_bytes = (int64_t)ldx * (x_type == F8 ? 1 : 2);
  a->M = M; a->N = N; a->K = K; a->w_rows = w_rows; a->kb = (K + 127) / 128;
  a->y = reinterpret_cast<char*>(y);
  a->ldy = ldy; a->y_type = y_type;
  return QG_OK;
}

int check_act(int act, int F) { return (act == QG_ACT_SILU || act == QG_ACT_GELU_TANH) && F >= 0 && F % 16 == 0 && F <= INT_MAX / 2 - 512 ? QG_OK : QG_E_ARG; }

template <int T>
void launch_quantize(const void* v, int ldx, int M, int K, int block, bool turn, uint8_t* codes, float* scales, hipStream_t s) {
  typedef typename Elem<T>::type E;
  const E* x = reinterpret_cast<const E*>(v);
  const int kb = (K + 127) / 128;
  if (block == 1 && !turn) {
    const int64_t n = (int64_t)M * kb;
    const dim3 grid((unsigned)std::min<int64_t>((n + EW_THREADS / 16 - 1) / (EW_THREADS / 16), 256 * 16));
    hipLaunchKernelGGL(f8_quantize_rows_kernel<T>, grid, dim3(EW_THREADS), 0, s, x, (int64_t)ldx, K, kb, n, codes, scales);
    return;
  }
  const dim3 grid((unsigned)kb, (unsigned)(((int64_t)M + 127) / 128)), threads(512);
  const int wide = (M + 15) / 16 * 16;
  if (!turn) hipLaunchKernelGGL((f8_quantize_tiles_kernel<T, true, false>), grid, threads, 0, s, x, (int64_t)ldx, M, K, wide, codes, scales);
  else if (block == 1) hipLaunchKernelGGL((f8_quantize_tiles_kernel<T, false, true>), grid, threads, 0, s, x, (int64_t)ldx, M, K, wide, codes, scales);
  else hipLaunchKernelGGL((f8_quantize_tiles_kernel<T, true, true>), grid, threads, 0, s, x, (int64_t)ldx, M, K, wide, codes, scales);
}

}  // namespace
}  // namespace qg

using namespace qg;

extern "C" int qf8_plan(int gated, int M, int N, int K, int x_type, int y_type, int w_block, int out[3]) {
  if ((gated != 0 && gated != 1) || M < 0 || N < 0 || K < 0 || K % 16 || (x_type != F16 && x_type != BF16 && x_type != F8) ||
      !float_type(y_type) || (w_block != 1 && w_block != 128) || (w_block == 1 && x_type != F8) || (gated && N % 16) || !out)
    return QG_E_ARG;
  if (M > INT_MAX - 512 || N > (gated ? INT_MAX / 2 : INT_MAX) - 512 || K > INT_MAX - 512) return QG_E_UNSUPPORTED;
  const F8Plan p = plan_f8(gated ? GATED : PRODUCT, M, N, K, (int64_t)K * (x_type == F8 ? 1 : 2), f8_kind(x_type, y_type, w_block));
  out[0] = p.tile;
  out[1] = p.nw;
  out[2] = (int)std::min<int64_t>(p.workgroups, INT_MAX);
  return QG_OK;
}

extern "C" int qf8_quantize(const void* x, int ldx, int x_type, int M, int K, int block, int transpose, uint8_t* codes,
                            float* scales, void* stream) {
  if (!float_type(x_type) || M < 0 || K < 0 || K % 16 || (block != 1 && block != 128) || (transpose != 0 && transpose != 1))
    return QG_E_ARG;
  if (M == 0 || K == 0) return QG_OK;
  if (!x || !codes || !scales || ldx < K) return QG_E_ARG;
  if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 4) || ldx % 8) return QG_E_ALIGN;
  if (M > INT_MAX - 512 || K > INT_MAX - 512) return QG_E_UNSUPPORTED;
  if ((block != 1 || transpose) && (M > 65535 * 128 || K > (1 << 30) - 128)) return QG_E_UNSUPPORTED;   // the tiles' grid
  int st = device_present();
  if (st != QG_OK) return st;
  const void* ptrs[3] = {x, codes, scales};
  st = check_device_pointers(ptrs, 3);
  if (st != QG_OK) return st;
  clear_pending_error();
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (x_type == F16) launch_quantize<F16>(x, ldx, M, K, block, transpose, codes, scales, s);
  else if (x_type == BF16) launch_quantize<BF16>(x, ldx, M, K, block, transpose, codes, scales, s);
  else launch_quantize<F32>(x, ldx, M, K, block, transpose, codes, scales, s);
  return launch_status();
}

extern "C" int qf8_dequantize(const uint8_t* codes, const float* scales, int block, int M, int K, void* y, int ldy,
                              int y_type, void* stream) {
  if (!float_type(y_type) || M < 0 || K < 0 || K % 16 || (block != 1 && block != 128)) return QG_E_ARG;
  if (M == 0 || K == 0) return QG_OK;
  if (!y || !codes || !scales || ldy < K) return QG_E_ARG;
  if (!aligned(y, 16) || !aligned(codes, 16) || !aligned(scales, 4) || ldy % 8) return QG_E_ALIGN;
  int st = device_present();
  if (st != QG_OK) return st;
  const void* ptrs[3] = {codes, scales, y};
  st = check_device_pointers(ptrs, 3);
  if (st != QG_OK) return st;
  clear_pending_error();
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const uint32_t per = y_type == F32 ? K / 4 : K / 8;
  const int64_t n = (int64_t)M * per;
  const int shift = block == 1 ? 0 : 7, kb = (int)(((int64_t)K + 127) / 128);
  const dim3 grid((unsigned)std::min<int64_t>((n + EW_THREADS - 1) / EW_THREADS, 256 * 16)), threads(EW_THREADS);
  if (y_type == F16)
    hipLaunchKernelGGL(f8_dequantize_kernel<F16>, grid, threads, 0, s, codes, scales, shift, kb, per, n, reinterpret_cast<f16*>(y), (int64_t)ldy);
  else if (y_type == BF16)
    hipLaunchKernelGGL(f8_dequantize_kernel<BF16>, grid, threads, 0, s, codes, scales, shift, kb, per, n, reinterpret_cast<bf16*>(y), (int64_t)ldy);
  else
    hipLaunchKernelGGL(f8_dequantize_kernel<F32>, grid, threads, 0, s, codes, scales, shift, kb, per, n, reinterpret_cast<float*>(y), (int64_t)ldy);
  return launch_status();
}

extern "C" int qf8_gemm(const void* x, int ldx, int x_type, const float* x_scales, const uint8_t* w, const float* w_scales,
                        int w_block, const void* residual, int ldr, int M, int N, int K, void* y, int ldy, int y_type,
                        void* stream) {
  F8Args a;
  int st = setup_f8(x, ldx, x_type, x_scales, w, w_scales, w_block, M, N, N, K, y, ldy, y_type, &a);
  if (st != QG_OK) return st;
  if (M == 0 || N == 0) return QG_OK;
  if (residual) {
    if (ldr < N || (residual == y && ldr != ldy)) return QG_E_ARG;
    if (!aligned(residual, 16)) return QG_E_ALIGN;
    a.resid = reinterpret_cast<const char*>(residual);
    a.ldr = ldr;
  }
  return run_f8<PRODUCT>(a, x_type, w_block, stream);
}

extern "C" int qf8_gated(const void* x, int ldx, int x_type, const float* x_scales, const uint8_t* w, const float* w_scales,
                         int act, int M, int F, int K, void* h, int ldh, int h_type, void* stream) {
  F8Args a;
  int st = check_act(act, F);
  if (st == QG_OK) st = setup_f8(x, ldx, x_type, x_scales, w, w_scales, 128, M, F, 2 * F, K, h, ldh, h_type, &a);
  if (st != QG_OK) return st;
  if (M == 0 || F == 0) return QG_OK;
  a.F = F;
  a.act = act;
  return run_f8<GATED>(a, x_type, 128, stream);
}

extern "C" int qf8_gated_grad(const void* dh, int lddh, const void* x, int ldx, int x_type, const float* x_scales,
                              const uint8_t* w, const float* w_scales, int act, int M, int F, int K, void* d, int ldd,
                              int d_type, void* stream) {
  F8Args a;
  int st = check_act(act, F);
  if (st == QG_OK) st = setup_f8(x, ldx, x_type, x_scales, w, w_scales, 128, M, 2 * F, 2 * F, K, d, ldd, d_type, &a);
  if (st != QG_OK) return st;
  if (M == 0 || F == 0) return QG_OK;
  if (!dh || lddh < F || dh == d) return QG_E_ARG;
  if (!aligned(dh, 16)) return QG_E_ALIGN;
  a.F = F;
  a.act = act;
  a.dh = reinterpret_cast<const char*>(dh);
  a.ldd = lddh;
  return run_f8<GRAD>(a, x_type, 128, stream);
}
