// mx.hip - microscaled 4-bit floating point (MXFP4): quantising and reading
// back, the product y = x . W^T with MXFP4 weights, and that product grouped
// by expert with ragged sizes.  The format and the entry points are described
// in include/qgemm.h.
//
// Kernels
//   mx_quantize, mx_dequantize   elementwise, HBM-bound; the device's own fp4
//                        conversions (round to nearest even, saturating).
//                        8192 x 8192 bf16 there and back: 61 us, 5.0 TB/s
//                        of 304 MB (a large copy reaches 5.14).
//   mx_rows              few rows.  W and its scales go from memory straight to
//                        the matrix instruction's registers in their stored
//                        order, x through LDS; waves split K.  1 x 6144 x 2048
//                        with fp16 x 4.8 us, 8 x 2048 x 8192 with bf16 x 7.1 to
//                        7.7 us, 1 x 8192 x 8192 with bf16 x 10.1 us (3.5 TB/s),
//                        each in a replayed graph with the operands in the
//                        on-die cache; evicted 5.7, 8.1 to 8.4 and 10.8 us.
//   mx_tile              more rows.  x and W through a ring of LDS stages by
//                        direct loads.  MXFP4 x: 4096 x 8192 x 8192 138 to 142 us
//                        (3.9 PFLOP/s), evicted 157 to 166; bf16 x: 2048 x 8192 x
//                        8192 216 us (1.27 PFLOP/s; the library's bf16 product
//                        reaches 1.39), evicted 249.
//   mx_no_k              a product without a k: the residual, or zeros.
// The stored form needs no packing step: 16 consecutive bytes of a row are one
// block of 32, which is what one lane supplies to v_mfma_scale_f32_16x16x128 and
// 32x32x64 (fp4 operands, one scale byte a lane), so the products read
// checkpoints' own layout.
// Precision.  MXFP4 values meet 16-bit x exactly: code times scale is an exact
// bf16 number below 2^128 (subnormal for the smallest scales), so bf16 x uses bf16 matrix instructions and loses nothing; with
// fp16 x it is an exact fp16 number for scales of 2^-23 .. 2^8, and where a wave
// meets others it multiplies bf16 weights with x split in two exact bf16 parts.
// Sums are fp32; the one rounding is at the store.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <type_traits>

#include "../../include/qgemm.h"
#include "internal.h"

namespace qg {
namespace {

typedef _Float16 f16;
typedef __bf16 bf16;
typedef f16 h2 __attribute__((ext_vector_type(2)));
typedef f16 h8 __attribute__((ext_vector_type(8)));
typedef bf16 b2 __attribute__((ext_vector_type(2)));
typedef bf16 b8 __attribute__((ext_vector_type(8)));
typedef float f2 __attribute__((ext_vector_type(2)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef int i8v __attribute__((ext_vector_type(8)));
typedef float f16v __attribute__((ext_vector_type(16)));

constexpr int F16 = QG_MX_F16, BF16 = QG_MX_BF16, F32 = QG_MX_F32, FP4 = QG_MX_FP4;

template <int T> struct Elem;
template <> struct Elem<F16> { typedef f16 type; };
template <> struct Elem<BF16> { typedef bf16 type; };
template <> struct Elem<F32> { typedef float type; };

__device__ __forceinline__ float bits_f32(uint32_t v) { return __builtin_bit_cast(float, v); }
__device__ __forceinline__ uint32_t f32_bits(float v) { return __builtin_bit_cast(uint32_t, v); }

// The E8M0 byte s as the conversions take their scale: the exponent field of
// an fp32 number (field 0 is 2^-127 there, 255 NaN).
__device__ __forceinline__ float scale_f32(uint32_t s) { return bits_f32(s << 23); }

// ---------------------------------------------------------------------------
// quantise and read back
// ---------------------------------------------------------------------------
// Elementwise over blocks of 32: bound by HBM.  A lane takes 8 consecutive
// elements (one 16-byte load of 16-bit input), so four lanes share a block and
// find its largest magnitude with two quad permutes; a wave's codes are 256
// contiguous bytes.  The maximum is taken over the bit patterns without the
// sign, which order like the magnitudes and put infinities and NaN on top.
constexpr int EW_THREADS = 256;

template <int T> __device__ __forceinline__ void load8(const void* p, float v[8]) {
  if constexpr (T == F32) {
    const f4 a = reinterpret_cast<const f4*>(p)[0], b = reinterpret_cast<const f4*>(p)[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[i + 4] = b[i];
    }
  } else if constexpr (T == BF16) {
    const u4 a = *reinterpret_cast<const u4*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bits_f32(a[i] << 16);
      v[2 * i + 1] = bits_f32(a[i] & 0xffff0000u);
    }
  } else {
    const h8 a = *reinterpret_cast<const h8*>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)a[i];
  }
}

// largest of the four lanes of a quad (quad_perm 1,0,3,2 then 2,3,0,1)
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xf, 0xf, true));
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xf, 0xf, true));
}

// Rows of n8 groups of 8 elements (a contiguous matrix is one long row).
// The four lanes of a block are active together: n8 is a multiple of 4.
template <int T>
__global__ __launch_bounds__(EW_THREADS) void mx_quantize_kernel(const typename Elem<T>::type* __restrict__ x,
                                                                 int64_t ldx, int64_t rows, int64_t n8,
                                                                 uint32_t* __restrict__ codes,
                                                                 uint8_t* __restrict__ scales) {
  const int64_t step = (int64_t)gridDim.x * EW_THREADS;
  for (int64_t r = blockIdx.y; r < rows; r += gridDim.y)
    for (int64_t i = (int64_t)blockIdx.x * EW_THREADS + threadIdx.x; i < n8; i += step) {
      float v[8];
      load8<T>(x + r * ldx + i * 8, v);
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) top = max(top, f32_bits(v[j]) & 0x7fffffffu);
      const uint32_t e = quad_max(top) >> 23;   // biased exponent of the largest magnitude
      const uint32_t s = e == 255u ? 255u : e >= 2u ? e - 2u : 0u;
      uint32_t c = 0;
      const float sf = scale_f32(s);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], sf, 0);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], sf, 1);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], sf, 2);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], sf, 3);
      codes[r * n8 + i] = s == 255u ? 0u : c;
      if ((i & 3) == 0) scales[(r * n8 + i) >> 2] = (uint8_t)s;
    }
}

template <int T>
__global__ __launch_bounds__(EW_THREADS) void mx_dequantize_kernel(const uint32_t* __restrict__ codes,
                                                                   const uint8_t* __restrict__ scales,
                                                                   int64_t rows, int64_t n8,
                                                                   typename Elem<T>::type* __restrict__ y,
                                                                   int64_t ldy) {
  const int64_t step = (int64_t)gridDim.x * EW_THREADS;
  for (int64_t r = blockIdx.y; r < rows; r += gridDim.y)
    for (int64_t i = (int64_t)blockIdx.x * EW_THREADS + threadIdx.x; i < n8; i += step) {
      const uint32_t c = codes[r * n8 + i];
      const float sf = scale_f32(scales[(r * n8 + i) >> 2]);
      typename Elem<T>::type* d = y + r * ldy + i * 8;
      if constexpr (T == F32) {
        const f2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, sf, 0);
        const f2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, sf, 1);
        const f2 e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, sf, 2);
        const f2 f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, sf, 3);
        reinterpret_cast<f4*>(d)[0] = f4{a.x, a.y, b.x, b.y};
        reinterpret_cast<f4*>(d)[1] = f4{e.x, e.y, f.x, f.y};
      } else if constexpr (T == BF16) {
        const b2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sf, 0);
        const b2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sf, 1);
        const b2 e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sf, 2);
        const b2 f = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sf, 3);
        *reinterpret_cast<b8*>(d) = b8{a.x, a.y, b.x, b.y, e.x, e.y, f.x, f.y};
      } else {
        const h2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, sf, 0);
        const h2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, sf, 1);
        const h2 e = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, sf, 2);
        const h2 f = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, sf, 3);
        *reinterpret_cast<h8*>(d) = h8{a.x, a.y, b.x, b.y, e.x, e.y, f.x, f.y};
      }
    }
}

// ---------------------------------------------------------------------------
// products
// ---------------------------------------------------------------------------
struct MxArgs {
  const char* x; const uint8_t* xs; const uint8_t* w; const uint8_t* ws;
  const int32_t* rows; const int32_t* offsets; const float* row_scale;
  const char* resid; char* y;
  int64_t ldx_bytes, ldr, ldy;      // x row pitch in bytes, the others in elements
  int x_rows, E, M, N, K;           // M: rows of y (the slots of a grouped product)
  int y_type;
  int step;                         // mx_rows_kernel: rows at a time, at most 16
};

// 8 codes -> 8 exact 16-bit values (code times the block's scale)
__device__ __forceinline__ b8 codes_bf16(uint32_t c, float sf) {
  const b2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sf, 0);
  const b2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sf, 1);
  const b2 e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sf, 2);
  const b2 f = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, sf, 3);
  return b8{a.x, a.y, b.x, b.y, e.x, e.y, f.x, f.y};
}
__device__ __forceinline__ h8 codes_f16(uint32_t c, float sf) {
  const h2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, sf, 0);
  const h2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, sf, 1);
  const h2 e = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, sf, 2);
  const h2 f = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, sf, 3);
  return h8{a.x, a.y, b.x, b.y, e.x, e.y, f.x, f.y};
}

// Scale bytes for which every code times the scale is an exact fp16 number,
// 104..135: 0.5 * 2^(104 - 127) = 2^-24 is fp16's smallest (141 would be the
// first too large; 32 in a row are told apart by their upper bits).
__device__ __forceinline__ bool scale_fits_f16(uint32_t s) { return ((s - 104u) & ~31u) == 0; }
// not 0 where one of a word's four bytes does not fit (subtraction byte by byte)
__device__ __forceinline__ uint32_t scales_unfit_f16(uint32_t w) {
  return (((w | 0x80808080u) - 0x68686868u) ^ (~w & 0x80808080u)) & 0xe0e0e0e0u;
}

// fp16 x = hi + lo exactly in two bf16 numbers: fp16 has 11 significant bits,
// hi keeps the upper 8 (truncated), lo the at most 3 left over.  Infinities
// and NaN stay in hi (lo would be NaN for them: it is 0).
__device__ __forceinline__ void split_f16(h8 x, b8& hi, b8& lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t hb[2], lb[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float v = (float)x[2 * i + j];
      const uint32_t b = f32_bits(v);
      hb[j] = b & 0xffff0000u;
      const bool special = (b & 0x7f800000u) == 0x7f800000u;
      lb[j] = special ? 0u : f32_bits(v - bits_f32(hb[j]));
    }
    h[i] = (hb[0] >> 16) | hb[1];
    l[i] = (lb[0] >> 16) | (lb[1] & 0xffff0000u);
  }
  hi = __builtin_bit_cast(b8, u4{h[0], h[1], h[2], h[3]});
  lo = __builtin_bit_cast(b8, u4{l[0], l[1], l[2], l[3]});
}

__device__ __forceinline__ f4 mfma_fp4(u4 a, uint32_t sa, u4 b, uint32_t sb, f4 c) {
  const i8v av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const i8v bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

// S: which byte of the lanes' scale words counts
template <int S> __device__ __forceinline__ f16v mfma_fp4_32(u4 a, uint32_t sa, u4 b, uint32_t sb, f16v c) {
  const i8v av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const i8v bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, S, (int)sa, S, (int)sb);
}

// C 16- or 32-bit values at element alignment, in vectors of up to 16 bytes
template <int C, typename E> __device__ __forceinline__ void get(const E* p, E (&v)[C]) {
  constexpr int B = C * sizeof(E) >= 16 ? 16 : 8;
  typedef uint32_t vec __attribute__((ext_vector_type(B / 4), aligned(2)));
#pragma unroll
  for (int i = 0; i < (int)(C * sizeof(E)) / B; ++i) {
    const vec t = reinterpret_cast<const vec*>(p)[i];
    __builtin_memcpy(reinterpret_cast<char*>(v) + i * B, &t, B);
  }
}
template <int C, typename E> __device__ __forceinline__ void put(E* p, const E (&v)[C]) {
  constexpr int B = C * sizeof(E) >= 16 ? 16 : 8;
  typedef uint32_t vec __attribute__((ext_vector_type(B / 4), aligned(2)));
#pragma unroll
  for (int i = 0; i < (int)(C * sizeof(E)) / B; ++i) {
    vec t;
    __builtin_memcpy(&t, reinterpret_cast<const char*>(v) + i * B, B);
    reinterpret_cast<vec*>(p)[i] = t;
  }
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(f16 v) { return (float)v; }
__device__ __forceinline__ float to_f32(bf16 v) { return bits_f32((uint32_t)__builtin_bit_cast(uint16_t, v) << 16); }

// C (4 or 8) consecutive outputs of one row, columns n .. n+C-1 of row m: the
// factor and the residual in fp32, one rounding.  Rows of any pitch are stored
// in one piece (the device takes vector accesses at element alignment).
template <int YT, int C> __device__ __forceinline__ void store_cols_as(const MxArgs& a, int m, int n, float (&v)[C], float factor) {
  typedef typename Elem<YT>::type E;
  const bool whole = n + C <= a.N;
  const int have = min(a.N - n, C);
#pragma unroll
  for (int i = 0; i < C; ++i) v[i] *= factor;
  if (a.resid) {
    E r[C] = {};
    const E* rp = reinterpret_cast<const E*>(a.resid) + (int64_t)m * a.ldr + n;
    if (whole) get(rp, r);
    else for (int i = 0; i < C; ++i) if (i < have) r[i] = rp[i];
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] += to_f32(r[i]);
  }
  E q[C];
#pragma unroll
  for (int i = 0; i < C; ++i) q[i] = (E)v[i];
  E* y = reinterpret_cast<E*>(a.y) + (int64_t)m * a.ldy + n;
  if (whole) put(y, q);
  else for (int i = 0; i < C; ++i) if (i < have) y[i] = q[i];
}
template <int C> __device__ __forceinline__ void store_cols(const MxArgs& a, int m, int n, float (&v)[C], float factor) {
  if (a.y_type == F32) store_cols_as<F32, C>(a, m, n, v, factor);
  else if (a.y_type == F16) store_cols_as<F16, C>(a, m, n, v, factor);
  else store_cols_as<BF16, C>(a, m, n, v, factor);
}

// A grouped product's slots of expert e, kept within [0, T] whatever the
// offsets hold.
__device__ __forceinline__ void group_bounds(const MxArgs& a, int e, int& begin, int& end) {
  begin = min(max(a.offsets[e], 0), a.M);
  end = min(max(a.offsets[e + 1], begin), a.M);
}

// The row of x that slot m reads: its own where it has one, else some row of x
// (the outputs of such a slot are not stored, or stored as zeros).
template <bool GROUPED> __device__ __forceinline__ int x_row(const MxArgs& a, int m, int m_end) {
  m = min(m, m_end - 1);
  if (GROUPED && a.rows) m = a.rows[m];
  return m >= 0 && m < a.x_rows ? m : 0;
}

// Whether slot m has a row of x at all.
template <bool GROUPED> __device__ __forceinline__ bool has_row(const MxArgs& a, int m) {
  if (!GROUPED || !a.rows) return true;
  m = a.rows[m];
  return m >= 0 && m < a.x_rows;
}

typedef const void __attribute__((address_space(1)))* gptr;
typedef void __attribute__((address_space(3)))* lptr;

// At most N of this wave's global loads are on their way, and none of its LDS
// reads (s_waitcnt vmcnt(N) lgkmcnt(0), GFX9 encoding).
template <int N> __device__ __forceinline__ void wait_loads() {
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}

// Few rows: bound by the weights' bytes, and next to them by the number of
// vector loads (one takes a CU's address unit about 16 cycles however little it
// brings).  A workgroup owns 16*NT columns of y (rows of W) and up to 16 rows
// of it; its NW waves take K's chunks of 512 in turn and are summed through LDS
// in wave order.  Lane l = 16 g + r of a wave loads the four 16-byte blocks
// 4 u + g of a chunk of row r, which are the operand of
// v_mfma_scale_f32_16x16x128 as they are, and the row's 16 scale bytes at once;
// 16-bit x takes four 16x16x32 steps on a block's four words converted to 16
// bits.  x goes straight to the wave's own LDS, a kilobyte a load and no more
// rows than there are; row r keeps its 16-byte chunk c at place c ^ r, so 16
// rows' reads touch the 64 banks once.  A workgroup goes through its share of
// the column blocks (every gridDim.x-th), the next block's weights on their way
// while one is multiplied and summed; where every wave has one chunk, x stays.
// W is the first operand, so a lane ends with four consecutive outputs of one
// row.

// All of this wave's LDS reads have arrived (s_waitcnt lgkmcnt(0)).
__device__ __forceinline__ void wait_lds() { __builtin_amdgcn_s_waitcnt(0xc07f); }

// A barrier that waits for LDS accesses only: loads stay on their way.
__device__ __forceinline__ void lds_barrier() {
  wait_lds();
  asm volatile("" ::: "memory");        // no LDS access moves across the barrier
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// LDS of a wave for a chunk of x: whole direct loads of a kilobyte (four MXFP4 rows, one 16-bit row)
template <int XT> __host__ __device__ constexpr int rows_x_bytes(int M, int step) {
  const int rows = M < step ? M : step;
  return 1024 * (XT == FP4 ? (rows + 3) / 4 : rows);
}

template <int XT, int NT, int NW, bool SHORT, bool MULTI, bool GROUPED>
__global__ __launch_bounds__(NW * 64) void mx_rows_kernel(MxArgs a) {
  constexpr int XC = XT == FP4 ? 256 : 1024;     // bytes of an x row a chunk
  // Without groups a workgroup has one set of 16 rows, and the constant lets the compiler see that the loop over
  // rows runs once: with the step from the arguments 1 x 8192 x 8192 took 12.2 us instead of 10.0 (bf16 x).
  const int step = GROUPED ? a.step : 16;
  const int xbytes = rows_x_bytes<XT>(a.M, step);   // a wave's part of the LDS
  extern __shared__ __align__(1024) uint8_t rows_lds[];
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nkb = a.x_rows > 0 ? a.K >> 5 : 0;   // no x to read: all rows are zero
  const int chunks = (nkb + 15) >> 4, turns = (chunks + NW - 1) / NW;   // a wave's chunks: wave, wave + NW, ..
  const int blocks = (a.N + 16 * NT - 1) / (16 * NT);
  int m_begin, m_end;
  if constexpr (GROUPED) {
    group_bounds(a, blockIdx.y, m_begin, m_end);
  } else {
    m_begin = blockIdx.y * 16;
    m_end = min(a.M, m_begin + 16);
  }
  // 16 scale bytes of a row from block 16 c on (a row's last ones at most), or
  // where K < 512 the lane's own four, one a word.  scale_words() puts them in
  // place when they are used: doing so at once would wait for the load.
  auto load_scales = [&](const uint8_t* p, int c) {
    typedef uint32_t vec __attribute__((ext_vector_type(4), aligned(1)));
    u4 v;
    if constexpr (!SHORT) {
      v = *reinterpret_cast<const vec*>(p + min(c * 16, nkb - 16));
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = p[min(4 * u + g, nkb - 1)];
    }
    return v;
  };
  auto scale_words = [&](u4 v, int c) {   // word u: the four scale bytes of blocks 4 u .. 4 u + 3, this lane's first
    if constexpr (SHORT) return v;
    const int sh = 8 * max(c * 16 - (nkb - 16), 0);
    if (sh) {
      const uint64_t lo = v.x | ((uint64_t)v.y << 32), hi = v.z | ((uint64_t)v.w << 32);
      const uint64_t l = sh >= 64 ? hi >> (sh - 64) : (lo >> sh) | (hi << (64 - sh));
      const uint64_t u = sh >= 64 ? 0 : hi >> sh;
      v = u4{(uint32_t)l, (uint32_t)(l >> 32), (uint32_t)u, (uint32_t)(u >> 32)};
    }
    return u4{v.x >> (8 * g), v.y >> (8 * g), v.z >> (8 * g), v.w >> (8 * g)};
  };
  constexpr int WLOADS = NT * (SHORT ? 8 : 5);   // loads of load_w
  struct W { u4 c[NT][4], s[NT]; };
  auto load_w = [&](int nb, int c, W& w) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int64_t row = (GROUPED ? (int64_t)blockIdx.y * a.N : 0) + min((nb * NT + j) * 16 + r, a.N - 1);
      const uint8_t* wp = a.w + row * (a.K >> 1);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        w.c[j][u] = *reinterpret_cast<const u4*>(wp + (int64_t)min(c * 16 + 4 * u + g, nkb - 1) * 16);
      w.s[j] = load_scales(a.ws + row * (a.K >> 5), c);
    }
  };
  auto dma = [](const char* from, uint8_t* to) { __builtin_amdgcn_global_load_lds((gptr)from, (lptr)to, 16, 0, 0); };
  uint8_t* const xl = rows_lds + wave * xbytes;

  for (int m0 = m_begin; m0 < m_end; m0 += step) {
    // what belongs to row m0 + r is loaded first, so that no later wait is for it, and looked at
    // only when the first weights have been sent for
    const int rows = min(step, m_end - m0), rr = min(r, rows - 1);
    int xr = m0 + rr;
    float factor = 1.f;
    if constexpr (GROUPED) {
      if (a.rows) xr = a.rows[m0 + rr];
      if (a.row_scale) factor = a.row_scale[m0 + rr];
    }
    W w0, w1;
    int nb = blockIdx.x, turn = 0, buf = 0;
    if (chunks > 0) load_w(nb, min(wave, chunks - 1), w0);
    const bool has = !GROUPED || (xr >= 0 && xr < a.x_rows);
    xr = has ? xr : 0;
    // x: a whole chunk of the rows there are (past K: a row's last piece again)
    auto load_x = [&](int c) {
      if constexpr (XT == FP4) {
        for (int i = 0; i < rows; i += 4) {
          const int row = i + (lane >> 4);
          dma(a.x + __shfl(xr, row) * a.ldx_bytes + (int64_t)min(c * 16 + ((lane & 15) ^ row), nkb - 1) * 16, xl + i * XC);
        }
      } else {
        for (int i = 0; i < rows; ++i)
          dma(a.x + __builtin_amdgcn_readlane(xr, i) * a.ldx_bytes + (int64_t)min(c * 64 + (lane ^ i), nkb * 4 - 1) * 16,
              xl + i * XC);
      }
    };
    u4 xs = {0, 0, 0, 0};
    f4 acc[NT];
    const uint8_t* const xsp = XT == FP4 ? a.xs + (int64_t)xr * (a.K >> 5) : nullptr;
    if (turns == 1 && wave < chunks) {
      load_x(wave);
      if constexpr (XT == FP4) xs = load_scales(xsp, wave);
    }
    // one chunk of one block: its products, and after a block's last chunk the sums
    auto item = [&](auto MORE, W& w, W& next) {   // MORE: another item follows
      const int c = wave + turn * NW;
      const bool last = turn + 1 >= turns;
      if (turns > 1 && c < chunks) {
        load_x(c);
        if constexpr (XT == FP4) xs = load_scales(xsp, c);
      }
      // the next item's weights (a wave without a chunk loads some); all loads but those are waited for
      if constexpr (decltype(MORE)::value) {
        load_w(last ? nb + (int)gridDim.x : nb, min(last ? wave : c + NW, chunks - 1), next);
        wait_loads<WLOADS>();
      } else {
        wait_loads<0>();
      }
      if (turn == 0) {
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[j] = f4{0.f, 0.f, 0.f, 0.f};
      }
      if (c < chunks) {
        u4 ws[NT];
        bool fits = true;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          ws[j] = scale_words(w.s[j], c);
          if constexpr (XT == F16) {
#pragma unroll
            for (int u = 0; u < 4; ++u) fits = fits && (c * 16 + 4 * u + g >= nkb || scale_fits_f16(ws[j][u] & 255));
          }
        }
        if constexpr (XT == F16) fits = __all(fits);
        const u4 xw = scale_words(xs, c);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (c * 16 + 4 * u >= nkb) break;
          const bool past = c * 16 + 4 * u + g >= nkb;   // zero operands, factor 1
          uint32_t s[NT];
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            s[j] = past ? 127u : ws[j][u] & 255;
            if (past) w.c[j][u] = u4{0, 0, 0, 0};
          }
          if constexpr (XT == FP4) {
            u4 xv = *reinterpret_cast<const u4*>(xl + rr * XC + (((4 * u + g) ^ rr) * 16));
            if (past) xv = u4{0, 0, 0, 0};
            const uint32_t xsc = past ? 127u : xw[u];
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[j] = mfma_fp4(w.c[j][u], s[j], xv, xsc, acc[j]);
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              u4 xv = *reinterpret_cast<const u4*>(xl + rr * XC + (((16 * u + 4 * g + q) ^ rr) * 16));
              if (past) xv = u4{0, 0, 0, 0};
#pragma unroll
              for (int j = 0; j < NT; ++j) {
                if constexpr (XT == BF16) {
                  acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes_bf16(w.c[j][u][q], scale_f32(s[j])),
                                                                   __builtin_bit_cast(b8, xv), acc[j], 0, 0, 0);
                } else if (fits) {
                  acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(codes_f16(w.c[j][u][q], scale_f32(s[j])),
                                                                  __builtin_bit_cast(h8, xv), acc[j], 0, 0, 0);
                } else {   // beyond fp16's range: bf16 weights, x in two exact parts
                  const b8 wv = codes_bf16(w.c[j][u][q], scale_f32(s[j]));
                  b8 hi, lo;
                  split_f16(__builtin_bit_cast(h8, xv), hi, lo);
                  acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv, hi, acc[j], 0, 0, 0);
                  acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv, lo, acc[j], 0, 0, 0);
                }
              }
            }
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
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if (wave != (buf * NT + j) % NW) continue;   // the waves take the sums in turn
        f4 v = part[j * 64 + lane];
#pragma unroll
        for (int k = 1; k < NW; ++k) v += part[(k * NT + j) * 64 + lane];
        const int m = m0 + r, n = (nb * NT + j) * 16 + 4 * g;
        if (r < rows && n < a.N) {
          if (!has) {   // zero whatever the slot's factor holds: a padding slot's may be unset
            v = f4{0.f, 0.f, 0.f, 0.f};
            factor = 1.f;
          }
          float o[4] = {v.x, v.y, v.z, v.w};
          store_cols<4>(a, m, n, o, factor);
        }
      }
      buf ^= 1;
      turn = 0;
      nb += gridDim.x;
    };
    int left = nb < blocks ? ((blocks - 1 - nb) / (int)gridDim.x + 1) * max(turns, 1) : 0;
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
    lds_barrier();   // the sums have been read before the next 16 rows' are written
  }
}

// ---------------------------------------------------------------------------
// more rows
// ---------------------------------------------------------------------------
// Where a workgroup's tile lies: group e, rows m0 .. m_end of y (at most TM of
// them), column tile tn.  Returns false when there is no tile for it.
// Tiles are numbered row tile fastest within blocks of 8 row tiles, and a number range
// goes to one XCD (workgroup b runs on XCD b % 8), so the tiles whose operands
// an XCD's L2 holds run together.  A grouped product finds its row tiles from
// the offsets: lane by lane the tiles of 64 groups, a running sum, a vote.
struct Tile { int e, m0, m_end, tn; };

// the sum of v over the lanes up to and with this one
__device__ __forceinline__ int wave_running_sum(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);    // row_shr:1, then 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);   // row 0's sum to row 1, row 2's to row 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);   // the first two rows' to the others
  return v;
}

template <int TM, bool GROUPED>
__device__ __forceinline__ bool find_tile(const MxArgs& a, int tiles_n, Tile& t) {
  int tiles_m = 0, b = 0, e = 0, n = 0, sum = 0;
  const int lane = threadIdx.x & 63;
  auto scan = [&](int e0) {   // this lane's group: its rows b .. e, its tiles n, the tiles up to and with it
    n = b = e = 0;
    if (e0 + lane < a.E) {
      group_bounds(a, e0 + lane, b, e);
      n = (e - b + TM - 1) / TM;
    }
    sum = wave_running_sum(n);
  };
  if constexpr (GROUPED) {
    for (int e0 = 0; e0 < a.E; e0 += 64) {
      scan(e0);
      tiles_m += __builtin_amdgcn_readlane(sum, 63);
    }
  } else {
    tiles_m = (a.M + TM - 1) / TM;
  }
  const int64_t total = (int64_t)tiles_m * tiles_n;
  const int xcd = blockIdx.x & 7;
  const int64_t lo = total * xcd / 8, hi = total * (xcd + 1) / 8;
  const int64_t id = lo + (blockIdx.x >> 3);
  if (id >= hi) return false;
  const int64_t per = (int64_t)8 * tiles_n;
  const int blk = (int)(id / per), in = (int)(id - blk * per);
  const int bm = min(8, tiles_m - blk * 8);
  int tm = blk * 8 + in % bm;
  t.tn = in / bm;
  t.e = 0;
  if constexpr (GROUPED) {
    for (int e0 = 0; e0 < a.E; e0 += 64) {
      if (a.E > 64) scan(e0);
      const uint64_t vote = __ballot(sum > tm);
      if (vote) {
        const int who = __builtin_ctzll(vote);
        const int end = __builtin_amdgcn_readlane(e, who);
        t.e = e0 + who;
        t.m0 = __builtin_amdgcn_readlane(b, who) + (tm - __builtin_amdgcn_readlane(sum - n, who)) * TM;
        t.m_end = min(end, t.m0 + TM);
        return t.m0 >= 0 && t.m0 < t.m_end;
      }
      tm -= __builtin_amdgcn_readlane(sum, 63);
    }
    return false;
  }
  t.m0 = tm * TM;
  t.m_end = min(a.M, t.m0 + TM);
  return true;
}

// Stores a wave's MI x NI blocks of 32 x 32 (element 4 q + k of lane 32 h + r:
// column 8 q + 4 h + k, row r) at rows row0 of the tile and column n0.  Each
// strip of 32 rows passes through LDS (the wave's own `strip`, rows padded by
// 16 bytes), so that a lane stores 8 consecutive outputs and 4 NI lanes a
// contiguous row piece.  `info`: a row's factor and whether it has a row of x.
template <int YT, int MI, int NI, bool GROUPED>
__device__ __forceinline__ void store_blocks_as(const MxArgs& a, const Tile& t, uint8_t* strip, int row0, int n0,
                                                const f2* info, const f16v (&acc)[MI][NI]) {
  constexpr int PITCH = 32 * NI + 4, LANES = 4 * NI, ROWS = 64 / LANES;
  const int lane = threadIdx.x & 63;
  float* s = reinterpret_cast<float*>(strip);
#pragma unroll
  for (int i = 0; i < MI; ++i) {
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<f4*>(s + (lane & 31) * PITCH + 32 * j + 8 * q + 4 * (lane >> 5)) =
            f4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    const int n = n0 + (lane % LANES) * 8;
#pragma unroll
    for (int p = 0; p < 32 / ROWS; ++p) {
      const int r = p * ROWS + lane / LANES, row = row0 + i * 32 + r, m = t.m0 + row;
      if (m >= t.m_end || n >= a.N) continue;
      float v[8], factor = 1.f;
      __builtin_memcpy(v, s + r * PITCH + (lane % LANES) * 8, sizeof(v));
      if constexpr (GROUPED) {
        const f2 f = info[row];
        factor = f.x;
        if (f.y == 0.f) {
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = 0.f;
        }
      }
      store_cols_as<YT, 8>(a, m, n, v, factor);
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
}
template <int MI, int NI, bool GROUPED>
__device__ __forceinline__ void store_blocks(const MxArgs& a, const Tile& t, uint8_t* strip, int row0, int n0,
                                             const f2* info, const f16v (&acc)[MI][NI]) {
  __syncthreads();                                   // every wave has read its last stage
  if (a.y_type == F32) store_blocks_as<F32, MI, NI, GROUPED>(a, t, strip, row0, n0, info, acc);
  else if (a.y_type == F16) store_blocks_as<F16, MI, NI, GROUPED>(a, t, strip, row0, n0, info, acc);
  else store_blocks_as<BF16, MI, NI, GROUPED>(a, t, strip, row0, n0, info, acc);
}

// A 32 x 32 x 16 product of 16-bit operands.
__device__ __forceinline__ f16v mfma_16(b8 a, b8 b, f16v c) { return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0); }
__device__ __forceinline__ f16v mfma_16(h8 a, h8 b, f16v c) { return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0); }

// x and W stream through a ring of RING LDS stages of 128 k: a workgroup of WM
// x WN waves, each MI x NI blocks of 32 x 32 outputs.  The loads go straight to
// LDS, RING - 1 stages ahead.  A row's 16-byte chunks change places by the
// row's number, so that the fragment reads of 16 consecutive rows touch the 64
// banks once: MXFP4 rows are 64 bytes (chunk c at c ^ (row / 4 % 4)), 16-bit
// rows 256 (c ^ (row % 16)).  A stage is two steps of 64 k, lane half h taking
// the 32-block h of a step: with MXFP4 x one scaled matrix instruction a
// block, with 16-bit x four of 16 k on the weights' words converted to 16 bits.
// The fragments of one step are read while the other's are multiplied.  The
// one barrier a stage, in between, says both that everyone's loads of the next
// stage have arrived and that this stage has been read.  Every stage issues the
// same loads, so a count of the outstanding ones tells which have arrived.  W
// is the first operand of the matrix instruction: a lane's outputs run along a
// row of y.
template <int XT, int MI, int NI, int WM, int WN, int RING, bool GROUPED>
__global__ __launch_bounds__(WM * WN * 64) void mx_tile_kernel(MxArgs a, int tiles_n) {
  constexpr int NW = WM * WN, TM = 32 * MI * WM, TN = 32 * NI * WN;
  constexpr bool FP = XT == FP4;
  constexpr int XB = FP ? 64 : 256, XR = 1024 / XB;        // bytes of an x row a stage, rows a direct load brings
  constexpr int QA = TM / XR / NW, QB = TN / 16 / NW, QD = QA + QB;   // direct loads of 1 KiB a wave and stage
  static_assert(QA * XR * NW == TM && QB * 16 * NW == TN, "rows split evenly over the waves");
  constexpr int SROWS = FP ? TM + TN : TN, SOFF = FP ? TM : 0;   // rows with scales; W's first
  constexpr int STAGE = TM * XB + TN * 64;
  static_assert(RING >= 3 && RING <= 5, "a group's scales are older than what the last stage before it leaves on its way");
  static_assert(SROWS % 64 == 0, "a load brings the scales of 64 rows");
  constexpr int QS = (SROWS / 64 + NW - 1) / NW;               // such loads a wave and group
  static_assert(NW * 32 * (32 * NI + 4) * 4 <= RING * STAGE, "store_blocks' strips");
  // one array: with two, the compiler waits for every direct load before each read
  __shared__ __align__(1024) uint8_t smem[RING * STAGE + 2 * SROWS * 16 + (GROUPED ? TM * 8 : 0)];
  uint8_t* const sc = smem + RING * STAGE;   // scales: two groups of four stages, 16 bytes a row
  f2* const info = reinterpret_cast<f2*>(sc + 2 * SROWS * 16);   // grouped: a row's factor, and 1 where it has a row of x
  Tile t;
  if (!find_tile<TM, GROUPED>(a, tiles_n, t)) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int n0 = t.tn * TN;
  const int nkb = a.K >> 5;

  if constexpr (GROUPED) {
    for (int i = tid; i < t.m_end - t.m0; i += NW * 64) {
      const float factor = a.row_scale ? a.row_scale[t.m0 + i] : 1.f;   // loaded beside the row's number
      const bool has = has_row<true>(a, t.m0 + i);   // without a row: zero whatever the slot's factor holds
      info[i] = f2{has ? factor : 1.f, has ? 1.f : 0.f};
    }
  }
  // direct loads: lane l brings a 16-byte chunk of row l / 4 of 16 (16-bit x: row l / 16 of 4)
  const char* src[QD];
#pragma unroll
  for (int q = 0; q < QA; ++q)
    src[q] = a.x + x_row<GROUPED>(a, t.m0 + (wave * QA + q) * XR + lane / (64 / XR), t.m_end) * a.ldx_bytes;
#pragma unroll
  for (int q = 0; q < QB; ++q)
    src[QA + q] = reinterpret_cast<const char*>(a.w) +
                  ((int64_t)t.e * a.N + min(n0 + (wave * QB + q) * 16 + (lane >> 2), a.N - 1)) * (a.K >> 1);
  // scales: the 16 bytes of a group of stages of row l of 64 (waves to spare bring the same rows again)
  const uint8_t* ssrc[QS];
#pragma unroll
  for (int q = 0; q < QS; ++q) {
    const int r = (wave * QS + q) % (SROWS / 64) * 64 + lane;
    ssrc[q] = FP && r < TM ? a.xs + (int64_t)x_row<GROUPED>(a, t.m0 + r, t.m_end) * nkb
                           : a.ws + ((int64_t)t.e * a.N + min(n0 + r - SOFF, a.N - 1)) * nkb;
  }
  // fragments: lane l reads row l % 32, MXFP4 chunk 2 s + l / 32 of step s, 16-bit chunks 8 s + 4 (l / 32) + 0..3
  const int fr = lane & 31, h = lane >> 5;
  uint32_t foff[2], xoff[2][4];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    foff[s] = fr * 64 + (((2 * s + h) ^ ((fr >> 2) & 3)) * 16);
#pragma unroll
    for (int c = 0; c < 4; ++c) xoff[s][c] = fr * 256 + (((8 * s + 4 * h + c) ^ (fr & 15)) * 16);
  }
  // a wave of one block keeps two sums of it, so that a product need not wait for the one before
  constexpr int ACCS = MI * NI == 1 ? 2 : 1;
  f16v acc[MI][NI], other[1];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int k = 0; k < 16; ++k) acc[i][j][k] = 0.f;
#pragma unroll
  for (int k = 0; k < 16; ++k) other[0][k] = 0.f;
  auto sum = [&](int i, int j, int c) -> f16v& { return ACCS == 2 && (c & 1) ? other[0] : acc[i][j]; };

  auto dma = [](const char* from, uint8_t* to) { __builtin_amdgcn_global_load_lds((gptr)from, (lptr)to, 16, 0, 0); };
  // this lane's chunk of a stage, in 16 bytes
  auto chunk = [&](int q) { return FP || q >= QA ? (lane & 3) ^ (lane >> 4) : (lane & 15) ^ (lane >> 4) ^ (4 * ((wave * QA + q) & 3)); };
#pragma unroll
  for (int q = 0; q < QD; ++q) src[q] += chunk(q) * 16;
  auto place = [&](uint8_t* to, int q) { return to + (q < QA ? (wave * QA + q) * 1024 : TM * XB + (wave * QB + q - QA) * 1024); };
  const int whole = nkb >> 2;   // stages that lie within K
  // past those: the last of them again, into a place that is not read any more
  auto issue = [&](int it, uint8_t* to, int q) { dma(src[q] + (int64_t)min(it, whole - 1) * (q < QA ? XB : 64), place(to, q)); };
  // the stage that K ends in: pieces past K are a row's last one
  auto issue_part = [&](uint8_t* to) {
#pragma unroll
    for (int q = 0; q < QD; ++q) {
      const int per = q < QA ? XB / 16 : 4, last = (nkb & 3) * (per / 4) - 1;
      dma(src[q] + (int64_t)whole * (16 * per) + (min(chunk(q), last) - chunk(q)) * 16, place(to, q));
    }
  };
  auto issue_scales = [&](int group) {   // the row's last 16 bytes at most
#pragma unroll
    for (int q = 0; q < QS; ++q)
      dma(reinterpret_cast<const char*>(ssrc[q]) + min(group * 16, nkb - 16),
          sc + (group & 1) * (SROWS * 16) + (wave * QS + q) % (SROWS / 64) * 1024);
  };
  auto barrier = [] {
    asm volatile("" ::: "memory");   // no LDS access moves across it
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  struct Frag { u4 a[MI][FP ? 1 : 4], b[NI]; };
  auto read = [&](const uint8_t* from, int s) {
    Frag f;
#pragma unroll
    for (int j = 0; j < NI; ++j) f.b[j] = *reinterpret_cast<const u4*>(from + TM * XB + (wn * NI + j) * 2048 + foff[s]);
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int c = 0; c < (FP ? 1 : 4); ++c)
        f.a[i][c] = *reinterpret_cast<const u4*>(from + (wm * MI + i) * 32 * XB + (FP ? foff[s] : xoff[s][c]));
    return f;
  };
  // the scale words of a stage: byte 0 and byte 2 are this lane half's blocks of the two steps
  struct Scales { uint32_t a[FP ? MI : 1], b[NI]; };
  // the products of one step; `between` runs after each of MI * NI parts
  auto multiply = [&](auto S, const Frag& f, const Scales& w, auto between) {
    constexpr int s = decltype(S)::value;
    if constexpr (FP) {
#pragma unroll
      for (int k = 0; k < MI * NI; ++k) {
        const int i = k / NI, j = k % NI;
        sum(i, j, s) = mfma_fp4_32<2 * s>(f.b[j], w.b[j], f.a[i][0], w.a[i], sum(i, j, s));
        between(k);
      }
    } else {
      float sf[NI];
#pragma unroll
      for (int j = 0; j < NI; ++j) sf[j] = scale_f32((w.b[j] >> (16 * s)) & 255);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if constexpr (XT == F16) {
          h8 wv[NI];
#pragma unroll
          for (int j = 0; j < NI; ++j) wv[j] = codes_f16(f.b[j][c], sf[j]);
#pragma unroll
          for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j) sum(i, j, c) = mfma_16(wv[j], __builtin_bit_cast(h8, f.a[i][c]), sum(i, j, c));
        } else {
          b8 wv[NI];
#pragma unroll
          for (int j = 0; j < NI; ++j) wv[j] = codes_bf16(f.b[j][c], sf[j]);
#pragma unroll
          for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j) sum(i, j, c) = mfma_16(wv[j], __builtin_bit_cast(b8, f.a[i][c]), sum(i, j, c));
        }
        // between() MI * NI times in all, spread over the four words
#pragma unroll
        for (int k = 0; k < MI * NI; ++k)
          if (k * 4 / (MI * NI) == c) between(k);
      }
    }
  };
  auto nothing = [](int) {};
  // fp16 x and weights beyond fp16's range: a stage on bf16 weights and x in two
  // exact parts, operands taken from LDS as they are needed.  The row's scale
  // bytes at `scales` begin with block `first`.
  auto wide_stage = [&](int it, const uint8_t* place, const uint8_t* scales, int first) {
#pragma unroll 1
    for (int n = 0; n < 8; ++n) {
      const int s = n >> 2, c = n & 3, kb = it * 4 + 2 * s + h;
      b8 wv[NI];
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const int row = (wn * NI + j) * 32 + fr;
        const uint8_t* p = place + TM * XB + row * 64 + (((2 * s + h) ^ ((fr >> 2) & 3)) * 16) + 4 * c;
        const uint32_t word = kb < nkb ? *reinterpret_cast<const uint32_t*>(p) : 0u;
        wv[j] = codes_bf16(word, kb < nkb ? scale_f32(scales[row * 16 + kb - first]) : 1.f);
      }
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const uint8_t* p = place + ((wm * MI + i) * 32 + fr) * XB + (((8 * s + 4 * h + c) ^ (fr & 15)) * 16);
        h8 xv = *reinterpret_cast<const h8*>(p);
        if (kb >= nkb) xv = h8{};
        b8 hi, lo;
        split_f16(xv, hi, lo);
#pragma unroll
        for (int j = 0; j < NI; ++j) acc[i][j] = mfma_16(wv[j], lo, mfma_16(wv[j], hi, acc[i][j]));
      }
    }
  };
  constexpr std::integral_constant<int, 0> s0{};
  constexpr std::integral_constant<int, 1> s1{};

  if (nkb >= 16) {
    issue_scales(0);
  } else {   // K < 512: fewer than 16 bytes a row, brought one by one
    for (int row = tid; row < SROWS; row += NW * 64) {
      const uint8_t* p = FP && row < TM ? a.xs + (int64_t)x_row<GROUPED>(a, t.m0 + row, t.m_end) * nkb
                                        : a.ws + ((int64_t)t.e * a.N + min(n0 + row - SOFF, a.N - 1)) * nkb;
#pragma unroll
      for (int b = 0; b < 15; ++b) sc[row * 16 + b] = p[min(b, nkb - 1)];
    }
  }
#pragma unroll
  for (int it = 0; it < RING; ++it)
    if (nkb >= 16 || it < whole) {   // the waits below count all RING of them
#pragma unroll
      for (int q = 0; q < QD; ++q) issue(it, smem + it * STAGE, q);
    }
  wait_loads<(RING - 1) * QD>();
  barrier();
  Frag f0 = read(smem, 0), f1;
  const int groups = nkb >> 4;
  uint8_t* cur = smem;   // the place of the stage at hand
  auto next_place = [&](uint8_t* p) { return p == smem + (RING - 1) * STAGE ? smem : p + STAGE; };
  u4 sa[FP ? MI : 1], sb[NI];   // a group's scale bytes of this lane's rows
  auto read_scales = [&](int g) {
    const uint8_t* sp = sc + (g & 1) * (SROWS * 16) + fr * 16;
    if constexpr (FP) {
#pragma unroll
      for (int i = 0; i < MI; ++i) sa[i] = *reinterpret_cast<const u4*>(sp + (wm * MI + i) * 512);
    }
#pragma unroll
    for (int j = 0; j < NI; ++j) sb[j] = *reinterpret_cast<const u4*>(sp + (SOFF + (wn * NI + j) * 32) * 16);
  };
  read_scales(0);
#pragma unroll 1
  for (int g = 0; g < groups; ++g) {
    if constexpr (XT == F16) {
      uint32_t unfit = 0;
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) unfit |= scales_unfit_f16(sb[j][k]);
      if (__any(unfit != 0)) {
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {   // the same waits, barriers and loads as below
          const int it = g * 4 + k;
          wide_stage(it, cur, sc + (g & 1) * (SROWS * 16), g * 16);
          wait_loads<(RING - 2) * QD>();
          barrier();
          if (k == 0) issue_scales(g + 1);
#pragma unroll
          for (int q = 0; q < QD; ++q) issue(it + RING, cur, q);
          cur = next_place(cur);
        }
        f0 = read(cur, 0);
        read_scales(g + 1);
        continue;
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int it = g * 4 + k;
      Scales w;
      if constexpr (FP) {
#pragma unroll
        for (int i = 0; i < MI; ++i) w.a[i] = sa[i][k] >> (8 * h);
      }
#pragma unroll
      for (int j = 0; j < NI; ++j) w.b[j] = sb[j][k] >> (8 * h);
      wait_lds();   // the first step's operands are here; later this would wait for the second's too
      f1 = read(cur, 1);
      __builtin_amdgcn_sched_barrier(0);
      multiply(s0, f0, w, nothing);
      __builtin_amdgcn_sched_barrier(0);
      // stage it + 1 has arrived (those after it are on their way), stage it
      // has been read: its place takes stage it + RING
      // (and in stages 1 and 2 the next group's scales, which are read after stage 3)
      if (k >= 1 && k <= 2 && k <= RING - 2) wait_loads<(RING - 2) * QD + QS>();
      else wait_loads<(RING - 2) * QD>();
      barrier();
      if (k == 0) issue_scales(g + 1);
      uint8_t* const nxt = next_place(cur);
      f0 = read(nxt, 0);
      if (k == 3) read_scales(g + 1);
      __builtin_amdgcn_sched_barrier(0);
      multiply(s1, f1, w, [&](int n) {   // the loads spread over the products: issued at once they hold the wave up
#pragma unroll
        for (int q = 0; q < QD; ++q)
          if (q * (MI * NI) / QD == n) {
            issue(it + RING, cur, q);
            __builtin_amdgcn_sched_barrier(FP ? 0 : 2);   // 16 bits: the conversions may pass
          }
      });
      cur = nxt;
    }
  }
  wait_loads<0>();   // nothing is on its way to LDS any more
  barrier();
  // The stages of a last group that is not whole (at most four; RING of them
  // are there, but for the one that K ends in: the others are sent for here).
  for (int it = groups * 4; it * 4 < nkb; ++it) {
    if (it == groups * 4 + RING || it == whole) {
      barrier();     // the places have been read
      if (it == whole) {
        issue_part(cur);
      } else {
#pragma unroll
        for (int q = 0; q < QD; ++q) issue(it, cur, q);
      }
      wait_loads<0>();
      barrier();
    }
    // its 16 scale bytes are the row's last ones (K < 512: all); past K: factor 1, zero operands
    const int k0 = it * 4 + h;
    auto scale = [&](int row) {
      const uint8_t* p = sc + (groups & 1) * (SROWS * 16) + (row + fr) * 16 - max(nkb - 16, 0);
      return (k0 < nkb ? (uint32_t)p[k0] : 127u) | (k0 + 2 < nkb ? (uint32_t)p[k0 + 2] : 127u) << 16;
    };
    Scales w;
    if constexpr (FP) {
#pragma unroll
      for (int i = 0; i < MI; ++i) w.a[i] = scale((wm * MI + i) * 32);
    }
#pragma unroll
    for (int j = 0; j < NI; ++j) w.b[j] = scale(SOFF + (wn * NI + j) * 32);
    if constexpr (XT == F16) {
      bool fits = true;
#pragma unroll
      for (int j = 0; j < NI; ++j) fits = fits && scale_fits_f16(w.b[j] & 255) && scale_fits_f16(w.b[j] >> 16);
      if (!__all(fits)) {
        wide_stage(it, cur, sc + (groups & 1) * (SROWS * 16), max(nkb - 16, 0));
        cur = next_place(cur);
        continue;
      }
    }
    f0 = read(cur, 0);
    f1 = read(cur, 1);
    auto clear = [](Frag& f) {
#pragma unroll
      for (int j = 0; j < NI; ++j) f.b[j] = u4{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int c = 0; c < (FP ? 1 : 4); ++c) f.a[i][c] = u4{0, 0, 0, 0};
    };
    if (k0 >= nkb) clear(f0);
    if (k0 + 2 >= nkb) clear(f1);
    multiply(s0, f0, w, nothing);
    multiply(s1, f1, w, nothing);
    cur = next_place(cur);
  }
  if constexpr (ACCS == 2) acc[0][0] += other[0];
  store_blocks<MI, NI, GROUPED>(a, t, smem + wave * (32 * (32 * NI + 4) * 4), wm * MI * 32, n0 + wn * NI * 32, info, acc);
}

// A product without a k, one element a lane: the residual, or zero.
template <int YT> __global__ __launch_bounds__(EW_THREADS) void mx_no_k_kernel(MxArgs a) {
  typedef typename Elem<YT>::type E;
  const int64_t step = (int64_t)gridDim.x * EW_THREADS, n = (int64_t)a.M * a.N;
  for (int64_t i = (int64_t)blockIdx.x * EW_THREADS + threadIdx.x; i < n; i += step) {
    const int64_t row = i / a.N, col = i - row * a.N;
    const float r = a.resid ? to_f32(reinterpret_cast<const E*>(a.resid)[row * a.ldr + col]) : 0.f;
    reinterpret_cast<E*>(a.y)[row * a.ldy + col] = (E)(0.f + r);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
bool float_type(int t) { return t == F16 || t == BF16 || t == F32; }
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_matrix(const void* v, int ld, int type, int M, int K, const void* codes, const void* scales) {
  if (!float_type(type) || M < 0 || K < 0 || K % 32) return QG_E_ARG;
  if (M == 0 || K == 0) return QG_OK;
  if (!v || !codes || !scales || ld < K) return QG_E_ARG;
  if (!aligned(v, 16) || !aligned(codes, 16) || ld % 8) return QG_E_ALIGN;
  return QG_OK;
}

// Grid of an elementwise kernel over rows x n8 groups: as many workgroups along
// a row as fill the chip's wave slots twice (16 a CU, of 4 waves), the rest by
// the kernel's own loops.  A matrix whose rows follow each other is one row
// here; strided rows narrower than a workgroup's 256 groups leave lanes idle
// (K = 32: 4 of 256 work).
dim3 ew_grid(int64_t rows, int64_t n8) {
  const int64_t bx = std::min<int64_t>((n8 + EW_THREADS - 1) / EW_THREADS, 256 * 16);
  return dim3((unsigned)std::max<int64_t>(bx, 1), (unsigned)std::min<int64_t>(rows, 65535));
}

// Which kernel takes a product.  tile 0: mx_rows_kernel with nt column blocks
// and nw waves a workgroup; 1..4: mx_tile_kernel on 64 x 64, 64 x 128, 128 x 128
// and 256 x 256 tiles (16-bit x: 128 x 256).  QMX_TILE=0..4 in the environment
// forces one (tests, tuning).
// fits: whether a grid holds it (65535 blocks along y, and along x 2^32 - 1
// lanes).
struct MxPlan { int tile, nt, nw, step; int64_t workgroups; bool fits; };

// The rule is a model of the time in nanoseconds, from what the kernels
// measured on graph-replayed products of 1..2048 rows with 2048 and 8192
// columns and K, and on products of 32..16384 rows grouped over 8..64 matrices.
// A tile's stage of 128 k takes `alone` when its CU runs one tile (latency)
// and `shared` for each of the CU's tiles when the chip is full; `start` is
// a tile's first loads and stores, of which the share `more` shows again for every
// further tile of the CU.  The rows kernel takes `item` for a block of 16 x 16
// outputs and chunk of 512 k, over the whole chip, and a pause between 16 rows
// of a group and the next.  For instance 8192 x 8192
// weights and bf16 x: 16 rows 13.4 us (64 x 64 tiles 21.4), 64 rows on 64 x 64
// tiles 21.6 (rows kernel 42), 512 rows on 128 x 128 66 (64 x 64 96, 128 x 256
// 87), 2048 rows on 128 x 256 224 (128 x 128 258).  How many row tiles a
// grouped product has is estimated: each group's last one half empty.
struct MxTileCost { int rows, cols, threads; double alone, shared, start, more; };
constexpr MxTileCost MX_TILES[2][4] = {
    {{64, 64, 256, 385, 345, 3000, 0.3}, {64, 128, 256, 490, 510, 3200, 0.5},
     {128, 128, 512, 770, 1030, 3500, 0.5}, {128, 256, 512, 1290, 1730, 4000, 0.8}},
    {{64, 64, 256, 165, 180, 2900, 0.3}, {64, 128, 256, 215, 255, 3000, 0.8},
     {128, 128, 256, 265, 390, 3300, 0.4}, {256, 256, 512, 720, 1130, 5500, 1.0}}};

// Workgroups of a tiled product (E = 0: not grouped): a grouped one has at
// most this many row tiles, whatever its offsets hold.
int64_t tile_grid(int M, int N, int E, int rows, int cols) {
  const int64_t tm = E > 0 ? M / rows + std::min(E, M) : ((int64_t)M + rows - 1) / rows;
  return (((int64_t)N + cols - 1) / cols * tm + 7) / 8 * 8;
}

MxPlan plan_product(int M, int N, int K, int E, int x_type) {
  const bool fp = x_type == FP4;
  MxPlan p = {0, 1, 1, 16, 0, true};
  if (M == 0 || N == 0) return p;   // nothing to launch; below, a grouped call has at least one active group
  const int64_t chunks = ((int64_t)K + 511) / 512, stages = ((int64_t)K + 127) / 128;
  const int active = E > 0 ? std::min(E, M) : 1;
  auto row_tiles = [&](int rows) -> int64_t {
    if (E == 0) return ((int64_t)M + rows - 1) / rows;
    return std::max<int64_t>(active, M / rows + active / 2);
  };
  if (K > 0) {
    const double item = E > 0 ? (fp ? 0.5 : M <= 2 * E ? 0.8 : 1.2) : (fp ? 0.9 : 1.7);
    double best = 2300 + item * (double)(row_tiles(16) * (((int64_t)N + 15) / 16) * chunks);
    // a grouped call's workgroups go through their group's rows 16 at a time; some groups are large
    if (E > 0) best += 2500 * (double)(M / (8 * (int64_t)active));
    if (row_tiles(16) > 65535) best = 1e300;   // the rows kernel's grid
    int64_t tiles[4];
    for (int i = 0; i < 4; ++i) {
      const MxTileCost& c = MX_TILES[fp][i];
      tiles[i] = row_tiles(c.rows) * (((int64_t)N + c.cols - 1) / c.cols);
      const double turns = (double)((tiles[i] + 255) / 256);
      const double cost = (double)stages * std::max(c.alone, c.shared * turns) + c.start * (1 + c.more * (turns - 1));
      if (cost < best) best = cost, p.tile = i + 1;
    }
    const int forced = env_int("QMX_TILE", -1);
    if (forced >= 0 && forced <= 4) p.tile = forced;
    if (p.tile) p.workgroups = tiles[p.tile - 1];
  }
  if (p.tile) {
    const MxTileCost& c = MX_TILES[fp][p.tile - 1];
    p.fits = tile_grid(M, N, E, c.rows, c.cols) * c.threads <= (int64_t)UINT32_MAX;
  } else {
    // without a k: a workgroup of one wave for every block of a group's columns; without groups another kernel
    p.fits = E > 0 ? K > 0 || ((int64_t)N + 15) / 16 * 64 <= (int64_t)UINT32_MAX : K == 0 || row_tiles(16) <= 65535;
    // a wave for every chunk, so that x stays in LDS; where that is more than
    // fits, and x is read again for every block, two blocks share the reading
    p.nw = K < 512 ? 1 : chunks <= 2 ? 2 : chunks <= 4 ? 4 : chunks <= 8 ? 8 : 16;
    // a grouped call of few rows a group: with 8 at a time instead of 16 a 16-bit x takes half the LDS, and
    // twice the workgroups are resident (32 rows over 32 matrices of 2048 x 2048, bf16: 12.8
    // us instead of 15.0)
    if (E > 0 && !fp && M <= 2 * E) p.step = 8;
    const int rows = std::min(M, p.step);
    const int64_t lds = (int64_t)p.nw * 1024 * ((fp ? (rows + 3) / 4 : rows) + 2);
    if (lds > 160 * 1024) {
      p.nw = 8;
      if ((int64_t)N * active >= 16 * 512) p.nt = 2;
    }
    p.workgroups = row_tiles(16) * (((int64_t)N + 16 * p.nt - 1) / (16 * p.nt));
  }
  return p;
}

int launch_status() { return hip_status(hipGetLastError()); }

// QG_OK when there is a device to launch on.  Asking takes the runtime about a
// microsecond; once one was there it is not asked again.
int device_present() {
  static std::atomic<bool> seen{false};
  if (seen.load(std::memory_order_relaxed)) return QG_OK;
  int dev = 0;
  const int st = current_device(&dev);
  if (st == QG_OK) seen.store(true, std::memory_order_relaxed);
  return st;
}

template <int XT, int NT, int NW, bool SHORT, bool GROUPED> void launch_rows(const MxArgs& a, hipStream_t s) {
  const int64_t gy = GROUPED ? a.E : ((int64_t)a.M + 15) / 16;
  const size_t lds = (size_t)NW * rows_x_bytes<XT>(a.M, a.step) + 2 * NW * NT * 1024;
  // column blocks a workgroup takes: no more workgroups than keep 32 waves on every CU.  A grouped product
  // without a k to go through takes one (the kernel for several sends for the next block's weights).
  const int64_t blocks = (a.N + 16 * NT - 1) / (16 * NT), active = GROUPED ? std::min(a.E, a.M) : gy;
  const bool none = GROUPED && SHORT && (a.K == 0 || a.x_rows == 0);
  const int64_t slots = 256 * 32 / NW, share = none ? 1 : (blocks * active + slots - 1) / slots;
  const dim3 grid((unsigned)((blocks + share - 1) / share), (unsigned)gy);
  if constexpr (NT == 1) {   // two blocks are for a K of several chunks a wave
    if (none || (share == 1 && a.K <= 512 * NW)) {
      hipLaunchKernelGGL((mx_rows_kernel<XT, NT, NW, SHORT, false, GROUPED>), grid, dim3(NW * 64), lds, s, a);
      return;
    }
  }
  hipLaunchKernelGGL((mx_rows_kernel<XT, NT, NW, SHORT, true, GROUPED>), grid, dim3(NW * 64), lds, s, a);
}

template <int XT, int MI, int NI, int WM, int WN, int RING, bool GROUPED> void launch_tiles(const MxArgs& a, hipStream_t s) {
  constexpr int TM = 32 * MI * WM, TN = 32 * NI * WN;
  const dim3 grid((unsigned)tile_grid(a.M, a.N, GROUPED ? a.E : 0, TM, TN));
  hipLaunchKernelGGL((mx_tile_kernel<XT, MI, NI, WM, WN, RING, GROUPED>), grid, dim3(WM * WN * 64), 0, s, a, (a.N + TN - 1) / TN);
}

template <int XT, bool GROUPED> void launch_product(const MxArgs& a, const MxPlan& p, hipStream_t s) {
  if constexpr (XT == FP4) {
    if (p.tile == 4) return launch_tiles<XT, 4, 2, 2, 4, 4, GROUPED>(a, s);
    if (p.tile == 3) return launch_tiles<XT, 2, 2, 2, 2, 4, GROUPED>(a, s);
    if (p.tile == 2) return launch_tiles<XT, 1, 2, 2, 2, 4, GROUPED>(a, s);
    if (p.tile == 1) return launch_tiles<XT, 1, 1, 2, 2, 4, GROUPED>(a, s);
  } else {
    if (p.tile == 4) return launch_tiles<XT, 2, 2, 2, 4, 3, GROUPED>(a, s);
    if (p.tile == 3) return launch_tiles<XT, 2, 1, 2, 4, 3, GROUPED>(a, s);
    if (p.tile == 2) return launch_tiles<XT, 2, 1, 1, 4, 3, GROUPED>(a, s);
    if (p.tile == 1) return launch_tiles<XT, 1, 1, 2, 2, 3, GROUPED>(a, s);
  }
  if (a.K < 512 || a.x_rows == 0) return launch_rows<XT, 1, 1, true, GROUPED>(a, s);
  if constexpr (XT != FP4) {   // 16 rows of MXFP4 x fit into LDS for 16 waves
    if (p.nt == 2) return launch_rows<XT, 2, 8, false, GROUPED>(a, s);
  }
  if (p.nw == 2) return launch_rows<XT, 1, 2, false, GROUPED>(a, s);
  if (p.nw == 4) return launch_rows<XT, 1, 4, false, GROUPED>(a, s);
  if (p.nw == 8) return launch_rows<XT, 1, 8, false, GROUPED>(a, s);
  return launch_rows<XT, 1, 16, false, GROUPED>(a, s);
}

void launch_no_k(const MxArgs& a, hipStream_t s) {
  const dim3 grid = ew_grid(1, (int64_t)a.M * a.N), block(EW_THREADS);
  if (a.y_type == F32) hipLaunchKernelGGL(mx_no_k_kernel<F32>, grid, block, 0, s, a);
  else if (a.y_type == F16) hipLaunchKernelGGL(mx_no_k_kernel<F16>, grid, block, 0, s, a);
  else hipLaunchKernelGGL(mx_no_k_kernel<BF16>, grid, block, 0, s, a);
}

template <bool GROUPED> int run_product(MxArgs& a, int x_type, void* stream) {
  const MxPlan p = plan_product(a.M, a.N, a.x_rows > 0 ? a.K : 0, GROUPED ? a.E : 0, x_type);
  if (!p.fits) return QG_E_UNSUPPORTED;
  a.step = p.step;
  int st = device_present();
  if (st != QG_OK) return st;
  const void* ptrs[9] = {a.x, a.xs, a.w, a.ws, a.rows, a.offsets, a.row_scale, a.resid, a.y};
  st = check_device_pointers(ptrs, 9);
  if (st != QG_OK) return st;
  clear_pending_error();
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (!GROUPED && a.K == 0) {
    launch_no_k(a, s);
    return launch_status();
  }
  if (x_type == FP4) launch_product<FP4, GROUPED>(a, p, s);
  else if (x_type == BF16) launch_product<BF16, GROUPED>(a, p, s);
  else launch_product<F16, GROUPED>(a, p, s);
  return launch_status();
}

// Checks shared by the two products; fills the fields that both use.
int setup_product(const void* x, int ldx, int x_type, const uint8_t* xs, int x_rows, const uint8_t* w,
                  const uint8_t* ws, int E, int M, int N, int K, void* y, int ldy, int y_type, MxArgs* a) {
  if (x_type != F16 && x_type != BF16 && x_type != FP4) return QG_E_ARG;
  if (!float_type(y_type) || M < 0 || N < 0 || K < 0 || x_rows < 0 || K % 32) return QG_E_ARG;
  if ((x_type == FP4) != (xs != nullptr) && K > 0 && x_rows > 0) return QG_E_ARG;
  if (E == 0 || M == 0 || N == 0) return QG_OK;
  if (M > INT_MAX - 512 || N > INT_MAX - 512) return QG_E_UNSUPPORTED;   // the kernels round them up in 32 bits
  if (!y || ldy < N) return QG_E_ARG;
  if (K > 0) {
    if (!w || !ws || (x_rows > 0 && !x)) return QG_E_ARG;
    if (x_type == FP4 ? ldx != K : ldx < K) return QG_E_ARG;
    if (!aligned(x, 16) || !aligned(w, 16) || ldx % 8) return QG_E_ALIGN;
  }
  if (!aligned(y, 16)) return QG_E_ALIGN;
  a->x = reinterpret_cast<const char*>(x);
  a->xs = xs; a->w = w; a->ws = ws;
  a->ldx_bytes = x_type == FP4 ? K / 2 : (int64_t)ldx * 2;
  a->x_rows = x_rows; a->M = M; a->N = N; a->K = K;
  a->y = reinterpret_cast<char*>(y);
  a->ldy = ldy; a->y_type = y_type;
  a->rows = nullptr; a->offsets = nullptr; a->row_scale = nullptr; a->E = E;
  a->resid = nullptr; a->ldr = N;
  return QG_OK;
}

}  // namespace
}  // namespace qg

using namespace qg;

extern "C" int qmx_plan(int M, int N, int K, int E, int x_type, int out[4]) {
  if (M < 0 || N < 0 || K < 0 || E < 0 || K % 32 || (x_type != F16 && x_type != BF16 && x_type != FP4) || !out) return QG_E_ARG;
  if (E > 65535 || M > INT_MAX - 512 || N > INT_MAX - 512) return QG_E_UNSUPPORTED;   // as the products
  const MxPlan p = plan_product(M, N, K, E, x_type);
  out[0] = p.tile;
  out[1] = p.tile ? 0 : p.nt;
  out[2] = p.tile ? 0 : p.nw;
  out[3] = (int)std::min<int64_t>(p.workgroups, INT_MAX);
  return QG_OK;
}

extern "C" int qmx_quantize(const void* x, int ldx, int x_type, int M, int K, uint8_t* codes, uint8_t* scales,
                            void* stream) {
  int st = check_matrix(x, ldx, x_type, M, K, codes, scales);
  if (st != QG_OK) return st;
  if (M == 0 || K == 0) return QG_OK;
  st = device_present();
  if (st != QG_OK) return st;
  const void* ptrs[3] = {x, codes, scales};
  st = check_device_pointers(ptrs, 3);
  if (st != QG_OK) return st;
  clear_pending_error();
  const bool flat = ldx == K || M == 1;
  const int64_t rows = flat ? 1 : M, n8 = (flat ? (int64_t)M : 1) * (K / 8);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  uint32_t* c = reinterpret_cast<uint32_t*>(codes);
  const dim3 grid = ew_grid(rows, n8), block(EW_THREADS);
  if (x_type == F16)
    hipLaunchKernelGGL(mx_quantize_kernel<F16>, grid, block, 0, s, reinterpret_cast<const f16*>(x), (int64_t)ldx, rows, n8, c, scales);
  else if (x_type == BF16)
    hipLaunchKernelGGL(mx_quantize_kernel<BF16>, grid, block, 0, s, reinterpret_cast<const bf16*>(x), (int64_t)ldx, rows, n8, c, scales);
  else
    hipLaunchKernelGGL(mx_quantize_kernel<F32>, grid, block, 0, s, reinterpret_cast<const float*>(x), (int64_t)ldx, rows, n8, c, scales);
  return launch_status();
}

extern "C" int qmx_dequantize(const uint8_t* codes, const uint8_t* scales, int M, int K, void* y, int ldy,
                              int y_type, void* stream) {
  int st = check_matrix(y, ldy, y_type, M, K, codes, scales);
  if (st != QG_OK) return st;
  if (M == 0 || K == 0) return QG_OK;
  st = device_present();
  if (st != QG_OK) return st;
  const void* ptrs[3] = {codes, scales, y};
  st = check_device_pointers(ptrs, 3);
  if (st != QG_OK) return st;
  clear_pending_error();
  const bool flat = ldy == K || M == 1;
  const int64_t rows = flat ? 1 : M, n8 = (flat ? (int64_t)M : 1) * (K / 8);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const uint32_t* c = reinterpret_cast<const uint32_t*>(codes);
  const dim3 grid = ew_grid(rows, n8), block(EW_THREADS);
  if (y_type == F16)
    hipLaunchKernelGGL(mx_dequantize_kernel<F16>, grid, block, 0, s, c, scales, rows, n8, reinterpret_cast<f16*>(y), (int64_t)ldy);
  else if (y_type == BF16)
    hipLaunchKernelGGL(mx_dequantize_kernel<BF16>, grid, block, 0, s, c, scales, rows, n8, reinterpret_cast<bf16*>(y), (int64_t)ldy);
  else
    hipLaunchKernelGGL(mx_dequantize_kernel<F32>, grid, block, 0, s, c, scales, rows, n8, reinterpret_cast<float*>(y), (int64_t)ldy);
  return launch_status();
}

extern "C" int qmx_gemm(const void* x, int ldx, int x_type, const uint8_t* x_scales, const uint8_t* w,
                        const uint8_t* w_scales, const void* residual, int ldr, int M, int N, int K, void* y,
                        int ldy, int y_type, void* stream) {
  MxArgs a;
  int st = setup_product(x, ldx, x_type, x_scales, M, w, w_scales, 1, M, N, K, y, ldy, y_type, &a);
  if (st != QG_OK) return st;
  if (M == 0 || N == 0) return QG_OK;
  if (residual) {
    if (ldr < N || (residual == y && ldr != ldy)) return QG_E_ARG;
    if (!aligned(residual, 16)) return QG_E_ALIGN;
    a.resid = reinterpret_cast<const char*>(residual);
    a.ldr = ldr;
  }
  return run_product<false>(a, x_type, stream);
}

extern "C" int qmx_gemm_grouped(const void* x, int ldx, int x_type, const uint8_t* x_scales, int x_rows,
                                const int32_t* rows, const uint8_t* w, const uint8_t* w_scales,
                                const int32_t* offsets, int E, int T, const float* row_scale, int N, int K,
                                void* y, int ldy, int y_type, void* stream) {
  if (E < 0) return QG_E_ARG;
  MxArgs a;
  int st = setup_product(x, ldx, x_type, x_scales, x_rows, w, w_scales, E, T, N, K, y, ldy, y_type, &a);
  if (st != QG_OK) return st;
  if (E == 0 || T == 0 || N == 0) return QG_OK;
  if (!offsets || (!rows && x_rows < T)) return QG_E_ARG;
  if (!aligned(offsets, 4) || !aligned(rows, 4) || !aligned(row_scale, 4)) return QG_E_ALIGN;
  if (E > 65535) return QG_E_UNSUPPORTED;
  a.rows = rows;
  a.offsets = offsets;
  a.row_scale = row_scale;
  return run_product<true>(a, x_type, stream);
}
