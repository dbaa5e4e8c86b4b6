// mx.hip - microscaled 4-bit floating point (MXFP4): quantising and reading
// back, the product y = x . W^T with MXFP4 weights, and that product grouped
// by expert with ragged sizes.  The format and the entry points are described
// in include/qgemm.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <climits>

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
  int y_type, vec;                  // vec: 4 consecutive outputs of a row may be stored at once
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

// Scale bytes for which every code times the scale is an exact fp16 number:
// 0.5 * 2^(104 - 127) = 2^-24, fp16's smallest, and 6 * 2^(140 - 127) = 49152.
__device__ __forceinline__ bool scale_fits_f16(uint32_t s) { return s - 104u <= 36u; }

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

// Four consecutive outputs of one row: columns n .. n+3 of row m.
__device__ __forceinline__ void store4(const MxArgs& a, int m, int n, f4 v, float rs) {
  if (a.row_scale) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] *= rs;
  }
  const int64_t o = (int64_t)m * a.ldy + n, ro = (int64_t)m * a.ldr + n;
  if (a.y_type == F32) {
    float* y = reinterpret_cast<float*>(a.y);
    const float* r = reinterpret_cast<const float*>(a.resid);
    if (a.vec && n + 3 < a.N) {
      if (r) v += *reinterpret_cast<const f4*>(r + ro);
      *reinterpret_cast<f4*>(y + o) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < a.N) y[o + i] = r ? v[i] + r[ro + i] : v[i];
    }
    return;
  }
  uint16_t* y = reinterpret_cast<uint16_t*>(a.y);
  const uint16_t* r = reinterpret_cast<const uint16_t*>(a.resid);
  const bool half = a.y_type == F16;
  const bool wide = a.vec && n + 3 < a.N;
  uint16_t rv[4] = {0, 0, 0, 0}, q[4];
  if (r) {
    if (wide) {
      const u2 t = *reinterpret_cast<const u2*>(r + ro);
      rv[0] = (uint16_t)t.x; rv[1] = (uint16_t)(t.x >> 16); rv[2] = (uint16_t)t.y; rv[3] = (uint16_t)(t.y >> 16);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < a.N) rv[i] = r[ro + i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] += half ? (float)__builtin_bit_cast(f16, rv[i]) : bits_f32((uint32_t)rv[i] << 16);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    q[i] = half ? __builtin_bit_cast(uint16_t, (f16)v[i]) : __builtin_bit_cast(uint16_t, (bf16)v[i]);
  if (wide) {
    *reinterpret_cast<u2*>(y + o) = u2{q[0] | ((uint32_t)q[1] << 16), q[2] | ((uint32_t)q[3] << 16)};
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < a.N) y[o + i] = q[i];
  }
}

// A grouped product's slots of expert e, kept within [0, T] whatever the
// offsets hold.
__device__ __forceinline__ void group_bounds(const MxArgs& a, int e, int& begin, int& end) {
  begin = min(max(a.offsets[e], 0), a.M);
  end = min(max(a.offsets[e + 1], begin), a.M);
}

// Few rows: bound by the weights' bytes.  A workgroup owns 16 columns of y (16
// rows of W) and 16*MT rows of it; its NW waves share K in tiles of 128 and
// are summed through LDS in wave order.  Lane l = 16 g + r of a wave loads the
// 16-byte block 4 t + g of row r (with its scale byte), which is the operand of
// v_mfma_scale_f32_16x16x128 as it is; 16-bit x takes four 16x16x32 steps on
// the block's four words converted to 16 bits, x read at the same k.  W is the
// first operand, so a lane ends with four consecutive outputs of one row.
template <int XT, int MT, int NW, bool GROUPED>
__global__ __launch_bounds__(NW * 64) void mx_rows_kernel(MxArgs a) {
  __shared__ f4 part[NW][MT][64];
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n0 = blockIdx.x * 16;
  const int nkb = a.x_rows > 0 ? a.K >> 5 : 0;   // no x to read: all rows are zero
  const int tiles = (nkb + 3) >> 2;
  int m_begin, m_end;
  int64_t wrow = min(n0 + r, a.N - 1);
  if constexpr (GROUPED) {
    group_bounds(a, blockIdx.y, m_begin, m_end);
    wrow += (int64_t)blockIdx.y * a.N;
  } else {
    m_begin = blockIdx.y * (16 * MT);
    m_end = min(a.M, m_begin + 16 * MT);
  }
  const uint8_t* wp = a.w + wrow * (a.K >> 1);
  const uint8_t* sp = a.ws + wrow * (a.K >> 5);
  for (int m0 = m_begin; m0 < m_end; m0 += 16 * MT) {
    const char* xp[MT];
    const uint8_t* xsp[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      int m = min(m0 + mt * 16 + r, m_end - 1);
      if (GROUPED && a.rows) m = a.rows[m];
      if (m < 0 || m >= a.x_rows) m = 0;         // such a row's sums are not used
      xp[mt] = a.x + m * a.ldx_bytes;
      xsp[mt] = XT == FP4 ? a.xs + (int64_t)m * (a.K >> 5) : nullptr;
    }
    f4 acc[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) acc[mt] = f4{0.f, 0.f, 0.f, 0.f};
    for (int t = wave; t < tiles; t += NW) {
      const bool in = 4 * t + g < nkb;           // past K: zero codes, zero x
      const int kb = min(4 * t + g, nkb - 1);
      u4 c = *reinterpret_cast<const u4*>(wp + kb * 16);
      uint32_t s = sp[kb];
      if (!in) c = u4{0, 0, 0, 0}, s = 127;
      const float sf = scale_f32(s);
      if constexpr (XT == FP4) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          u4 xc = *reinterpret_cast<const u4*>(xp[mt] + kb * 16);
          uint32_t xsc = xsp[mt][kb];
          if (!in) xc = u4{0, 0, 0, 0}, xsc = 127;
          acc[mt] = mfma_fp4(c, s, xc, xsc, acc[mt]);
        }
      } else {
        u4 xv[MT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            xv[mt][j] = reinterpret_cast<const u4*>(xp[mt] + kb * 64)[j];
            if (!in) xv[mt][j] = u4{0, 0, 0, 0};
          }
        if constexpr (XT == BF16) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const b8 wv = codes_bf16(c[j], sf);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
              acc[mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv, __builtin_bit_cast(b8, xv[mt][j]), acc[mt], 0, 0, 0);
          }
        } else if (__all(scale_fits_f16(s))) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const h8 wv = codes_f16(c[j], sf);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
              acc[mt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(wv, __builtin_bit_cast(h8, xv[mt][j]), acc[mt], 0, 0, 0);
          }
        } else {   // scales beyond fp16's range: bf16 weights, x in two exact parts
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const b8 wv = codes_bf16(c[j], sf);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              b8 hi, lo;
              split_f16(__builtin_bit_cast(h8, xv[mt][j]), hi, lo);
              acc[mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv, hi, acc[mt], 0, 0, 0);
              acc[mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv, lo, acc[mt], 0, 0, 0);
            }
          }
        }
      }
    }
    if (m0 != m_begin) __syncthreads();          // the last chunk's sums have been read
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) part[wave][mt][lane] = acc[mt];
    __syncthreads();
    for (int mt = wave; mt < MT; mt += NW) {
      f4 v = part[0][mt][lane];
#pragma unroll
      for (int w = 1; w < NW; ++w) v += part[w][mt][lane];
      const int m = m0 + mt * 16 + r, n = n0 + 4 * g;
      if (m < m_end && n < a.N) {
        if (GROUPED && a.rows) {
          const int xr = a.rows[m];
          if (xr < 0 || xr >= a.x_rows) v = f4{0.f, 0.f, 0.f, 0.f};
        }
        store4(a, m, n, v, GROUPED && a.row_scale ? a.row_scale[m] : 1.f);
      }
    }
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

// Grid of an elementwise kernel over rows x n8 groups: enough workgroups to
// fill the chip eight times over, the rest by the kernel's own loops.
dim3 ew_grid(int64_t rows, int64_t n8) {
  const int64_t bx = std::min<int64_t>((n8 + EW_THREADS - 1) / EW_THREADS, 256 * 16);
  return dim3((unsigned)std::max<int64_t>(bx, 1), (unsigned)std::min<int64_t>(rows, 65535));
}

int launch_status() { return hip_status(hipGetLastError()); }

template <int XT, bool GROUPED> void launch_rows(const MxArgs& a, hipStream_t s) {
  constexpr int NW = 8;
  const unsigned nb = (unsigned)((a.N + 15) / 16);
  const int mt = a.M <= 16 ? 1 : a.M <= 32 ? 2 : 4;
  const unsigned gy = GROUPED ? (unsigned)a.E : (unsigned)((a.M + 16 * mt - 1) / (16 * mt));
  if (mt == 1) hipLaunchKernelGGL((mx_rows_kernel<XT, 1, NW, GROUPED>), dim3(nb, gy), dim3(NW * 64), 0, s, a);
  else if (mt == 2) hipLaunchKernelGGL((mx_rows_kernel<XT, 2, NW, GROUPED>), dim3(nb, gy), dim3(NW * 64), 0, s, a);
  else hipLaunchKernelGGL((mx_rows_kernel<XT, 4, NW, GROUPED>), dim3(nb, gy), dim3(NW * 64), 0, s, a);
}

template <bool GROUPED> int run_product(const MxArgs& a, int x_type, void* stream) {
  int dev = 0;
  int st = current_device(&dev);
  if (st != QG_OK) return st;
  const void* ptrs[9] = {a.x, a.xs, a.w, a.ws, a.rows, a.offsets, a.row_scale, a.resid, a.y};
  st = check_device_pointers(ptrs, 9);
  if (st != QG_OK) return st;
  clear_pending_error();
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (x_type == FP4) launch_rows<FP4, GROUPED>(a, s);
  else if (x_type == BF16) launch_rows<BF16, GROUPED>(a, s);
  else launch_rows<F16, GROUPED>(a, s);
  return launch_status();
}

// Checks shared by the two products; fills the fields that both use.
int setup_product(const void* x, int ldx, int x_type, const uint8_t* xs, int x_rows, const uint8_t* w,
                  const uint8_t* ws, int E, int M, int N, int K, void* y, int ldy, int y_type, MxArgs* a) {
  if (x_type != F16 && x_type != BF16 && x_type != FP4) return QG_E_ARG;
  if (!float_type(y_type) || M < 0 || N < 0 || K < 0 || x_rows < 0 || K % 32) return QG_E_ARG;
  if ((x_type == FP4) != (xs != nullptr) && K > 0 && x_rows > 0) return QG_E_ARG;
  if (E == 0 || M == 0 || N == 0) return QG_OK;
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
  a->vec = ldy % 4 == 0;
  return QG_OK;
}

}  // namespace
}  // namespace qg

using namespace qg;

extern "C" int qmx_quantize(const void* x, int ldx, int x_type, int M, int K, uint8_t* codes, uint8_t* scales,
                            void* stream) {
  int st = check_matrix(x, ldx, x_type, M, K, codes, scales);
  if (st != QG_OK) return st;
  if (M == 0 || K == 0) return QG_OK;
  int dev = 0;
  st = current_device(&dev);
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
  int dev = 0;
  st = current_device(&dev);
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
    a.vec = a.vec && ldr % 4 == 0;
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
