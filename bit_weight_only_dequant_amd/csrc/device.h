// device.h - what the floating-point kernels (mx.hip, f8.hip) share: vector
// types, loads and stores of rows, waits, and the host's small helpers.  Each
// source that includes it has its own copies.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

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
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef int i8v __attribute__((ext_vector_type(8)));

constexpr int F16 = QG_MX_F16, BF16 = QG_MX_BF16, F32 = QG_MX_F32;

template <int T> struct Elem;
template <> struct Elem<F16> { typedef f16 type; };
template <> struct Elem<BF16> { typedef bf16 type; };
template <> struct Elem<F32> { typedef float type; };

__device__ __forceinline__ float bits_f32(uint32_t v) { return __builtin_bit_cast(float, v); }
__device__ __forceinline__ uint32_t f32_bits(float v) { return __builtin_bit_cast(uint32_t, v); }

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

typedef const void __attribute__((address_space(1)))* gptr;
typedef void __attribute__((address_space(3)))* lptr;

// At most N of this wave's global loads are on their way, and none of its LDS
// reads (s_waitcnt vmcnt(N) lgkmcnt(0), GFX9 encoding).
template <int N> __device__ __forceinline__ void wait_loads() {
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}

// All of this wave's LDS reads have arrived (s_waitcnt lgkmcnt(0)).
__device__ __forceinline__ void wait_lds() { __builtin_amdgcn_s_waitcnt(0xc07f); }

// A barrier that waits for LDS accesses only: loads stay on their way.
__device__ __forceinline__ void lds_barrier() {
  wait_lds();
  asm volatile("" ::: "memory");        // no LDS access moves across the barrier
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
bool float_type(int t) { return t == F16 || t == BF16 || t == F32; }
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Grid of an elementwise kernel over rows x n8 groups: as many workgroups along
// a row as fill the chip's wave slots twice (16 a CU, of 4 waves), the rest by
// the kernel's own loops.  A matrix whose rows follow each other is one row
// here; strided rows narrower than a workgroup's 256 groups leave lanes idle
// (K = 32: 4 of 256 work).
dim3 ew_grid(int64_t rows, int64_t n8) {
  const int64_t bx = std::min<int64_t>((n8 + EW_THREADS - 1) / EW_THREADS, 256 * 16);
  return dim3((unsigned)std::max<int64_t>(bx, 1), (unsigned)std::min<int64_t>(rows, 65535));
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

}  // namespace
}  // namespace qg
