// What the paged 8-bit cache's kernels share: the device-side description of a
// sequence with its checks, e4m3 conversions, and the error word.
#pragma once
#include <cuda_fp16.h>

#include "dev.cuh"
#include "kernels.h"

namespace thrift {
namespace kv8 {

// One word per translation unit (bit 0: a bad length, range or page number; bit 1: a
// wait that ran out); read_and_clear_* below reads the unit's own.
static __device__ uint32_t g_error_word;

static inline cudaError_t read_and_clear_word(uint32_t* word) {
  uint32_t w = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&w, g_error_word, sizeof(w));
  if (e == cudaSuccess && w != 0) {
    const uint32_t zero = 0;
    e = cudaMemcpyToSymbol(g_error_word, &zero, sizeof(zero));
  }
  *word = w;
  return e;
}

__device__ __forceinline__ void raise_bad() { atomicOr(&g_error_word, 1u); }

// Sequence b of a call: its length, its rows of new tokens and the position of the first
// (negative where there are more new tokens than the length holds).  What the host could
// not check is checked here: a bad length makes the sequence empty, a bad range of new
// tokens makes it have none; `bad` tells the caller to report it.
struct Seq {
  int len, q0, nq, pos0;
  bool bad;
};
__device__ __forceinline__ Seq load_seq(const int32_t* lens, const int32_t* cu, int b, int n, int max_q, int max_len) {
  Seq s;
  s.len = __ldg(lens + b);
  s.bad = s.len < 0 || s.len > max_len;
  if (s.bad) s.len = 0;
  if (cu != nullptr) {
    const int a = __ldg(cu + b), z = __ldg(cu + b + 1);
    const bool wrong = a < 0 || z < a || z > n || z - a > max_q;
    s.bad |= wrong;
    s.q0 = wrong ? 0 : a;
    s.nq = wrong ? 0 : z - a;
  } else {
    s.q0 = b;
    s.nq = 1;
  }
  s.pos0 = s.len - s.nq;
  return s;
}

// Loads of read-only data that stay where they are written: an ordinary
// load may be moved down to its first use, past the wait that it is meant to overlap.
__device__ __forceinline__ uint4 ldg16_now(const void* a) {
  uint4 u;
  asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(a));
  return u;
}
__device__ __forceinline__ uint2 ldg8_now(const void* a) {
  uint2 u;
  asm volatile("ld.global.nc.v2.u32 {%0,%1}, [%2];" : "=r"(u.x), "=r"(u.y) : "l"(a));
  return u;
}
__device__ __forceinline__ float ldg4_now(const float* a) {
  float x;
  asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(x) : "l"(a));
  return x;
}

// Two e4m3 codes (low byte first) -> f16x2, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tmov.b16 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(r) : "h"((unsigned short)two));
  return r;
}
// f16x2 -> two e4m3 codes, round to nearest even, saturating.
__device__ __forceinline__ uint32_t h2_to_e4m3x2(uint32_t h2) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h2));
  return (uint32_t)r;
}

// Four codes of a page with exponent e, rounded again for exponent e + k (k >= 0).  The
// f16 product is exact down to 2^-24; below that it cannot reach 2^-10, half of e4m3's
// smallest step, so its own rounding never changes the code.
__device__ __forceinline__ uint32_t recode4(uint32_t w, __half2 down) {
  const uint32_t lo = e4m3x2_to_h2(w & 0xFFFFu), hi = e4m3x2_to_h2(w >> 16);
  const __half2 a = __hmul2(*reinterpret_cast<const __half2*>(&lo), down);
  const __half2 b = __hmul2(*reinterpret_cast<const __half2*>(&hi), down);
  return h2_to_e4m3x2(*reinterpret_cast<const uint32_t*>(&a)) | (h2_to_e4m3x2(*reinterpret_cast<const uint32_t*>(&b)) << 16);
}
// 2^-k as f16x2; from k = 19 on every code rounds to zero, so larger k may stand as 24.
__device__ __forceinline__ __half2 recode_factor(int k) {
  return __float2half2_rn(pow2f(-(k > 24 ? 24 : k)));
}

// A pair of 16-bit inputs as FP32.
__device__ __forceinline__ float2 pair_to_float2(uint32_t w, bool fp16) {
  if (fp16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t float2_to_pair(float a, float b, bool fp16) {
  if (fp16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  return cvt_bf16x2(a, b);
}

// e + 127 -> 2^e, exact (code 0 gives the subnormal 2^-127).
__device__ __forceinline__ float scale_value(uint32_t code) {
  return code > 0u ? __uint_as_float(code << 23) : __uint_as_float(0x00400000u);
}

}  // namespace kv8
}  // namespace thrift
