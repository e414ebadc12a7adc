// What the kernels that append rows to a KV cache share: the rounding to e4m3 and the
// checks of a sequence.
#pragma once

#include <cuda_fp8.h>

#include "tr_kv.cuh"

// x / s rounded to the nearest fp32, as far as its rounding to e4m3 can tell, from
// r = RN(1 / s): q0 = x r, q = q0 + r (x - q0 s) (Markstein 1990: with fused
// multiply-adds the last step rounds correctly).  For s in [2^-60, 2^60]: x is
// first held to +-most, a bf16 number between 1024 s and 1033 s (the quotient is
// past 448 either way, and nothing overflows; NaN stays), and where the remainder
// underflows the quotient is below 2^-40, which rounds to 0 either way.  The remainder
// is exact and a zero one is made -0, which takes no sign from q0: -0 / s stays -0.
// Other scales (r = 0) take the division itself, which costs two to three times as much.
struct Scale {
  float s, r;
  uint32_t most;  // twice
};
__device__ __forceinline__ Scale make_scale(float s) {
  const uint32_t m = (__float_as_uint(1024.f * s) + 0xFFFFu) >> 16;
  return {s, s >= 0x1p-60f && s <= 0x1p60f ? __frcp_rn(s) : 0.f, m | (m << 16)};
}

// Two fp32 values in one instruction: a * b, and a * b + c.
__device__ __forceinline__ void mul2(float &x, float &y, float a, float b, float m) {
  asm("{ .reg .b64 p, q; mov.b64 p, {%2, %3}; mov.b64 q, {%4, %4}; mul.rn.f32x2 p, p, q; mov.b64 {%0, %1}, p; }"
      : "=f"(x), "=f"(y)
      : "f"(a), "f"(b), "f"(m));
}
__device__ __forceinline__ void fma2(float &x, float &y, float a, float b, float m, float c, float d) {
  asm("{ .reg .b64 p, q, r; mov.b64 p, {%2, %3}; mov.b64 q, {%4, %4}; mov.b64 r, {%5, %6};"
      " fma.rn.f32x2 p, p, q, r; mov.b64 {%0, %1}, p; }"
      : "=f"(x), "=f"(y)
      : "f"(a), "f"(b), "f"(m), "f"(c), "f"(d));
}
// The same rounded down: where the sum is exact only the sign of a zero differs, which is -0
// unless both terms are +0.
__device__ __forceinline__ void fma2_down(float &x, float &y, float a, float b, float m, float c, float d) {
  asm("{ .reg .b64 p, q, r; mov.b64 p, {%2, %3}; mov.b64 q, {%4, %4}; mov.b64 r, {%5, %6};"
      " fma.rm.f32x2 p, p, q, r; mov.b64 {%0, %1}, p; }"
      : "=f"(x), "=f"(y)
      : "f"(a), "f"(b), "f"(m), "f"(c), "f"(d));
}
// bf16 pairs held to +-most; NaN stays.
__device__ __forceinline__ uint32_t hold2(uint32_t x, uint32_t most) {
  uint32_t r;
  asm("{ .reg .b32 p; min.NaN.bf16x2 p, %1, %2; max.NaN.bf16x2 %0, p, %3; }"
      : "=r"(r)
      : "r"(x), "r"(most), "r"(most | 0x80008000u));
  return r;
}

// Eight bf16 values divided by the head's scale and rounded to e4m3 (one
// rounding of the fp32 quotient to nearest even, clamped to +-448).
__device__ __forceinline__ uint2 e4m3_of(const uint4 &x, const Scale &sc) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t r[4];
  if (sc.r != 0.f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t h = hold2(w[i], sc.most);
      const float lo = __uint_as_float(h << 16), hi = __uint_as_float(h & 0xFFFF0000u);
      float p, q, u, v;
      mul2(p, q, lo, hi, sc.r);
      fma2_down(u, v, p, q, -sc.s, lo, hi);
      fma2(p, q, u, v, sc.r, p, q);
      r[i] = __nv_cvt_float2_to_fp8x2(make_float2(p, q), __NV_SATFINITE, __NV_E4M3);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float lo = __uint_as_float(w[i] << 16), hi = __uint_as_float(w[i] & 0xFFFF0000u);
      r[i] = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(lo, sc.s), __fdiv_rn(hi, sc.s)), __NV_SATFINITE, __NV_E4M3);
    }
  }
  return make_uint2(r[0] | (r[1] << 16), r[2] | (r[3] << 16));
}

// The same of eight fp32 values.
__device__ __forceinline__ uint2 e4m3_of(const float (&x)[8], const Scale &sc) {
  uint32_t r[4];
  const float most = __uint_as_float(sc.most << 16);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float p, q;
    if (sc.r != 0.f) {
      float lo, hi, u, v;
      asm("{ .reg .f32 a; min.NaN.f32 a, %1, %2; max.NaN.f32 %0, a, %3; }" : "=f"(lo) : "f"(x[2 * i]), "f"(most), "f"(-most));
      asm("{ .reg .f32 a; min.NaN.f32 a, %1, %2; max.NaN.f32 %0, a, %3; }" : "=f"(hi) : "f"(x[2 * i + 1]), "f"(most), "f"(-most));
      mul2(p, q, lo, hi, sc.r);
      fma2_down(u, v, p, q, -sc.s, lo, hi);
      fma2(p, q, u, v, sc.r, p, q);
    } else {
      p = __fdiv_rn(x[2 * i], sc.s);
      q = __fdiv_rn(x[2 * i + 1], sc.s);
    }
    r[i] = __nv_cvt_float2_to_fp8x2(make_float2(p, q), __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(r[0] | (r[1] << 16), r[2] | (r[3] << 16));
}

// Whether a sequence can take its rows (the same answer in every thread of the
// block; contains a barrier): the rows to copy, or -1 with the status bit set.
__device__ __forceinline__ int append_rows(const KvDev &c, int b, int Lb, int n, int T, unsigned *status) {
  const bool bad_len = Lb < 0 || Lb > c.cap || n < 0 || n > T;
  const bool full = !bad_len && n > c.cap - Lb;
  const bool bad_page = kv_bad_pages(c, b, Lb, bad_len || full ? Lb : Lb + n);
  if (!bad_len && !full && !bad_page) return n;
  if (threadIdx.x == 0) tr_flag(status, bad_len ? TR_DEV_BAD_LENGTH : full ? TR_DEV_CACHE_FULL : TR_DEV_BAD_PAGE);
  return -1;
}
