// AdamW over many tensors in one launch, with fp32 or e4m3 moments.
//
// One step of every element is the float32 arithmetic of poetx_adamw_multi_step (include/poetx.h).
// With e4m3 moments, 256 consecutive elements of a tensor share two scales, u_m = max|m| / 448 and
// u_r = max sqrt(v) / 448, and hold m / u_m and sqrt(v) / u_r as e4m3 codes.  One warp owns one such
// block: it reads parameters, gradients, codes and scales once, steps in fp32, finds the two new
// maxima with shuffles and writes everything back, so a step is one pass over memory (16 bytes per
// element with fp32 parameters and gradients, against 28 with fp32 moments).
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"
#include "sm100.cuh"

namespace poetx {

constexpr int kMomentBlock = POETX_MOMENT_BLOCK;    // elements that share a pair of moment scales
constexpr int kMultiThreads = 256;
constexpr int kMultiTile = 8 * kMultiThreads;       // elements of one tile: eight per thread
// Tensors of one launch: the table is a kernel argument, copied with every launch, so a short list
// takes a small one.  16 tensors of 4096 elements: 4.3 us of host time a call and 13.7 until a lone one is done with the
// small table, 5.4 and 16.4 with the large one (17 tensors: 5.4 and 16.4); a table between the two could save a
// list that is longer than 16 no more than that, and calls on larger tensors nothing (16 of a million: 51.3 and 51.4).
constexpr int kMultiFew = 16, kMultiMany = 448;

// One tensor of the table.  flags: bit 0 bf16 parameters, bit 1 bf16 gradients, bit 2 e4m3 moments.
struct MultiTensor {
  void* p;
  const void* g;
  void* m;
  void* v;
  float2* scale;
  long n;
  float eta, decay;
  uint32_t salt, flags;
};
struct MultiCfg {
  float beta1, beta2, inv_bc1, inv_sqrt_bc2, eps, minus_zero;
  int count;
  uint32_t stochastic, tiles;
};
template <int MAX>
struct MultiArgs {
  MultiCfg c;
  uint32_t first[MAX];  // first tile of each tensor
  MultiTensor t[MAX];
};
static_assert(sizeof(MultiArgs<kMultiMany>) <= 32764, "the largest kernel argument");

// 32 random bits of element i + e of a tensor (i a multiple of four, e < 4): two rounds of multiply and
// xor-shift over the element's number and the tensor's salt (odd multipliers: fractional bits of the
// golden ratio, sqrt 2 and sqrt 3), then h ^ (h >> 16), which element_finish adds.  A pure function of
// (seed, tensor, element), so a step is reproducible.
__device__ __forceinline__ uint32_t element_bits(long i, int e, uint32_t salt) {
  uint32_t h = (uint32_t)i * 0x9E3779B1u + salt + (uint32_t)((unsigned long)i >> 32) * 0x6A09E667u +
               (uint32_t)e * 0x9E3779B1u;
  h = (h ^ (h >> 16)) * 0x6A09E667u;
  return (h ^ (h >> 15)) * 0xBB67AE85u;
}
__device__ __forceinline__ uint32_t element_finish(uint32_t h) { return h ^ (h >> 16); }
__device__ __forceinline__ uint32_t element_low16(uint32_t h) { return (h ^ (h >> 16)) & 0xFFFFu; }
__device__ __forceinline__ uint32_t element_high16(uint32_t h) { return h >> 16; }

// Pairs of floats in one 64-bit register: one instruction for two roundings (each as the scalar one).
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float lo, float hi) {
  f32x2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void unpair(f32x2 x, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ f32x2 both(float x) { return pair(x, x); }
// A product that keeps its own rounding.  The compiler merges a packed product into the packed sum that follows
// it (one rounding instead of two) even where both say .rn, and sees through a constant zero; with a -0 that
// it cannot know, a b + -0 is a b rounded, in the one instruction a product takes anyway.
__device__ __forceinline__ f32x2 mul2_alone(f32x2 a, f32x2 b, float minus_zero) { return fma2(a, b, both(minus_zero)); }

// |a| <= 448 (or a rounding above) to the e4m3 grid, away from zero with the probability of the part that is cut off
// (16 random bits; the bias is at most 2^-17 of a step); the sign is a bit of its own and stays.  From 2^-6 on the grid
// has 3 mantissa bits: the bits below them are cut after the addition, which carries into the exponent where it
// should (beyond 448 the conversion saturates).  Exact zero stays zero.
__device__ __forceinline__ float e4m3_stochastic(float a, uint32_t rnd16) {
  return __uint_as_float((__float_as_uint(a) + (rnd16 << 4)) & 0xFFF00000u);
}
// The same for 0 <= a < 2^-6, where the grid is the multiples of 2^-9: floor(512 a + rnd / 2^16), the floor by adding
// 2^23 rounded down (exact for these sizes, and no slow conversion instruction).
__device__ __forceinline__ float e4m3_stochastic_small(float a, uint32_t rnd16) {
  const float r = __uint_as_float(0x3F800000u | (rnd16 << 7)) - 1.f;
  return __fmaf_rn(__fadd_rd(__fmaf_rn(a, 512.f, r), 8388608.f), 0.001953125f, -16384.f);
}

// sqrt(v) rounded to nearest, without a branch: s = v y and h = y / 2 from the approximate y = 1 / sqrt(v), then one
// correction s + (v - s^2) h in fused arithmetic (Markstein's final step).  Equal to __fsqrt_rn for every
// float32 from 2^-100 up to the largest finite one (all of them compared: poetx_test_sqrt).
constexpr float kSqrtLow = 7.888609052210118e-31f;  // 2^-100
constexpr float kMaxFinite = 3.402823466e38f;
__device__ __forceinline__ float rsqrt_approx(float v) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v));
  return y;
}
__device__ __forceinline__ f32x2 sqrt2_normal(f32x2 v) {
  float a, b;
  unpair(v, a, b);
  const f32x2 y = pair(rsqrt_approx(a), rsqrt_approx(b));
  const f32x2 s = mul2(v, y);
  return fma2(fma2(mul2(s, both(-1.f)), s, v), mul2(both(0.5f), y), s);
}
// Largest magnitude and largest of three, a NaN on top; smallest magnitude and smallest of three.
__device__ __forceinline__ float max3_abs_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float min3_abs(float a, float b, float c) {
  float d;
  asm("min.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Four values of an fp32 or bf16 array at its element i; the last, partial block of a tensor is
// read value by value, zeros past the end (a zero gradient and moment change nothing there).
template <bool BF>
__device__ __forceinline__ void load4(const void* base, long i, float (&x)[4]) {
  if (BF) {
    const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + i);
    x[0] = __uint_as_float(u.x << 16); x[1] = __uint_as_float(u.x & 0xFFFF0000u);
    x[2] = __uint_as_float(u.y << 16); x[3] = __uint_as_float(u.y & 0xFFFF0000u);
  } else {
    const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
    x[0] = f.x; x[1] = f.y; x[2] = f.z; x[3] = f.w;
  }
}
template <bool BF>
__device__ __forceinline__ void load4_tail(const void* base, long i, long n, float (&x)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = i + e < n ? load_elem(base, i + e, BF ? BF16 : F32) : 0.f;
}
// bf16 results come in already on the bf16 grid or are rounded to nearest here.
template <bool BF>
__device__ __forceinline__ void store4(void* base, long i, const float (&x)[4]) {
  if (BF) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + i) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(base) + i) = make_float4(x[0], x[1], x[2], x[3]);
  }
}
__device__ __forceinline__ uint2 pack4_bf16(const float (&x)[4]) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
template <bool BF>
__device__ __forceinline__ void store4_tail(void* base, long i, long n, const float (&x)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (i + e < n) store_elem(base, i + e, BF ? BF16 : F32, x[e]);
}
__device__ __forceinline__ uint32_t codes4_tail(const uint8_t* c, long i, long n) {
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (i + e < n) w |= (uint32_t)c[i + e] << (8 * e);
  return w;
}
__device__ __forceinline__ void store_codes4_tail(uint8_t* c, long i, long n, uint32_t w) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (i + e < n) c[i + e] = (uint8_t)(w >> (8 * e));
}
__device__ __forceinline__ void decode4(uint32_t w, float (&x)[4]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * h)), __NV_E4M3);
    const float2 f = __half22float2(__half2(r));
    x[2 * h] = f.x;
    x[2 * h + 1] = f.y;
  }
}
__device__ __forceinline__ uint32_t encode4(const float (&q)[4]) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(q[0], q[1]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(q[2], q[3]), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// Four codes of x * inv.  POSITIVE (the root of a second moment): a positive value gets at least the smallest
// code, since m / (0 + eps) must not happen where gradients were seen.  Values under 2^-6 of the grid are rare
// (3.5e-5 of the block's largest), so they take a branch.
template <bool POSITIVE>
__device__ __forceinline__ uint32_t encode_moments(const float (&x)[4], float inv, bool stochastic,
                                                   const uint32_t (&h)[4]) {
  float q[4];
  unpair(mul2(pair(x[0], x[1]), both(inv)), q[0], q[1]);
  unpair(mul2(pair(x[2], x[3]), both(inv)), q[2], q[3]);
  if (__builtin_expect(fminf(min3_abs(q[0], q[1], q[2]), fabsf(q[3])) < 0.015625f, 0)) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (stochastic) {
        const uint32_t r = POSITIVE ? element_high16(h[e]) : element_low16(h[e]);
        q[e] = copysignf(fabsf(q[e]) < 0.015625f ? e4m3_stochastic_small(fabsf(q[e]), r) : e4m3_stochastic(fabsf(q[e]), r),
                         x[e]);
      }
      if (POSITIVE && x[e] > 0.f) q[e] = fmaxf(q[e], 0.001953125f);
    }
  } else if (stochastic) {
#pragma unroll
    for (int e = 0; e < 4; ++e) q[e] = e4m3_stochastic(q[e], POSITIVE ? element_high16(h[e]) : element_low16(h[e]));
  }
  return encode4(q);
}

// Eight elements of one thread: 4 at i0 and 4 at i0 + 128 of the warp's 256-element block.  FULL: all of the
// block's elements exist.
template <bool PBF, bool GBF, bool E4M3, bool FULL>
__device__ __forceinline__ void adamw_block(const MultiTensor& t, const MultiCfg& a, long block, int lane) {
  const long i0 = block * kMomentBlock + 4 * lane;
  uint8_t* const cm = static_cast<uint8_t*>(t.m);
  uint8_t* const cv = static_cast<uint8_t*>(t.v);
  float p[2][4], g[2][4], m[2][4], v[2][4];
  uint32_t wm[2] = {0u, 0u}, wv[2] = {0u, 0u};
  float2 u = make_float2(0.f, 0.f);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (FULL) {
      load4<PBF>(t.p, i0 + 128 * h, p[h]);
      load4<GBF>(t.g, i0 + 128 * h, g[h]);
      if (E4M3) {
        wm[h] = *reinterpret_cast<const uint32_t*>(cm + i0 + 128 * h);
        wv[h] = *reinterpret_cast<const uint32_t*>(cv + i0 + 128 * h);
      } else {
        load4<false>(t.m, i0 + 128 * h, m[h]);
        load4<false>(t.v, i0 + 128 * h, v[h]);
      }
    } else {
      load4_tail<PBF>(t.p, i0 + 128 * h, t.n, p[h]);
      load4_tail<GBF>(t.g, i0 + 128 * h, t.n, g[h]);
      if (E4M3) {
        wm[h] = codes4_tail(cm, i0 + 128 * h, t.n);
        wv[h] = codes4_tail(cv, i0 + 128 * h, t.n);
      } else {
        load4_tail<false>(t.m, i0 + 128 * h, t.n, m[h]);
        load4_tail<false>(t.v, i0 + 128 * h, t.n, v[h]);
      }
    }
  }
  if (E4M3) u = t.scale[block];
  const bool stochastic = a.stochastic != 0;
  const float shrink = t.eta * t.decay, rate = t.eta * a.inv_bc1;
  float top_m = 0.f, top_r = 0.f;  // largest magnitudes, a NaN on top
  uint32_t rnd[2][4] = {};
  // The moments take one rounding per operation (no contraction), so that the codes are a
  // function of the inputs that a float32 restatement reproduces bit for bit.
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (E4M3) {
      decode4(wm[h], m[h]);
      decode4(wv[h], v[h]);
    }
    f32x2 r2[2], m2[2];
    float r[4];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      f32x2 mm = pair(m[h][2 * q], m[h][2 * q + 1]), vv = pair(v[h][2 * q], v[h][2 * q + 1]);
      const f32x2 gg = pair(g[h][2 * q], g[h][2 * q + 1]);
      if (E4M3) {
        mm = mul2(mm, both(u.x));
        vv = mul2(vv, both(u.y));
        vv = mul2(vv, vv);
      }
      m2[q] = add2(mul2_alone(both(a.beta1), mm, a.minus_zero), mul2_alone(both(1.f - a.beta1), gg, a.minus_zero));
      r2[q] = add2(mul2_alone(both(a.beta2), vv, a.minus_zero),
                   mul2_alone(mul2(both(1.f - a.beta2), gg), gg, a.minus_zero));
      unpair(m2[q], m[h][2 * q], m[h][2 * q + 1]);
      unpair(r2[q], v[h][2 * q], v[h][2 * q + 1]);
    }
    const float low = fminf(min3(v[h][0], v[h][1], v[h][2]), v[h][3]);
    const float high = fmaxf(max3(v[h][0], v[h][1], v[h][2]), v[h][3]);
    if (__builtin_expect(low >= kSqrtLow && high <= kMaxFinite, 1)) {
      r2[0] = sqrt2_normal(r2[0]);
      r2[1] = sqrt2_normal(r2[1]);
    } else {
      r2[0] = pair(__fsqrt_rn(v[h][0]), __fsqrt_rn(v[h][1]));
      r2[1] = pair(__fsqrt_rn(v[h][2]), __fsqrt_rn(v[h][3]));
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      unpair(r2[q], r[2 * q], r[2 * q + 1]);
      float d0, d1;
      unpair(fma2(r2[q], both(a.inv_sqrt_bc2), both(a.eps)), d0, d1);
      const f32x2 up = mul2(mul2(m2[q], both(rate)), pair(rcp_approx(d0), rcp_approx(d1)));
      const f32x2 th = pair(p[h][2 * q], p[h][2 * q + 1]);
      unpair(fma2(fma2(both(shrink), th, up), both(-1.f), th), p[h][2 * q], p[h][2 * q + 1]);
    }
    if (stochastic && (E4M3 || PBF)) {
#pragma unroll
      for (int e = 0; e < 4; ++e) rnd[h][e] = element_bits(i0 + 128 * h, e, t.salt);
    }
    uint2 pw = make_uint2(0u, 0u);  // bf16 parameters
    if (PBF) {
      const float any = max3_abs_nan(max3_abs_nan(p[h][0], p[h][1], p[h][2]), p[h][3], 0.f);
      if (stochastic && __builtin_expect(any == any, 1)) {
        // Random bits under the last one kept, the upper halves of the sums (an infinity keeps its bits).
        uint32_t x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = __float_as_uint(p[h][e]) + ((element_finish(rnd[h][e]) * 0xBB67AE85u) >> 16);
        pw = make_uint2(__byte_perm(x[0], x[1], 0x7632), __byte_perm(x[2], x[3], 0x7632));
      } else {
        if (stochastic) {  // a NaN stays one; its neighbours are rounded as ever
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (p[h][e] == p[h][e])
              p[h][e] = __uint_as_float((__float_as_uint(p[h][e]) + ((element_finish(rnd[h][e]) * 0xBB67AE85u) >> 16)) &
                                        0xFFFF0000u);
        }
        pw = pack4_bf16(p[h]);
      }
    }
    if (FULL) {
      if (PBF) *reinterpret_cast<uint2*>(static_cast<uint16_t*>(t.p) + i0 + 128 * h) = pw;
      else store4<false>(t.p, i0 + 128 * h, p[h]);
      if (!E4M3) {
        store4<false>(t.m, i0 + 128 * h, m[h]);
        store4<false>(t.v, i0 + 128 * h, v[h]);
      }
    } else {
      if (PBF) {
        p[h][0] = __uint_as_float(pw.x << 16); p[h][1] = __uint_as_float(pw.x & 0xFFFF0000u);
        p[h][2] = __uint_as_float(pw.y << 16); p[h][3] = __uint_as_float(pw.y & 0xFFFF0000u);
      }
      store4_tail<PBF>(t.p, i0 + 128 * h, t.n, p[h]);
      if (!E4M3) {
        store4_tail<false>(t.m, i0 + 128 * h, t.n, m[h]);
        store4_tail<false>(t.v, i0 + 128 * h, t.n, v[h]);
      }
    }
    if (E4M3) {
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        top_m = max3_abs_nan(top_m, m[h][e], m[h][e + 1]);
        top_r = max3_nan(top_r, r[e], r[e + 1]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) v[h][e] = r[e];
    }
  }
  if (!E4M3) return;
  // Bit patterns of magnitudes order as the numbers do, infinities and NaN on top.
  uint32_t most_m = __reduce_max_sync(0xffffffffu, __float_as_uint(top_m));
  uint32_t most_r = __reduce_max_sync(0xffffffffu, __float_as_uint(top_r));
  uint32_t bad_m[2] = {0u, 0u}, bad_r[2] = {0u, 0u};
  if (__builtin_expect(max(most_m, most_r) >= 0x7F800000u, 0)) {
    // A NaN or an infinity is left out of the block's maximum and stored as the NaN code.
    most_m = most_r = 0u;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (!(fabsf(m[h][e]) <= kMaxFinite)) { bad_m[h] |= 0x7Fu << (8 * e); m[h][e] = 0.f; }
        if (!(v[h][e] <= kMaxFinite)) { bad_r[h] |= 0x7Fu << (8 * e); v[h][e] = 0.f; }
        most_m = max(most_m, __float_as_uint(fabsf(m[h][e])));
        most_r = max(most_r, __float_as_uint(v[h][e]));
      }
    most_m = __reduce_max_sync(0xffffffffu, most_m);
    most_r = __reduce_max_sync(0xffffffffu, most_r);
  }
  // A block whose largest is under 2^-100 is stored as zeros (448 / top would overflow).  Odd lanes divide for the
  // roots, even ones for the first moments.
  const float top = __uint_as_float(lane & 1 ? most_r : most_m);
  const float tops = top < kSqrtLow ? 0.f : top;
  const float inv = tops > 0.f ? __fmul_rn(448.f, __frcp_rn(tops)) : 0.f;
  const float inv_m = __shfl_sync(0xffffffffu, inv, 0), inv_r = __shfl_sync(0xffffffffu, inv, 1);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    wm[h] = encode_moments<false>(m[h], inv_m, stochastic, rnd[h]) | bad_m[h];
    wv[h] = encode_moments<true>(v[h], inv_r, stochastic, rnd[h]) | bad_r[h];
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (FULL) {
      *reinterpret_cast<uint32_t*>(cm + i0 + 128 * h) = wm[h];
      *reinterpret_cast<uint32_t*>(cv + i0 + 128 * h) = wv[h];
    } else {
      store_codes4_tail(cm, i0 + 128 * h, t.n, wm[h]);
      store_codes4_tail(cv, i0 + 128 * h, t.n, wv[h]);
    }
  }
  if (lane < 2) reinterpret_cast<float*>(t.scale + block)[lane] = __fmul_rn(tops, 1.f / 448.f);
}

template <bool PBF, bool GBF, bool E4M3>
__device__ __forceinline__ void adamw_any(const MultiTensor& t, const MultiCfg& a, long block, int lane) {
  if ((block + 1) * kMomentBlock <= t.n) adamw_block<PBF, GBF, E4M3, true>(t, a, block, lane);
  else adamw_block<PBF, GBF, E4M3, false>(t, a, block, lane);
}

// Tiles of 2048 elements (eight 256-element blocks, one per warp) over all tensors.  Each block of threads
// takes a run of consecutive tiles: it finds the first one's tensor by bisection in the table and walks on from
// there.  The table is a kernel argument (constant memory): nothing is uploaded, and a captured launch keeps its own.
template <int MAX>
__global__ void __launch_bounds__(kMultiThreads, 4) adamw_multi_kernel(const __grid_constant__ MultiArgs<MAX> args) {
  sm100::griddep_wait();
  const MultiCfg& a = args.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t tile = (uint32_t)((unsigned long)a.tiles * blockIdx.x / gridDim.x);
  const uint32_t end = (uint32_t)((unsigned long)a.tiles * (blockIdx.x + 1) / gridDim.x);
  int at = 0, hi = a.count - 1;
  while (at < hi) {
    const int mid = (at + hi + 1) >> 1;
    if (args.first[mid] <= tile) at = mid; else hi = mid - 1;
  }
  for (; tile < end; ++tile) {
    if (at + 1 < a.count && tile >= args.first[at + 1]) ++at;  // every listed tensor has a tile
    const MultiTensor& t = args.t[at];
    const long block = (long)(tile - args.first[at]) * (kMultiTile / kMomentBlock) + warp;
    if (block * kMomentBlock >= t.n) continue;  // past the tensor's last block (the whole warp)
    switch (t.flags) {
      case 0: adamw_any<false, false, false>(t, a, block, lane); break;
      case 1: adamw_any<true, false, false>(t, a, block, lane); break;
      case 2: adamw_any<false, true, false>(t, a, block, lane); break;
      case 3: adamw_any<true, true, false>(t, a, block, lane); break;
      case 4: adamw_any<false, false, true>(t, a, block, lane); break;
      case 5: adamw_any<true, false, true>(t, a, block, lane); break;
      case 6: adamw_any<false, true, true>(t, a, block, lane); break;
      default: adamw_any<true, true, true>(t, a, block, lane); break;
    }
  }
}

}  // namespace poetx
