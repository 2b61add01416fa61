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
// takes a small one.
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
  float beta1, beta2, inv_bc1, inv_sqrt_bc2, eps;
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

// 32 random bits of element i of a tensor: two rounds of multiply and xor-shift over the element's
// number and the tensor's salt (odd multipliers: fractional bits of the golden ratio, sqrt 2 and
// sqrt 3).  A pure function of (seed, tensor, element), so a step is reproducible.
__device__ __forceinline__ uint32_t element_bits(long i, uint32_t salt) {
  uint32_t h = (uint32_t)i * 0x9E3779B1u + salt + (uint32_t)((unsigned long)i >> 32) * 0x6A09E667u;
  h = (h ^ (h >> 16)) * 0x6A09E667u;
  h = (h ^ (h >> 15)) * 0xBB67AE85u;
  return h ^ (h >> 16);
}

// |y| <= 448 rounded to the e4m3 grid, up with the probability of the part that is cut off (16 random
// bits; the bias is at most 2^-17 of a step).  From 2^-6 on the grid has 3 mantissa bits: the bits
// below them are cut after the addition, which carries into the exponent where it should; under 2^-6 it
// is the multiples of 2^-9.
__device__ __forceinline__ float e4m3_stochastic(float a, uint32_t rnd16) {
  const float normal = __uint_as_float((__float_as_uint(a) + (rnd16 << 4)) & 0xFFF00000u);
  const float small = floorf(__fadd_rn(a * 512.f, (float)rnd16 * (1.f / 65536.f))) * (1.f / 512.f);
  return fminf(a < 0.015625f ? small : normal, 448.f);
}

template <bool BF>
__device__ __forceinline__ void load4(const void* base, long i, long n, float (&x)[4]) {
  if (i + 4 <= n) {
    if (BF) {
      const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + i);
      x[0] = __uint_as_float(u.x << 16); x[1] = __uint_as_float(u.x & 0xFFFF0000u);
      x[2] = __uint_as_float(u.y << 16); x[3] = __uint_as_float(u.y & 0xFFFF0000u);
    } else {
      const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
      x[0] = f.x; x[1] = f.y; x[2] = f.z; x[3] = f.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = i + e < n ? load_elem(base, i + e, BF ? BF16 : F32) : 0.f;
  }
}

// bf16 results come in already on the bf16 grid or are rounded to nearest here.
template <bool BF>
__device__ __forceinline__ void store4(void* base, long i, long n, const float (&x)[4]) {
  if (i + 4 <= n) {
    if (BF) {
      const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + i) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    } else {
      *reinterpret_cast<float4*>(static_cast<float*>(base) + i) = make_float4(x[0], x[1], x[2], x[3]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (i + e < n) store_elem(base, i + e, BF ? BF16 : F32, x[e]);
  }
}

__device__ __forceinline__ uint32_t load4_codes(const uint8_t* c, long i, long n) {
  if (i + 4 <= n) return *reinterpret_cast<const uint32_t*>(c + i);
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (i + e < n) w |= (uint32_t)c[i + e] << (8 * e);
  return w;
}
__device__ __forceinline__ void store4_codes(uint8_t* c, long i, long n, uint32_t w) {
  if (i + 4 <= n) {
    *reinterpret_cast<uint32_t*>(c + i) = w;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (i + e < n) c[i + e] = (uint8_t)(w >> (8 * e));
  }
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

// Largest finite magnitude; a block whose largest is under 2^-100 is stored as zeros (448 / top would
// overflow).
__device__ __forceinline__ float warp_top(float top) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  return top < 7.888609052210118e-31f ? 0.f : top;
}
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.f;  // NaN and infinity count as nothing
}

// Eight elements of one thread: 4 at i0 and 4 at i0 + 128 of the warp's 256-element block.
template <bool PBF, bool GBF, bool E4M3>
__device__ __forceinline__ void adamw_block(const MultiTensor& t, const MultiCfg& a, long block, int lane) {
  const long n = t.n, i0 = block * kMomentBlock + 4 * lane;
  float p[2][4], g[2][4], m[2][4], v[2][4];
  float2 u = make_float2(0.f, 0.f);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const long i = i0 + 128 * h;
    load4<PBF>(t.p, i, n, p[h]);
    load4<GBF>(t.g, i, n, g[h]);
    if (E4M3) {
      const uint32_t cm = load4_codes(static_cast<const uint8_t*>(t.m), i, n);
      const uint32_t cv = load4_codes(static_cast<const uint8_t*>(t.v), i, n);
      decode4(cm, m[h]);
      decode4(cv, v[h]);
    } else {
      load4<false>(t.m, i, n, m[h]);
      load4<false>(t.v, i, n, v[h]);
    }
  }
  if (E4M3) u = t.scale[block];
  float top_m = 0.f, top_r = 0.f;
  uint32_t rnd[2][4];
  // The moments take one rounding per operation (no contraction), so that the codes are a
  // function of the inputs that a float32 restatement reproduces bit for bit.
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float gg = g[h][e];
      float mm = m[h][e], vv = v[h][e];
      if (E4M3) {
        mm = __fmul_rn(mm, u.x);
        const float r0 = __fmul_rn(vv, u.y);
        vv = __fmul_rn(r0, r0);
      }
      mm = __fadd_rn(__fmul_rn(a.beta1, mm), __fmul_rn(1.f - a.beta1, gg));
      vv = __fadd_rn(__fmul_rn(a.beta2, vv), __fmul_rn(__fmul_rn(1.f - a.beta2, gg), gg));
      const float r = __fsqrt_rn(vv);
      const float denom = r * a.inv_sqrt_bc2 + a.eps;
      float th = p[h][e];
      th = th - t.eta * (t.decay * th + __fdividef(mm * a.inv_bc1, denom));
      m[h][e] = mm;
      v[h][e] = E4M3 ? r : vv;
      if (a.stochastic && (E4M3 || PBF)) rnd[h][e] = element_bits(i0 + 128 * h + e, t.salt);
      if (PBF && a.stochastic) {
        const uint32_t b = __float_as_uint(th);
        if ((b & 0x7F800000u) != 0x7F800000u)
          th = __uint_as_float((b + ((rnd[h][e] * 0xBB67AE85u) >> 16)) & 0xFFFF0000u);
      }
      p[h][e] = th;
      if (E4M3) {
        top_m = fmaxf(top_m, finite_abs(mm));
        top_r = fmaxf(top_r, finite_abs(r));
      }
    }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const long i = i0 + 128 * h;
    store4<PBF>(t.p, i, n, p[h]);
    if (!E4M3) {
      store4<false>(t.m, i, n, m[h]);
      store4<false>(t.v, i, n, v[h]);
    }
  }
  if (!E4M3) return;
  top_m = warp_top(top_m);
  top_r = warp_top(top_r);
  const float inv_m = top_m > 0.f ? __fdiv_rn(448.f, top_m) : 0.f;
  const float inv_r = top_r > 0.f ? __fdiv_rn(448.f, top_r) : 0.f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float qm[4], qr[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = m[h][e], r = v[h][e];
      float am = fminf(fabsf(__fmul_rn(x, inv_m)), 448.f), ar = fminf(__fmul_rn(r, inv_r), 448.f);
      if (a.stochastic) {
        am = e4m3_stochastic(am, rnd[h][e] & 0xFFFFu);
        ar = e4m3_stochastic(ar, rnd[h][e] >> 16);
      }
      // The smallest code stands in for a second moment that would round to zero: m / (0 + eps) must
      // not happen where gradients were seen.
      if (r > 0.f) ar = fmaxf(ar, 0.001953125f);
      const float nan = __uint_as_float(0x7FC00000u);
      qm[e] = fabsf(x) <= 3.402823466e38f ? copysignf(am, x) : nan;
      qr[e] = r <= 3.402823466e38f ? ar : nan;
    }
    store4_codes(static_cast<uint8_t*>(t.m), i0 + 128 * h, n, encode4(qm));
    store4_codes(static_cast<uint8_t*>(t.v), i0 + 128 * h, n, encode4(qr));
  }
  if (lane == 0) t.scale[block] = make_float2(__fdiv_rn(top_m, 448.f), __fdiv_rn(top_r, 448.f));
}

// Tiles of 2048 elements (eight 256-element blocks, one per warp) over all tensors; a block of threads
// takes every gridDim-th tile and finds its tensor by bisection in the table, which sits in constant
// memory because it is a kernel argument: nothing is uploaded, and a captured launch keeps its own copy.
template <int MAX>
__global__ void __launch_bounds__(kMultiThreads) adamw_multi_kernel(const __grid_constant__ MultiArgs<MAX> args) {
  sm100::griddep_wait();
  const MultiCfg& a = args.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (uint32_t tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
    int lo = 0, hi = a.count - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (args.first[mid] <= tile) lo = mid; else hi = mid - 1;
    }
    const MultiTensor& t = args.t[lo];
    const long block = (long)(tile - args.first[lo]) * (kMultiTile / kMomentBlock) + warp;
    if (block * kMomentBlock >= t.n) continue;  // past the tensor's last block (the whole warp)
    switch (t.flags) {
      case 0: adamw_block<false, false, false>(t, a, block, lane); break;
      case 1: adamw_block<true, false, false>(t, a, block, lane); break;
      case 2: adamw_block<false, true, false>(t, a, block, lane); break;
      case 3: adamw_block<true, true, false>(t, a, block, lane); break;
      case 4: adamw_block<false, false, true>(t, a, block, lane); break;
      case 5: adamw_block<true, false, true>(t, a, block, lane); break;
      case 6: adamw_block<false, true, true>(t, a, block, lane); break;
      default: adamw_block<true, true, true>(t, a, block, lane); break;
    }
  }
}

}  // namespace poetx
