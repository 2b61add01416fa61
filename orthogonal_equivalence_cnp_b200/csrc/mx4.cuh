// MX4: a weight in 4 bits (the OCP microscaled format MXFP4) and its products with bf16 activations.
//
// codes[r][c / 2] holds the e2m1 codes of columns c (low nibble) and c + 1; scales[r][c / 32] is the
// exponent plus 127 of the power of two that 32 consecutive columns share (255: NaN).  A code is
// sign, two exponent bits (bias 1), one mantissa bit: 0, 1/2, 1, 3/2, 2, 3, 4, 6.
#pragma once

#include <cuda_fp4.h>

#include <type_traits>

#include "common.cuh"
#include "sm100.cuh"

namespace poetx {

constexpr int KID_MX4 = 9;  // kernel id in the device error word

// ------------------------------------------------------------------- codes to bf16, exactly
// bf16x2 factors of one scale: 2^(e - 1) as a product of two, since it may pass bf16's range (the
// second is 1 for e <= 128, so only scales above 2 take two multiplications).
struct Mx4Scale {
  uint32_t f1, f2;
  bool two;
};
__device__ __forceinline__ Mx4Scale mx4_scale(uint32_t e) {
  Mx4Scale s;
  const uint32_t lo = min(e, 128u);
  s.f1 = e == 255u ? 0x7FC07FC0u : (lo + 126u) * 0x00800080u;
  s.f2 = (e - 1u) * 0x00800080u;  // 2^(e - 128), read only for 128 < e < 255
  s.two = e > 128u && e < 255u;
  return s;
}
__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// A word of four nibbles in each half (bits 4i..4i+3) to four bf16x2: result i holds nibble i of both
// halves, times f1.  Masked, a nibble s e e m times 2^6 + 2^12 puts e e m at a bf16's lowest exponent and
// highest mantissa bits and s at its sign: the value times 2^-126 (a subnormal for 0 and 1/2), so one exact
// product with 2^126 times the scale finishes it.  Integer logic runs at half the rate of multiplications here and
// is what bounds decoding, hence the multiplication in place of two shifts: 9 logic operations for eight weights.
__device__ __forceinline__ void mx4_nibbles(uint32_t p, uint32_t f1, uint32_t (&o)[4]) {
  const uint32_t q = p >> 8;
  o[0] = bf16x2_mul(((p & 0x000F000Fu) * 0x1040u) & 0x81C081C0u, f1);
  o[1] = bf16x2_mul(((p & 0x00F000F0u) * 0x0104u) & 0x81C081C0u, f1);
  o[2] = bf16x2_mul(((q & 0x000F000Fu) * 0x1040u) & 0x81C081C0u, f1);
  o[3] = bf16x2_mul(((q & 0x00F000F0u) * 0x0104u) & 0x81C081C0u, f1);
}
// Eight codes (w: code e in bits 4e..4e+3) to eight bf16 values, times f1: in column order (four permutations
// more), or in the order 0, 4, 1, 5, 2, 6, 3, 7 as mx4_nibbles has them.
template <bool ORDERED = true>
__device__ __forceinline__ uint4 mx4_decode8(uint32_t w, uint32_t f1) {
  uint32_t o[4];
  mx4_nibbles(w, f1, o);
  if (!ORDERED) return make_uint4(o[0], o[1], o[2], o[3]);
  return make_uint4(__byte_perm(o[0], o[1], 0x5410), __byte_perm(o[2], o[3], 0x5410), __byte_perm(o[0], o[1], 0x7632),
                    __byte_perm(o[2], o[3], 0x7632));
}
template <bool ORDERED = true>
__device__ __forceinline__ uint4 mx4_decode8(uint32_t w, const Mx4Scale& s) {
  uint4 o = mx4_decode8<ORDERED>(w, s.f1);
  if (s.two) o = make_uint4(bf16x2_mul(o.x, s.f2), bf16x2_mul(o.y, s.f2), bf16x2_mul(o.z, s.f2), bf16x2_mul(o.w, s.f2));
  return o;
}

// --------------------------------------------------------------------------- quantisation
// A thread takes eight columns, four threads one scale: the block's largest magnitude meets by two
// shuffles, its exponent gives the scale, and the values times the scale's inverse (a power of two: exact)
// round to nearest even in the conversion instruction.  One pass, coalesced both ways: HBM bound, so each thread
// has MX4_AT_ONCE pieces' loads under way before it works on the first.
constexpr int MX4_AT_ONCE = 4;
template <bool BF>
__device__ __forceinline__ void mx4_quantize8(const uint4 (&in)[2], long i, uint32_t mask, uint32_t* codes, uint8_t* scales) {
  float x[8];
  const uint32_t w0[4] = {in[0].x, in[0].y, in[0].z, in[0].w}, w1[4] = {in[1].x, in[1].y, in[1].z, in[1].w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (BF) {
      x[2 * e] = __uint_as_float(w0[e] << 16);
      x[2 * e + 1] = __uint_as_float(w0[e] & 0xFFFF0000u);
    } else {
      x[e] = __uint_as_float(w0[e]);
      x[4 + e] = __uint_as_float(w1[e]);
    }
  }
  uint32_t top = 0u;  // magnitudes ordered as integers: infinities and NaN end on top
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(fabsf(x[e])));
  top = max(top, __shfl_xor_sync(mask, top, 1));
  top = max(top, __shfl_xor_sync(mask, top, 2));
  uint32_t w = 0u, scale = 255u;  // a block with a NaN or an infinity reads back as NaN
  if (top < 0x7F800000u) {
    scale = (uint32_t)max((int)(top >> 23) - 2, 0);
    const float inv = __uint_as_float((254u - scale) << 23);  // 2^(127 - scale); scale <= 252, so a normal number
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w |= (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(x[2 * e] * inv, x[2 * e + 1] * inv), __NV_E2M1,
                                              cudaRoundNearest)
           << (8 * e);
  }
  codes[i] = w;
  if ((i & 3) == 0) scales[i >> 2] = (uint8_t)scale;
}

template <bool BF>
__global__ void __launch_bounds__(256) mx4_quantize_kernel(const uint4* __restrict__ W, long chunks,
                                                           uint32_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  sm100::griddep_wait();
  constexpr int U = BF ? MX4_AT_ONCE : MX4_AT_ONCE / 2, V = BF ? 1 : 2;  // 16-byte loads per chunk: V
  // Batches while the whole warp has one; then piece by piece, where a warp may end in the middle: chunks and strides
  // are multiples of 4, so the four threads of a scale go together, and their shuffles name them alone.
  const long stride = (long)gridDim.x * blockDim.x;
  long i = (long)blockIdx.x * blockDim.x + threadIdx.x;
  for (; (i | 31) + (U - 1) * stride < chunks; i += U * stride) {
    uint4 in[U][2] = {};
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int v = 0; v < V; ++v) in[u][v] = W[(i + u * stride) * V + v];
#pragma unroll
    for (int u = 0; u < U; ++u) mx4_quantize8<BF>(in[u], i + u * stride, 0xffffffffu, codes, scales);
  }
  for (; i < chunks; i += stride) {
    uint4 in[2] = {};
#pragma unroll
    for (int v = 0; v < V; ++v) in[v] = W[i * V + v];
    mx4_quantize8<BF>(in, i, 0xFu << (threadIdx.x & 28), codes, scales);
  }
}

// bf16 values of codes and scales, eight columns per piece.
__global__ void __launch_bounds__(256) mx4_dequantize_kernel(const uint32_t* __restrict__ codes,
                                                             const uint8_t* __restrict__ scales, long chunks,
                                                             uint4* __restrict__ W) {
  sm100::griddep_wait();
  const long stride = (long)gridDim.x * blockDim.x;
  long i = (long)blockIdx.x * blockDim.x + threadIdx.x;
  for (; i + (MX4_AT_ONCE - 1) * stride < chunks; i += MX4_AT_ONCE * stride) {
    uint32_t w[MX4_AT_ONCE], e[MX4_AT_ONCE];
#pragma unroll
    for (int u = 0; u < MX4_AT_ONCE; ++u) {
      w[u] = codes[i + u * stride];
      e[u] = scales[(i + u * stride) >> 2];
    }
#pragma unroll
    for (int u = 0; u < MX4_AT_ONCE; ++u) W[i + u * stride] = mx4_decode8(w[u], mx4_scale(e[u]));
  }
  for (; i < chunks; i += stride) W[i] = mx4_decode8(codes[i], mx4_scale(scales[i >> 2]));
}

// ------------------------------------------------------------------- product, few tokens
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8 NT tokens a block.  For few tokens the product is bound by reading the codes once (and by decoding them), so
// nothing is staged: every thread loads codes straight into the registers that the warp-level tensor instruction
// takes them from.  The order of the K index inside an instruction is free as long as both operands agree, so a
// thread takes the K positions whose codes lie together in memory.  The warps of a block, and the blocks of a
// cluster, split K and add their sums in shared memory in a fixed order.
struct Mx4FewArgs {
  int M, N, K;  // features out, tokens, features in
  int splits;   // CTAs of a cluster, along K
  const __nv_bfloat16* X;
  const uint8_t* codes;
  const uint8_t* scales;
  __nv_bfloat16* Y;
};
constexpr int MX4_FEW_RT = 2;                   // forward: 16-row tiles per block
constexpr int MX4_FEW_ROWS = 16 * MX4_FEW_RT;   // features of a forward block
constexpr int MX4_FEW_COLS = 128;               // features of an adjoint block
// Warps of a block.  One token, 4096 x 14336 (31.2 MB of codes and scales, 4.8 us at the copy rate): forward 12.7 us
// with 4 warps and 4 blocks per SM, 13.5 with 8 and 2, 14.9 with 16 rows a block (12.3, 2.5 TB/s, since the sums
// meet no bank twice); adjoint 17.5 to 18.5 with 8 warps, 29 with 4 (too few warps for its 32 column tiles).
__host__ __device__ constexpr int mx4_few_warps(bool adj) { return adj ? 8 : 4; }
// A warp's sums in shared memory: [token][feature], a feature's place and the tokens' stride such that both the
// accumulators' stores (eight features 1 or 16 apart, four pairs of tokens) and the reads along the features meet
// no bank twice.
__host__ __device__ constexpr int mx4_few_stride(bool adj) { return adj ? 140 : 36; }
template <bool ADJ>
__device__ __forceinline__ int mx4_few_place(int feature) { return ADJ ? feature + (feature >> 4) : feature; }
__host__ __device__ constexpr size_t mx4_few_smem(bool adj, int nt) {
  return (size_t)mx4_few_warps(adj) * mx4_few_stride(adj) * 8 * nt * sizeof(float);
}

// Sums the warps' results and the cluster's, rounds once, stores; two features at a time (M is even).
template <bool ADJ, int T>
__device__ __forceinline__ void mx4_few_finish(const Mx4FewArgs& a, float* red, int m0, int n0, int split) {
  using namespace sm100;
  constexpr int F = ADJ ? MX4_FEW_COLS : MX4_FEW_ROWS, S = mx4_few_stride(ADJ), WARPS = mx4_few_warps(ADJ);
  const int pairs = F / 2 * min(T, a.N - n0);
  auto store = [&](int e, float lo, float hi) {
    const int n = n0 + e / (F / 2), m = m0 + e % (F / 2) * 2;
    if (m < a.M) *reinterpret_cast<uint32_t*>(a.Y + (size_t)n * a.M + m) = pack_bf16x2(lo, hi);
  };
  __syncthreads();
  for (int e = threadIdx.x; e < pairs; e += WARPS * 32) {
    float* at = red + e / (F / 2) * S;
    const int f = e % (F / 2) * 2, f0 = mx4_few_place<ADJ>(f), f1 = mx4_few_place<ADJ>(f + 1);
    float lo = at[f0], hi = at[f1];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) {
      lo += at[w * T * S + f0];
      hi += at[w * T * S + f1];
    }
    if (a.splits == 1) {
      store(e, lo, hi);
    } else {
      at[f0] = lo;
      at[f1] = hi;
    }
  }
  if (a.splits == 1) return;
  cluster_sync_all();
  for (int e = pairs * split / a.splits + threadIdx.x; e < pairs * (split + 1) / a.splits; e += WARPS * 32) {
    const int f = e % (F / 2) * 2;
    const uint32_t at = smem_u32(red + e / (F / 2) * S);
    const uint32_t a0 = at + 4 * mx4_few_place<ADJ>(f), a1 = at + 4 * mx4_few_place<ADJ>(f + 1);
    float lo = 0.f, hi = 0.f;
    for (int r = 0; r < a.splits; ++r) {
      lo += ld_cluster_f32(mapa_shared(a0, (uint32_t)r));
      hi += ld_cluster_f32(mapa_shared(a1, (uint32_t)r));
    }
    store(e, lo, hi);
  }
  cluster_sync_all();  // the peers have read this block's sums
}

// Forward: 32 features a block; a warp takes 128 input features at a time, thread (g, t) = (lane / 4, lane % 4) the
// 32 codes (one scale) of rows g, g + 8, .. at 32 t, and token g's 32 values there.
template <int NT>
__global__ void __launch_bounds__(mx4_few_warps(false) * 32, 4) mx4_few_forward(const Mx4FewArgs a) {
  using namespace sm100;
  extern __shared__ float red[];
  constexpr int RT = MX4_FEW_RT, WARPS = mx4_few_warps(false);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int split = (int)(blockIdx.x % a.splits), m0 = (int)(blockIdx.x / a.splits) * MX4_FEW_ROWS;
  const int n0 = blockIdx.y * (8 * NT);
  const int nb = (a.K + 127) / 128;
  const int b_lo = (int)((long)nb * split / a.splits), b_hi = (int)((long)nb * (split + 1) / a.splits);
  float acc[RT][NT][4] = {};
  griddep_wait();
  // Rows and tokens past the end repeat the last one: what they give is never stored.
  const uint8_t* code_at[2 * RT];
  const uint8_t* scale_at[2 * RT];
#pragma unroll
  for (int r = 0; r < 2 * RT; ++r) {
    const int m = min(m0 + 8 * r + g, a.M - 1);
    code_at[r] = a.codes + (size_t)m * (a.K / 2) + 16 * t;
    scale_at[r] = a.scales + (size_t)m * (a.K / 32) + t;
  }
  const __nv_bfloat16* x_at[NT];
#pragma unroll
  for (int u = 0; u < NT; ++u) x_at[u] = a.X + (size_t)min(n0 + 8 * u + g, a.N - 1) * a.K + 32 * t;
  constexpr bool X_AHEAD = NT == 1;  // registers for 16 tokens' values are only there once
  struct Block {
    uint4 c[2 * RT], x[NT][4];
    uint32_t e[2 * RT];
  };
  auto load_x = [&](Block& k, int b) {
#pragma unroll
    for (int u = 0; u < NT; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) k.x[u][i] = __ldg(reinterpret_cast<const uint4*>(x_at[u] + (size_t)b * 128) + i);
  };
  auto load = [&](Block& k, int b) {
#pragma unroll
    for (int r = 0; r < 2 * RT; ++r) {
      k.c[r] = __ldg(reinterpret_cast<const uint4*>(code_at[r] + (size_t)b * 64));
      k.e[r] = __ldg(scale_at[r] + (size_t)b * 4);
    }
    if (X_AHEAD) load_x(k, b);
  };
  // The last block of a K that 128 does not divide: threads past the end (K is a multiple of 32) multiply zeros.
  auto load_end = [&](Block& k, int b) {
    if (b * 128 + 32 * t < a.K) {
      load(k, b);
      if (!X_AHEAD) load_x(k, b);
    } else {
#pragma unroll
      for (int r = 0; r < 2 * RT; ++r) {
        k.c[r] = make_uint4(0, 0, 0, 0);
        k.e[r] = 127u;
      }
#pragma unroll
      for (int u = 0; u < NT; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) k.x[u][i] = make_uint4(0, 0, 0, 0);
    }
  };
  auto multiply = [&](const Block& k, auto far) {
    uint32_t f1[2 * RT], f2[2 * RT];
#pragma unroll
    for (int r = 0; r < 2 * RT; ++r) {
      if (far.value) {
        const Mx4Scale s = mx4_scale(k.e[r]);
        f1[r] = s.f1;
        f2[r] = s.two ? s.f2 : 0x3F803F80u;
      } else {
        f1[r] = (k.e[r] + 126u) * 0x00800080u;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w[2 * RT][4];
#pragma unroll
      for (int r = 0; r < 2 * RT; ++r) {
        mx4_nibbles(i == 0 ? k.c[r].x : i == 1 ? k.c[r].y : i == 2 ? k.c[r].z : k.c[r].w, f1[r], w[r]);
        if (far.value)
#pragma unroll
          for (int j = 0; j < 4; ++j) w[r][j] = bf16x2_mul(w[r][j], f2[r]);
      }
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        // Pairs of K positions j and j + 4, as the codes' halves have them.
        const uint4 v = k.x[u][i];
        const uint32_t y[4] = {__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                               __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632)};
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int r = 0; r < RT; ++r)
            mma_16816(acc[r][u], w[2 * r][2 * h], w[2 * r + 1][2 * h], w[2 * r][2 * h + 1], w[2 * r + 1][2 * h + 1],
                      y[2 * h], y[2 * h + 1]);
      }
    }
  };
  auto use = [&](const Block& k) {
    uint32_t top = k.e[0];
#pragma unroll
    for (int r = 1; r < 2 * RT; ++r) top = max(top, k.e[r]);
    if (__any_sync(0xffffffffu, top > 128u)) multiply(k, std::true_type()); else multiply(k, std::false_type());
  };
  // The next block is on its way while one is multiplied.
  const int b_full = min(b_hi, a.K / 128);
  Block k0, k1;
  int b = b_lo + warp;
  if (b < b_full) load(k0, b);
#pragma unroll 1
  while (b < b_full) {
    if (!X_AHEAD) load_x(k0, b);
    if (b + WARPS < b_full) load(k1, b + WARPS);
    use(k0);
    b += WARPS;
    if (b >= b_full) break;
    if (!X_AHEAD) load_x(k1, b);
    if (b + WARPS < b_full) load(k0, b + WARPS);
    use(k1);
    b += WARPS;
  }
  if (b < b_hi) {
    load_end(k0, b);
    use(k0);
  }
  griddep_launch();
  constexpr int T = 8 * NT, S = mx4_few_stride(false);
  float* out = red + (size_t)warp * T * S;
  const int live = a.N - n0;
#pragma unroll
  for (int u = 0; u < NT; ++u)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int token = 8 * u + 2 * t + q;
      if (token < live)
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          out[token * S + 16 * r + g] = acc[r][u][q];
          out[token * S + 16 * r + 8 + g] = acc[r][u][2 + q];
        }
    }
  mx4_few_finish<false, T>(a, red, m0, n0, split);
}

// Adjoint: 128 features a block; a warp takes 16 rows of the weight at a time, thread (g, t) the codes of 16
// features at 16 g in rows 4 t .. 4 t + 3, and token g's four values there.
template <int NT>
__global__ void __launch_bounds__(mx4_few_warps(true) * 32, 2) mx4_few_adjoint(const Mx4FewArgs a) {
  using namespace sm100;
  extern __shared__ float red[];
  constexpr int WARPS = mx4_few_warps(true);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int split = (int)(blockIdx.x % a.splits), m0 = (int)(blockIdx.x / a.splits) * MX4_FEW_COLS;
  const int n0 = blockIdx.y * (8 * NT);
  const int nb = (a.K + 15) / 16;
  const int b_lo = (int)((long)nb * split / a.splits), b_hi = (int)((long)nb * (split + 1) / a.splits);
  float acc[8][NT][4] = {};
  griddep_wait();
  // Features (a multiple of 32) and tokens past the end repeat the last ones: what they give is never stored.
  const int mg = min(m0 + 16 * g, a.M - 16);
  const size_t pitch = (size_t)a.M / 2, spitch = (size_t)a.M / 32;
  const uint8_t* code_at = a.codes + (size_t)(4 * t) * pitch + mg / 2;
  const uint8_t* scale_at = a.scales + (size_t)(4 * t) * spitch + mg / 32;
  const __nv_bfloat16* x_at[NT];
#pragma unroll
  for (int u = 0; u < NT; ++u) x_at[u] = a.X + (size_t)min(n0 + 8 * u + g, a.N - 1) * a.K + 4 * t;
  struct Block {
    uint2 c[4], x[NT];
    uint32_t e[4];
  };
  auto load = [&](Block& k, int b) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const size_t row = (size_t)b * 16 + r;
      k.c[r] = __ldg(reinterpret_cast<const uint2*>(code_at + row * pitch));
      k.e[r] = __ldg(scale_at + row * spitch);
    }
#pragma unroll
    for (int u = 0; u < NT; ++u) k.x[u] = __ldg(reinterpret_cast<const uint2*>(x_at[u] + (size_t)b * 16));
  };
  // The last eight rows of a K that 16 does not divide: the other threads multiply zeros.
  auto load_end = [&](Block& k, int b) {
    if (b * 16 + 4 * t < a.K) {
      load(k, b);
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        k.c[r] = make_uint2(0, 0);
        k.e[r] = 127u;
      }
#pragma unroll
      for (int u = 0; u < NT; ++u) k.x[u] = make_uint2(0, 0);
    }
  };
  auto multiply = [&](const Block& k, auto far) {
    // Rows in pairs, the lower one in the low halves.
    uint32_t f1[2], f2[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (far.value) {
        const Mx4Scale lo = mx4_scale(k.e[2 * h]), hi = mx4_scale(k.e[2 * h + 1]);
        f1[h] = __byte_perm(lo.f1, hi.f1, 0x5410);
        f2[h] = __byte_perm(lo.two ? lo.f2 : 0x3F803F80u, hi.two ? hi.f2 : 0x3F803F80u, 0x5410);
      } else {
        f1[h] = (k.e[2 * h + 1] * 0x10000u + k.e[2 * h]) * 0x80u + 126u * 0x00800080u;
      }
    }
#pragma unroll
    for (int v = 0; v < 2; ++v) {  // nibbles 0..3, 4..7 of the words
      const uint32_t sel = v == 0 ? 0x5410u : 0x7632u;
      uint32_t w[2][2][4];  // [word][pair of rows][nibble]
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mx4_nibbles(__byte_perm(q ? k.c[2 * h].y : k.c[2 * h].x, q ? k.c[2 * h + 1].y : k.c[2 * h + 1].x, sel), f1[h],
                      w[q][h]);
          if (far.value)
#pragma unroll
            for (int j = 0; j < 4; ++j) w[q][h][j] = bf16x2_mul(w[q][h][j], f2[h]);
        }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int u = 0; u < NT; ++u)
          mma_16816(acc[4 * v + j][u], w[0][0][j], w[1][0][j], w[0][1][j], w[1][1][j], k.x[u].x, k.x[u].y);
    }
  };
  auto use = [&](const Block& k) {
    const bool far = max(max(k.e[0], k.e[1]), max(k.e[2], k.e[3])) > 128u;
    if (__any_sync(0xffffffffu, far)) multiply(k, std::true_type()); else multiply(k, std::false_type());
  };
  // AHEAD - 1 blocks are on their way while one is multiplied.
  constexpr int AHEAD = NT == 1 ? 4 : 2;
  const int b_full = min(b_hi, a.K / 16);
  Block ring[AHEAD];
  int b = b_lo + warp;
#pragma unroll
  for (int i = 0; i < AHEAD - 1; ++i)
    if (b + i * WARPS < b_full) load(ring[i], b + i * WARPS);
#pragma unroll 1
  while (b < b_full) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (b + (AHEAD - 1) * WARPS < b_full) load(ring[(i + AHEAD - 1) % AHEAD], b + (AHEAD - 1) * WARPS);
      if (b < b_full) {
        use(ring[i]);
        b += WARPS;
      }
    }
  }
  if (b < b_hi) {
    load_end(ring[0], b);
    use(ring[0]);
  }
  griddep_launch();
  constexpr int T = 8 * NT, S = mx4_few_stride(true);
  float* out = red + (size_t)warp * T * S;
  const int live = a.N - n0;
  // Accumulator row g of product j is feature 16 g + j, row g + 8 feature 16 g + 8 + j.
#pragma unroll
  for (int u = 0; u < NT; ++u)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int token = 8 * u + 2 * t + q;
      if (token < live)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          out[token * S + mx4_few_place<true>(16 * g + j)] = acc[j][u][q];
          out[token * S + mx4_few_place<true>(16 * g + 8 + j)] = acc[j][u][2 + q];
        }
    }
  mx4_few_finish<true, T>(a, red, m0, n0, split);
}

// -------------------------------------------------------------------------------- product, many tokens
// Y[t][m] = sum_k w(m, k) X[t][k] with w(m, k) = W[m][k] (forward: m an output, k an input feature) or W[k][m]
// (adjoint), X and Y bf16, sums in fp32.
//
// The weight is the 128-row operand (MH of them per CTA: 128 or 256 features), the tokens are the columns (TN of
// them, a multiple of 16 up to 256), so that few tokens waste nothing of the tile.  A k step is 64 positions with 256
// features and 128 with 128, 16384 weights either way: less work per step and its hand-overs take longer than its
// products.  One warp streams X tiles and one the codes of MX4_CSTEPS steps at a time (whole 64- or 128-byte
// rows: with rows of 32 bytes the copies took longer than the products) with TMA into rings; sixteen converter warps
// turn a step's codes into a bf16 tile in the 128-byte-swizzled layout of the tensor core (forward: K-major, adjoint:
// MN-major) in the slot that X's tile of the step lands in; one thread issues tcgen05.mma; the accumulators have
// features in TMEM lanes, tokens in columns.  Where the tiles alone do not fill the SMs, a cluster of 2 or 4 CTAs splits
// K and each CTA sums its share of the tokens over the cluster's shared memory, in a fixed order.
// 2048 tokens, 4096 x 4096: 49.9 us (1.38 PFLOP/s; the tensor core is busy three quarters of the time) in short
// runs, 57.8 in long ones under the power cap, where the library's product with a bf16 weight takes 47.2 and 54.2.
struct Mx4Args {
  int M, N, K;           // features out, tokens, features in
  int TN, mt;            // tokens per tile; tiles along the features
  int slots, cs;         // ring depths: tiles of X and converted weight, codes
  int splits;            // CTAs of a cluster, along K
  const uint8_t* scales;
  long pitch;            // scales per row of the weight
  __nv_bfloat16* Y;
  // Give-up probe only (poetx_test_mx4_give_up): steps whose codes the grid's first block copies; the limit of waits.
  int probe_steps;
  unsigned long long probe_ns;
};

// Two groups of eight converter warps, each with every other step, so that one converts while the other waits for
// its tiles; then a warp for X (16), for the products (17), for the codes (18).
constexpr int MX4_GROUP = 256, MX4_CONV_WARPS = 16;
constexpr int MX4_THREADS = 32 * (MX4_CONV_WARPS + 3);
constexpr int MX4_CSTEPS = 2;                    // k steps of a code tile, one per group
constexpr int MX4_MAX_RING = 8;
constexpr uint32_t MX4_W_BYTES = 32768, MX4_C_BYTES = 8192 * MX4_CSTEPS;
__host__ __device__ constexpr int mx4_bk(int mh) { return 128 / mh; }  // K positions of a step
// A code tile: bytes of its rows, and its rows.
__host__ __device__ constexpr int mx4_code_row(int mh, bool adj) { return adj ? 64 * mh : mx4_bk(mh) / 2 * MX4_CSTEPS; }
__host__ __device__ constexpr int mx4_code_rows(int mh, bool adj) { return adj ? mx4_bk(mh) * MX4_CSTEPS : 128 * mh; }
__host__ __device__ constexpr size_t mx4_smem_bytes(int mh, int tn, int slots, int cs) {
  return (size_t)slots * (tn * mx4_bk(mh) * 2 + MX4_W_BYTES) + (size_t)cs * MX4_C_BYTES + 1024 + 512;
}

// A block that gives up: every role that misses its tile leaves its loop, so that the issuing warp misses one too and
// commits no accumulators; then all warps' last wait runs out, copies land, and nothing is stored (a cluster stores
// nothing of a tile that one of its blocks gave up).  PROBE: the same kernel with short limits, whose first block
// gets no more codes after some steps, so that a test sees this happen.
template <int MH, bool ADJ, bool PROBE = false>
__global__ void __launch_bounds__(MX4_THREADS, 1)
    mx4_gemm_tc(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmC, const Mx4Args a) {
  using namespace sm100;
  constexpr uint32_t W_BYTES = MX4_W_BYTES, C_BYTES = MX4_C_BYTES;
  constexpr int CS = MX4_CSTEPS, BK = mx4_bk(MH), KA = BK / 64;  // KA: 64-wide pieces of a step
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // A slot holds a step's converted weight, then its X (64-wide pieces one after the other).
  const uint32_t xa_bytes = (uint32_t)a.TN * 128, x_bytes = xa_bytes * KA, slot_bytes = W_BYTES + x_bytes;
  const uint32_t sw = smem_u32(smem), sc = sw + (uint32_t)a.slots * slot_bytes;
  const uint32_t sb = sc + (uint32_t)a.cs * C_BYTES;
  constexpr uint32_t R = MX4_MAX_RING;
  auto ready = [&](int s) { return sb + 8u * s; };            // X has arrived and the weight is converted
  auto taken = [&](int s) { return sb + 8u * (R + s); };      // the products are done
  auto cfull = [&](int s) { return sb + 8u * (2 * R + s); };  // code tile has arrived
  auto cempty = [&](int s) { return sb + 8u * (3 * R + s); }; // code tile read
  const uint32_t accum = sb + 8u * (4 * R);
  uint32_t* holder = reinterpret_cast<uint32_t*>(smem + (sb - sw) + 8 * (4 * R + 1));
  const uint32_t gave_up = sb + 8u * (4 * R + 2);  // set by a warp that gave up, read by the cluster
  auto wait = [&](uint32_t bar, uint32_t phase, int site) {
    return PROBE ? mbar_wait_limit(bar, phase, a.probe_ns, KID_MX4, site) : mbar_wait(bar, phase, KID_MX4, site);
  };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Blocks that run together share X tiles and read the whole weight between them.
  const uint32_t tile_id = blockIdx.x / (uint32_t)a.splits;
  const int split = (int)(blockIdx.x % (uint32_t)a.splits), m0 = (int)(tile_id % (uint32_t)a.mt) * (MH * 128);
  const int n0 = (int)(tile_id / (uint32_t)a.mt) * a.TN;
  const int KT = (a.K + BK - 1) / BK;
  const int kt0 = (int)((long)KT * split / a.splits), nkt = (int)((long)KT * (split + 1) / a.splits) - kt0;
  // TMEM columns: MH accumulators of TN, a power of two from 32 up.
  uint32_t cols = 32;
  while (cols < (uint32_t)(MH * a.TN)) cols <<= 1;

  if (threadIdx.x <= 4 * R) {
    // One barrier per thread.  ready: the converting group's warps and X's copy; cempty: all converters.
    const uint32_t kind = threadIdx.x / R;
    mbar_init(sb + 8u * threadIdx.x, kind == 0 ? MX4_GROUP / 32 + 1 : kind == 3 ? MX4_CONV_WARPS : 1);
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (threadIdx.x == 4 * R + 1) st_shared_b32(gave_up, 0u);
  if (warp == MX4_CONV_WARPS + 1 && lane == 0) prefetch_tmap(&tmX);
  if (warp == MX4_CONV_WARPS + 2 && lane == 0) prefetch_tmap(&tmC);
  if (warp == MX4_CONV_WARPS) {
    tmem_alloc(smem_u32(holder), cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *holder;
  griddep_wait();  // X, and just after a quantisation the codes, come from earlier launches

  if (warp == MX4_CONV_WARPS) {
    if (lane == 0) {
      // ---------------- X producer
      int t = 0;
      uint32_t phase = 1;
      for (int i = 0; i < nkt; ++i) {
        if (!wait(taken(t), phase, 1)) break;
        mbar_arrive_expect_tx(ready(t), x_bytes);
#pragma unroll
        for (int p = 0; p < KA; ++p)
          tma_load_2d(sw + t * slot_bytes + W_BYTES + p * xa_bytes, &tmX, ready(t), (kt0 + i) * BK + 64 * p, n0);
        if (++t == a.slots) { t = 0; phase ^= 1u; }
      }
    }
  } else if (warp == MX4_CONV_WARPS + 2) {
    if (lane == 0) {
      // ---------------- code producer
      int s = 0;
      uint32_t phase = 1;
      for (int i = 0; i < nkt; i += CS) {
        if (PROBE && blockIdx.x == 0 && i >= a.probe_steps) break;
        if (!wait(cempty(s), phase, 7)) break;
        mbar_arrive_expect_tx(cfull(s), C_BYTES);
        const int k0 = (kt0 + i) * BK;
        if (!ADJ) tma_load_2d(sc + s * C_BYTES, &tmC, cfull(s), k0 / 2, m0);
        else tma_load_2d(sc + s * C_BYTES, &tmC, cfull(s), m0 / 2, k0);
        if (++s == a.cs) { s = 0; phase ^= 1u; }
      }
    }
  } else if (warp == MX4_CONV_WARPS + 1) {
    // ---------------- MMA issuer.  Its scheduler also serves converter warps, so that every instruction between two
    // products costs several cycles: the descriptors' low words are sums with constants, one barrier says that both
    // operands are there, and one commit frees both.  (With two of each, and whole descriptors built per product,
    // a step's issue took 1300 cycles, more than its 1024 of products: 52.7 us for 2048 tokens of 4096 x 4096 against
    // 50.2, 26.0 for 64 tokens of 4096 x 14336 against 21.4.  One lane walking the steps alone: 51.2 and 24.0.)
    const uint32_t idesc = idesc_bf16_f32(128, a.TN, ADJ, false);
    // A weight tile: MH = 2, 128 features (16 KiB) after the other; MH = 1, forward 64 positions after the other,
    // adjoint 64 features after the other.
    const uint64_t wd0 = ADJ ? smem_desc_sw128(sw, BK * 128, 1024) : smem_desc_sw128(sw, 16, 1024);
    const uint64_t xd0 = smem_desc_sw128(sw + W_BYTES, 16, 1024);
    const uint32_t w_hi = (uint32_t)(wd0 >> 32), x_hi = (uint32_t)(xd0 >> 32);
    uint32_t w_lo = (uint32_t)wd0, x_lo = (uint32_t)xd0;  // addresses in units of 16 bytes: they never carry
    // The whole warp walks the steps, so that descriptors stay uniform, and one lane issues.
    const bool leader = elect_one();
    int t = 0, i = 0;
    uint32_t phase = 0;
    for (; i < nkt; ++i) {
      if (!__all_sync(0xffffffffu, wait(ready(t), phase, 2))) break;
      tc_fence_after();
      const uint32_t bar = taken(t), w = w_lo, x = x_lo;
      w_lo += slot_bytes >> 4;
      x_lo += slot_bytes >> 4;
      if (++t == a.slots) {
        t = 0;
        phase ^= 1u;
        w_lo = (uint32_t)wd0;
        x_lo = (uint32_t)xd0;
      }
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk) {
          const uint32_t xl = x + (kk >= 4 ? xa_bytes >> 4 : 0u) + (kk & 3) * 2;
#pragma unroll
          for (int h = 0; h < MH; ++h) {
            const uint32_t wl = w + (ADJ ? h * 1024 + kk * 128 : (h + (kk >> 2)) * 1024 + (kk & 3) * 2);
            mma_bf16_words(tmem + (uint32_t)(h * a.TN), wl, w_hi, xl, x_hi, idesc, kk > 0 || i > 0);
          }
        }
        mma_commit(bar);
      }
      __syncwarp();
    }
    if (leader && i == nkt) mma_commit(accum);
  } else {
    // ---------------- converters: two blocks of 32 codes (64 columns) of one row per thread and step
    // Forward: rows are features, columns K positions.  Adjoint: rows are K positions, columns features.
    const int ct = threadIdx.x % MX4_GROUP, group = threadIdx.x / MX4_GROUP;
    constexpr int ROWS = ADJ ? BK : 128 * MH;
    const int row = ct & (ROWS - 1), piece = ct / ROWS;  // row of a step's codes, 64 columns of it
    const int key = row & 7;                             // 128-byte swizzle of the bf16 tile
    const uint32_t dst = (uint32_t)(piece * ROWS * 128 + row * 128 + (key << 4));
    // Code tile: its 16-byte pieces are swizzled over 128 or 64 bytes; this group's step of it.
    constexpr int CROW = mx4_code_row(MH, ADJ);
    static_assert(CROW == 128 || CROW == 64, "swizzle widths");
    const uint32_t ckey = CROW == 128 ? (uint32_t)(row & 7) : (uint32_t)((row >> 1) & 3);
    const uint32_t cpiece = (uint32_t)((ADJ ? 0 : 2 * KA * group) + 2 * piece);
    const uint32_t c0 = (uint32_t)((row + (ADJ ? group * BK : 0)) * CROW) + ((cpiece ^ ckey) << 4);
    const uint32_t c1 = (uint32_t)((row + (ADJ ? group * BK : 0)) * CROW) + (((cpiece + 1) ^ ckey) << 4);
    // The two scales of a step, loaded two steps ahead (eight cost a longer loop body: 2 % more time).  Rows and
    // features past the end repeat the last (what they give is never stored); past the end of K, where codes and
    // tokens are zeros, any finite scale does.
    const int nblock = (int)a.pitch;
    const bool even = a.pitch % 2 == 0;
    const uint8_t* scale_at;
    long scale_step;            // from one step of this group to the next
    int scales_left, two_left;  // steps of this group whose first, whose second scale lies before the end
    if (!ADJ) {
      const int c = (kt0 + group) * (BK / 32) + 2 * piece, step = CS * (BK / 32);
      scale_at = a.scales + (long)min(m0 + row, a.M - 1) * a.pitch + c;
      scale_step = step;
      scales_left = (nblock - c + step - 1) / step;
      two_left = (nblock - c - 1 + step - 1) / step;
    } else {
      const int k = (kt0 + group) * BK + row;
      const int base = even ? min(m0 / 32 + 2 * piece, nblock - 2) : min(m0 / 32 + 2 * piece, nblock - 1);
      scale_at = a.scales + (long)k * a.pitch + base;
      scale_step = (long)CS * BK * a.pitch;
      scales_left = (a.K - k + CS * BK - 1) / (CS * BK);
      two_left = base + 1 < nblock ? scales_left : 0;
    }
    scales_left = min(scales_left, (nkt - group + CS - 1) / CS);
    // Joined only when they are used (joining at the load waits for it: 1 us before the first step with odd pitches).
    struct Pair {
      uint32_t lo, hi;
    };
    auto load_scales = [&]() -> Pair {
      Pair e = {127u, 127u};
      if (scales_left > 0) {
        if (even) {
          e.lo = __ldg(reinterpret_cast<const uint16_t*>(scale_at));
          e.hi = 0u;
        } else {
          e.lo = __ldg(scale_at);
          if (two_left > 0) e.hi = __ldg(scale_at + 1);
        }
      }
      scale_at += scale_step;
      --scales_left;
      --two_left;
      return e;
    };
    Pair next = load_scales();
    int s = 0, t = group;  // at least two slots
    uint32_t s_phase = 0, t_phase = 1;
    for (int i = group; i < nkt; i += CS) {
      const uint32_t scales = next.lo | next.hi << 8;
      next = load_scales();
      bool ok = wait(cfull(s), s_phase, 4);
      const uint4 c[2] = {ld_shared_v4(sc + s * C_BYTES + c0), ld_shared_v4(sc + s * C_BYTES + c1)};
      ok = ok && wait(taken(t), t_phase, 5);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint32_t tile = sw + t * slot_bytes + dst;  // piece j of the row: position j ^ key of its 128 bytes
      if (__any_sync(0xffffffffu, max(scales & 0xFFu, scales >> 8) > 128u)) {
        // Scales above 2, which take a second product, are rare: a branch of the whole warp, kept small.
#pragma unroll 1
        for (int u = 0; u < 2; ++u) {
          const Mx4Scale f = mx4_scale((scales >> (8 * u)) & 0xFFu);
          const uint4 v = u ? c[1] : c[0];
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) st_shared_v4(tile ^ ((4 * u + j) << 4), mx4_decode8<!ADJ>(w[j], f));
        }
      } else {
        const uint32_t w[8] = {c[0].x, c[0].y, c[0].z, c[0].w, c[1].x, c[1].y, c[1].z, c[1].w};
        const uint32_t f1[2] = {(scales & 0xFFu) * 0x00800080u + 126u * 0x00800080u,
                                (scales >> 8) * 0x00800080u + 126u * 0x00800080u};
#pragma unroll
        for (int j = 0; j < 8; ++j) st_shared_v4(tile ^ (j << 4), mx4_decode8<!ADJ>(w[j], f1[j >> 2]));
      }
      fence_proxy_async_smem();  // the tensor core reads what the threads wrote
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(ready(t));
        // Every lane has used its codes, fenced its reads of them against the asynchronous copy that refills the
        // tile, and met the others: only then is it given back.  Given back right after the loads, without the fence,
        // refills were seen to overtake them (which of the two was missing was not taken apart: both hold here).
        mbar_arrive(cempty(s));
      }
      if (++s == a.cs) { s = 0; s_phase ^= 1u; }
      t += CS;
      if (t >= a.slots) { t -= a.slots; t_phase ^= 1u; }
    }
  }
  __syncwarp();

  // ---------------- epilogue
  bool ok = wait(accum, 0, 6);
  ok = __all_sync(0xffffffffu, ok);
  if (!ok) {
    st_shared_b32(gave_up, 1u);
    // Copies still under way land within microseconds; they must find this block's memory.
    for (const unsigned long long t0 = global_timer_ns(); global_timer_ns() - t0 < 1000000ull;) {
    }
  }
  tc_fence_after();
  griddep_launch();
  // The adjoint's features stand in mx4_decode8's order within each eight: this lane's.
  const int feature = ADJ ? (lane & 24) | ((lane >> 1) & 3) | ((lane & 1) << 2) : lane;
  if (a.splits == 1) {
    // Warp w drains lanes 32 (w % 4).. of the accumulators, tokens 32 (w / 4).. of every 128: 32 at a time, turned
    // over in shared memory (the rings are idle: every load has been consumed) so that stores are 16 bytes.
    if (warp < MX4_CONV_WARPS && ok) {
      const int lq = (warp & 3) * 32;
      const uint32_t patch = sw + warp * 2048;  // bf16 [32 tokens][32 features]
#pragma unroll 1
      for (int h = 0; h < MH; ++h) {
        const uint32_t t0 = tmem + ((uint32_t)lq << 16) + (uint32_t)(h * a.TN);
        const int m = m0 + h * 128 + lq + (lane & 3) * 8;
#pragma unroll 1
        for (int c = (warp >> 2) * 32; c < a.TN; c += 128) {
          uint32_t v[4][8];
#pragma unroll
          for (int g = 0; g < 4; ++g)
            if (c + 8 * g < a.TN) tmem_ld_32x32b_x8(t0 + (uint32_t)(c + 8 * g), v[g]);
          tmem_wait_ld();
#pragma unroll
          for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int j = 0; j < 8; ++j)
              st_shared_b16(patch + ((8 * g + j) * 32 + feature) * 2, __float2bfloat16_rn(__uint_as_float(v[g][j])));
          __syncwarp();
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int n = n0 + c + 8 * g + (lane >> 2);
            if (c + 8 * g < a.TN && n < a.N && m < a.M)
              *reinterpret_cast<uint4*>(a.Y + (size_t)n * a.M + m) =
                  ld_shared_v4(patch + (8 * g + (lane >> 2)) * 64 + (lane & 3) * 16);
          }
          __syncwarp();
        }
      }
    }
  } else {
    // One 128-feature half after the other, fp32 sums [TN][128] through shared memory, at the start of the rings.
    const int share = a.TN / a.splits, c_lo = split * share;
#pragma unroll 1
    for (int h = 0; h < MH; ++h) {
      if (warp < MX4_CONV_WARPS && ok) {
        const uint32_t t0 = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)(h * a.TN);
        const uint32_t out = sw + ((warp & 3) * 32 + feature) * 4;
        for (int c = (warp >> 2) * 8; c < a.TN; c += 32) {
          uint32_t v[8];
          tmem_ld_32x32b_x8(t0 + (uint32_t)c, v);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 8; ++j) st_shared_b32(out + (uint32_t)(c + j) * 512, v[j]);
        }
      }
      cluster_sync_all();
      if (ok) {
        uint32_t lost = 0u;
        for (int r = 0; r < a.splits; ++r) lost |= ld_cluster_u32(mapa_shared(gave_up, (uint32_t)r));
        // Eight features of one token per step: sum over the cluster, round once, 16-byte store.
        for (int e = threadIdx.x; e < share * 16; e += MX4_THREADS) {
          const int c = c_lo + (e >> 4), f = (e & 15) * 8;
          const int n = n0 + c, m = m0 + h * 128 + f;
          if (n < a.N && m < a.M) {
            float x[8] = {};
            const uint32_t at = sw + (uint32_t)(c * 128 + f) * 4;
            for (int r = 0; r < a.splits; ++r) {
              float y[8];
              ld_cluster_v4(mapa_shared(at, (uint32_t)r), y);
              ld_cluster_v4(mapa_shared(at, (uint32_t)r) + 16, y + 4);
#pragma unroll
              for (int j = 0; j < 8; ++j) x[j] += y[j];
            }
            if (lost) continue;
            *reinterpret_cast<uint4*>(a.Y + (size_t)n * a.M + m) =
                make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
          }
        }
      }
      cluster_sync_all();  // the peers have read this CTA's sums before it reuses them or exits
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == MX4_CONV_WARPS) tmem_dealloc(tmem, cols);
}

}  // namespace poetx
