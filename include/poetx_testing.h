/*
 * poetx_testing.h — test hook of libpoetx: direct access to the batched GEMM core that every
 * contraction of the POET-X layer runs on (the block-diagonal products, the W0' products, the
 * per-block gradients, the Cayley–Neumann powers and the merge; replication review of POET-X,
 * "Summary": batch-parallel block-diagonal matmul).  Used by the tests to check each operand
 * layout and tile width against a plain fp32 matmul.  Not needed by users of the layer.
 *
 *   D[z][m][n] (+ split s) = alpha * sum_{k in split s} A[z][m][k] * B[z][n][k] + beta * C[z][m][n]
 *                            (+ 1 where m == n if diag)
 *   A (a_mn == 0): A[z][m][k] = a[(z*a_zrow + m) * a_ld + z*a_zcol + k]
 *     (a_mn == 1): A[z][m][k] = a[(z*a_zrow + k) * a_ld + z*a_zcol + m]      (B likewise with n)
 *   D[z][m][n] at d[(z*d_zrow + m) * d_ld + z*d_zcol + n + s*d_split_stride]; C like D (no split).
 * dtype selects the operand type (POETX_BF16: tcgen05 tensor cores; POETX_F32: fp32 CUDA cores);
 * d_dtype the output type; C is float32 or NULL.  All pointers are device pointers; the call
 * is asynchronous on `stream`.  a_rows/a_cols (b_rows/b_cols) are the extents of the whole
 * operand arrays; the call is rejected (POETX_ERR_INVALID_ARG) if any addressed element lies
 * outside them.
 */
#ifndef POETX_TESTING_H_
#define POETX_TESTING_H_

#include "poetx.h"

#ifdef __cplusplus
extern "C" {
#endif

poetx_status poetx_test_gemm(int dtype, int M, int N, int K, int batch, int splits,
                             const void* a, long long a_rows, long long a_cols, long long a_ld,
                             long long a_zrow, long long a_zcol, int a_mn,
                             const void* b, long long b_rows, long long b_cols, long long b_ld,
                             long long b_zrow, long long b_zcol, int b_mn,
                             void* d, int d_dtype, long long d_ld, long long d_zrow, long long d_zcol,
                             long long d_split_stride, float alpha, float beta, const float* c,
                             long long c_ld, long long c_zrow, long long c_zcol, int diag,
                             poetx_stream stream);

/* Failure-detection probe (the bounded device-side waits of every kernel; no GPU fault is
 * involved).  Launches one CTA that waits on a shared-memory mbarrier nothing arrives on, with the
 * wait bounded by limit_ns nanoseconds of the device's global timer (1 us .. 100 ms).  The wait
 * runs out, the kernel records a device timeout (poetx_device_status() then returns
 * POETX_ERR_DEVICE_TIMEOUT with detail (7 << 8) | 1) and writes 2 to *returned (a device int;
 * 1 would mean that the wait completed).  Errors: INVALID_ARG (NULL, limit out of range),
 * ALIGNMENT, CUDA. */
poetx_status poetx_test_wait_timeout(long long limit_ns, int* returned, poetx_stream stream);

/* Failure-detection probe of the tcgen05 products D = A . B^T (A [M, K], B [N, K], D [M, N], row-major bf16; N a multiple
 * of 256, K of 64): the kernel of `kind` with its waits bounded by limit_ns (1 ms .. 100 ms), whose first block loads only
 * its first `steps` tiles of K.
 *   kind 0: the generic kernel, 128 x 64 tiles         kind 1: with the block factor, 128 x 256 tiles
 *   kind 2: 256 x 256 tiles, with the block factor if out2 is not NULL       kind 3: as 2, B int8 codes with b_scale [N]
 * The block factor is out2 = D . Q^T per block of 256 columns (Q [N, 256] bf16: one 256 x 256 matrix per block); with
 * steps = K / 64 the first block misses Q.  Its waits run out: it records a device timeout (detail (1 << 8) | site) and
 * returns with what it has not computed as it was.  Errors: INVALID_ARG (a size, the limit, nothing to miss), ALIGNMENT,
 * CUDA. */
poetx_status poetx_test_gemm_give_up(int kind, int M, int N, int K, const void* a, const void* b, const float* b_scale,
                                     const void* q, void* d, void* out2, int steps, long long limit_ns,
                                     poetx_stream stream);

/* Failure-detection probe of the many-token MX4 product: poetx_mx4_matmul's tensor-core kernel with its waits bounded
 * by limit_ns (1 ms .. 100 ms), whose first block copies only the first `steps` steps of its codes (rounded up to
 * pairs).  That block's waits run out: it records a device timeout (detail (9 << 8) | site) and returns
 * with its tile of Y as it was, and so do the blocks of its cluster; every other tile is computed as ever.  *splits (a HOST int)
 * receives the number of blocks of a cluster.  Errors as poetx_mx4_matmul, and INVALID_ARG (n_tokens <= 0, the limit out of
 * range, as many steps as the block has). */
poetx_status poetx_test_mx4_give_up(int adjoint, int n_tokens, int d_in, int d_out, const void* X, const uint8_t* codes,
                                    const uint8_t* scales, void* Y, int steps, long long limit_ns, int* splits,
                                    poetx_stream stream);

/* Compares the square root of the 8-bit moments with CUDA's correctly rounded one for the float32 numbers with the
 * bit patterns first..last, all from 2^-100 (0x0D800000) up to the largest finite one (0x7F7FFFFF);
 * *mismatches (device memory, 8-byte aligned) receives how many differ. */
poetx_status poetx_test_sqrt(unsigned first, unsigned last, unsigned long long* mismatches, poetx_stream stream);

#ifdef __cplusplus
}
#endif
#endif /* POETX_TESTING_H_ */
