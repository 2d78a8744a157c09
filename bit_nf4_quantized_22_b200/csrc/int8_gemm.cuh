// int8_gemm.cuh -- host interface of the integer products (int8_gemm.cu).
#pragma once
#include "common.cuh"

namespace qlora {

// out(p, q) = (sum_d 256^(planes-1-d) sum_t A(p, t) B_d(q, t)) * qscale[q] * mul * pscale[p] + bias[p]
struct Int8Product {
    const int8_t *a;       // a_mn: A(p, t) at a[t * lda + p], else a[p * lda + t]
    int64_t lda;           // bytes, a multiple of 16
    int a_mn;
    const int8_t *b;       // B_d(q, t) at b[(d * plane_rows + q) * ldb + t]
    int64_t ldb;           // bytes, a multiple of 16
    int64_t plane_rows;
    int planes;            // 1, 2 or 3
    const uint8_t *deep;   // planes == 2, or NULL: rows q with a 1 here have four planes of digits
    int64_t P, Q, R;       // extents of p, q and the reduction t (R <= 131072)
    const float *qscale;
    const float *pscale;   // or NULL
    float mul;
    const void *bias;      // per p, in the output's dtype, or NULL
    void *out;             // q_inner: out[p * ldo + q] (fp32), else out[q * ldo + p]
    int64_t ldo;
    int q_inner;
    int pool;              // q_inner: 64 sums the rows p of each run of 64 (out has P / 64 rows), else 1 or 0
    int dtype;             // QLORA_DTYPE_*
    int pdl;               // launch beside the kernel before, which writes B and the scales but not A
};

int launch_int8_product(const Int8Product &g, uint32_t *d_status, cudaStream_t st);

// int8_gemv.cu: M <= 4 tokens whose codes fit in a CTA's share of shared memory
constexpr int64_t kGemvTokenBytes = 48 * 1024;
bool int8_gemv_takes(int64_t M, int64_t N, int64_t K);
int launch_int8_gemv(const void *X, int x_dtype, int64_t ldx, const int8_rows_t &X8, const int8_rows_t &W,
                     const void *bias, void *Y, int dtype, uint32_t *d_status, cudaStream_t st);

// An int32 sum of up to 131072 products of two codes.  They lie in (-2^31, 2^31]:
// 2^31 itself, of codes that are all -128, wraps to -2^31, which no sum is.  Negated
// both before and after the conversion it comes out right, and every other sum the same.
__device__ __forceinline__ float sum_float(uint32_t v) { return -(float)(int)(0u - v); }
__device__ __forceinline__ int64_t sum_int64(uint32_t v) { return -(int64_t)(int)(0u - v); }

__device__ __forceinline__ float load_any(const void *p, int64_t i, int dtype) {
    if (dtype == QLORA_DTYPE_FP32) return __ldg(static_cast<const float *>(p) + i);
    return dec16(__ldg(static_cast<const uint16_t *>(p) + i), dtype == QLORA_DTYPE_FP16);
}

// int8_rows.cu
int launch_int8_quantize(const void *X, int dtype, int64_t ldx, const int8_rows_t &q, uint32_t *d_status,
                         cudaStream_t st);
int launch_int8_row_digits(const uint16_t *Y, bool f16, int64_t rows, int64_t cols, const float *cscale,
                           int8_t *planes, int64_t ld, float *steps, uint8_t *deep, cudaStream_t st);
int launch_int8_col_digits(const void *S, int dtype, int64_t R, int r, const float *f, int8_t *planes, int64_t ld,
                           int rp, int rep, float *steps, cudaStream_t st);
int launch_int8_dequantize(const int8_rows_t &q, int dtype, void *out, cudaStream_t st);

}  // namespace qlora
