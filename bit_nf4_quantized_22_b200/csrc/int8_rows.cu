// int8_rows.cu -- the 8-bit row codec and the integer digits of the products
// that int8_gemm.cu computes.
//
// A row of codes (bitsandbytes article (CSDN) 4.1, absmax INT8, here with one
// scale for each token or output channel):
//   a = max |x|,  s = RN32(a / 127),  c = RNE(x / s), |c| <= 127
// with the exact quotient; a row of zeros (or s = 0) has codes 0, a row with a
// NaN or an infinity has s = NaN and codes 0.
//
// Where an operand is not 8-bit data already, it is written in fixed point and
// cut into signed base-256 digits, each an int8 plane of its own:
//   q = 256 d1 + d0  (16 bits, |q| <= 32639)      rows of dY * channel scale
//   q = 65536 d2 + 256 d1 + d0 (|q| <= 8355711)   columns of A, of scale * G
// so that the integer tensor cores give the product of the full operand, as
// the digits' products added with their weights.
#include <cooperative_groups.h>

#include "common.cuh"

namespace qlora {
namespace {

constexpr int kVec = 8;           // values per thread and step
// steps whose values stay in registers between the maximum and the codes
template <int DT> constexpr int kKeep = DT == QLORA_DTYPE_FP32 ? 2 : 4;
constexpr int kMaxRowThreads = 1024;
constexpr float kMagic = 12582912.f;   // 1.5 * 2^23: adding it rounds to an integer, ties to even

// Eight consecutive values of a row as they were loaded.
template <int DT>
struct Raw8 {
    uint32_t w[DT == QLORA_DTYPE_FP32 ? 8 : 4];
};

// Values [8 v, 8 v + 8) of a row, zeros past its end.  `aligned`: the row
// starts on a 16-byte border.
template <int DT>
__device__ __forceinline__ Raw8<DT> load8(const void *row, int64_t v, int64_t cols, bool aligned) {
    Raw8<DT> r;
    constexpr int kWords = sizeof(r.w) / 4;
    const int64_t e0 = v * kVec;
    if (aligned && e0 + kVec <= cols) {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const char *>(row) + e0 * (kWords / 2));
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) {
            const uint4 t = __ldg(p + i);
            r.w[4 * i] = t.x, r.w[4 * i + 1] = t.y, r.w[4 * i + 2] = t.z, r.w[4 * i + 3] = t.w;
        }
        return r;
    }
#pragma unroll
    for (int i = 0; i < kWords; ++i) r.w[i] = 0;
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
        if (e0 + e >= cols) break;
        if (DT == QLORA_DTYPE_FP32)
            r.w[e % kWords] = __ldg(static_cast<const uint32_t *>(row) + e0 + e);
        else
            r.w[e / 2] |= (uint32_t)__ldg(static_cast<const uint16_t *>(row) + e0 + e) << (16 * (e & 1));
    }
    return r;
}

template <int DT>
__device__ __forceinline__ float val8(const Raw8<DT> &r, int e) {
    if (DT == QLORA_DTYPE_FP32) return __uint_as_float(r.w[e % (sizeof(r.w) / 4)]);
    const uint32_t w = r.w[e / 2];
    return (e & 1) ? hi16(w, DT == QLORA_DTYPE_FP16) : lo16(w, DT == QLORA_DTYPE_FP16);
}

// Largest magnitude as fp32 bits: bit patterns of magnitudes order as the
// magnitudes do, infinities and NaNs above every finite value.
template <int DT>
__device__ __forceinline__ uint32_t absmax8(const Raw8<DT> &r, uint32_t m) {
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
        const uint32_t b = __float_as_uint(fabsf(val8(r, e)));
        m = b > m ? b : m;
    }
    return m;
}

__device__ __forceinline__ uint32_t block_max(uint32_t m) {
    __shared__ uint32_t part[32];
    m = __reduce_max_sync(0xffffffffu, m);
    const int warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    if (nw == 1) return m;
    if ((threadIdx.x & 31) == 0) part[warp] = m;
    __syncthreads();
    const uint32_t v = (threadIdx.x & 31) < nw ? part[threadIdx.x & 31] : 0u;
    return __reduce_max_sync(0xffffffffu, v);
}

// Code of x exactly: the quotient in fp64 is never within 2^-33 (relative) of
// a border between two codes without lying on it, since x and s have 24 bits.
__device__ __noinline__ int code_exact(float x, float s) {
    const double q = (double)x / (double)s;
    const int c = __double2int_rn(q > 127.0 ? 127.0 : (q < -127.0 ? -127.0 : q));
    return c;
}

// Store 8 code bytes at element e0 of a row (16-byte aligned start).
__device__ __forceinline__ void store8(int8_t *row, int64_t e0, int64_t cols, uint32_t lo, uint32_t hi) {
    if (e0 + kVec <= cols) {
        *reinterpret_cast<uint2 *>(row + e0) = make_uint2(lo, hi);
        return;
    }
    for (int e = 0; e < kVec && e0 + e < cols; ++e)
        row[e0 + e] = (int8_t)(uint8_t)((e < 4 ? lo >> (8 * e) : hi >> (8 * (e - 4))) & 255u);
}

__device__ __forceinline__ uint32_t bytes4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// Eight codes.  fma(x, 1/s, magic) rounds x * (1/s) to the nearest integer in
// its low bits; the rounded reciprocal puts the quotient at most 127 * 2^-23
// off, so a code is decided unless the quotient lies within 1e-4 of a border,
// where code_exact decides.
template <int DT>
__device__ __forceinline__ uint2 encode8(const Raw8<DT> &r, float s, float inv, bool tiny) {
    uint32_t c[kVec];
    float far = 0.f;
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
        const float x = val8(r, e);
        const float t = __fmaf_rn(x, inv, kMagic);
        c[e] = __float_as_uint(t);
        far = fmaxf(far, fabsf(__fmaf_rn(x, inv, -(t - kMagic))));
    }
    if (tiny || far > 0.4999f) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) c[e] = (uint32_t)code_exact(val8(r, e), s);
    }
    return make_uint2(bytes4(c[0], c[1], c[2], c[3]), bytes4(c[4], c[5], c[6], c[7]));
}

// One CTA per row (grid-stride); see launch_int8_quantize for its threads.
template <int DT>
__global__ void __launch_bounds__(kMaxRowThreads)
k_int8_quantize(const void *X, int64_t ldx, int64_t rows, int64_t cols, int8_t *codes, int64_t ld,
                float *scales, bool aligned, uint32_t *status) {
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    constexpr int esize = DT == QLORA_DTYPE_FP32 ? 4 : 2;
    const int64_t nv = (cols + kVec - 1) / kVec;
    for (int64_t m = blockIdx.x; m < rows; m += gridDim.x) {
        const char *row = static_cast<const char *>(X) + m * ldx * esize;
        constexpr int kKeepSteps = kKeep<DT>;
        Raw8<DT> keep[kKeepSteps];
        uint32_t am = 0;
#pragma unroll
        for (int i = 0; i < kKeepSteps; ++i) {
            const int64_t v = (int64_t)i * blockDim.x + threadIdx.x;
            if (v < nv) keep[i] = load8<DT>(row, v, cols, aligned);
        }
#pragma unroll
        for (int i = 0; i < kKeepSteps; ++i)
            if ((int64_t)i * blockDim.x + threadIdx.x < nv) am = absmax8<DT>(keep[i], am);
        for (int64_t v = (int64_t)kKeepSteps * blockDim.x + threadIdx.x; v < nv; v += blockDim.x)
            am = absmax8<DT>(load8<DT>(row, v, cols, aligned), am);
        am = block_max(am);
        const bool fin = am < 0x7f800000u;
        const float s = fin ? __fdiv_rn(__uint_as_float(am), 127.f) : __uint_as_float(0x7fffffffu);
        if (threadIdx.x == 0) {
            scales[m] = s;
            if (!fin && status) atomicOr(status, QLORA_STATUS_NONFINITE);
        }
        int8_t *dst = codes + m * ld;
        const bool zero = !fin || s == 0.f;
        const bool tiny = s < 0x1p-120f;       // 1/s may overflow: every code by code_exact
        const float inv = zero || tiny ? 0.f : __frcp_rn(s);
#pragma unroll
        for (int i = 0; i < kKeepSteps; ++i) {
            const int64_t v = (int64_t)i * blockDim.x + threadIdx.x;
            if (v < nv) {
                const uint2 c = zero ? make_uint2(0u, 0u) : encode8<DT>(keep[i], s, inv, tiny);
                store8(dst, v * kVec, cols, c.x, c.y);
            }
        }
        for (int64_t v = (int64_t)kKeepSteps * blockDim.x + threadIdx.x; v < nv; v += blockDim.x) {
            const uint2 c = zero ? make_uint2(0u, 0u)
                                 : encode8<DT>(load8<DT>(row, v, cols, aligned), s, inv, tiny);
            store8(dst, v * kVec, cols, c.x, c.y);
        }
        if (blockDim.x > 32) __syncthreads();   // block_max's shared words are free again
    }
}

// Rows of D = dY * scale[column] (RN32) in 16-bit fixed point, q = RN(D / step),
// step = a / 32639, as two digit planes.  A rounding is off by half a step,
// a / 65278, so a row by at most sqrt(cols) / 65278 of its norm whatever its
// values (about 4e-5 for normal ones): below the 16-bit output's own rounding.
template <int DT>
__global__ void __launch_bounds__(kMaxRowThreads)
k_int8_row_digits(const void *Y, int64_t rows, int64_t cols, const float *__restrict__ cscale,
                  int8_t *planes, int64_t ld, float *steps, bool aligned) {
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const int64_t nv = (cols + kVec - 1) / kVec;
    for (int64_t m = blockIdx.x; m < rows; m += gridDim.x) {
        const char *row = static_cast<const char *>(Y) + m * cols * 2;
        auto product = [&](const Raw8<DT> &r, int64_t v, float (&d)[kVec]) {
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                d[e] = v * kVec + e < cols ? __fmul_rn(val8(r, e), __ldg(cscale + v * kVec + e)) : 0.f;
        };
        uint32_t am = 0;
        for (int64_t v = threadIdx.x; v < nv; v += blockDim.x) {
            float d[kVec];
            product(load8<DT>(row, v, cols, aligned), v, d);
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const uint32_t b = __float_as_uint(fabsf(d[e]));
                am = b > am ? b : am;
            }
        }
        am = block_max(am);
        const bool fin = am < 0x7f800000u;
        // magnitudes below 2^-60 are raised by 2^64 first, so that 1/step stays finite
        const float up = am < 0x21800000u ? 0x1p64f : 1.f;
        const float a = __uint_as_float(am) * up;
        const float inv = fin && a > 0.f ? __fdiv_rn(32639.f, a) : 0.f;
        if (threadIdx.x == 0)
            steps[m] = fin ? __fdiv_rn(a, 32639.f) / up : __uint_as_float(0x7fffffffu);
        int8_t *hi = planes + m * ld, *lo = planes + (rows + m) * ld;
        for (int64_t v = threadIdx.x; v < nv; v += blockDim.x) {
            float d[kVec];
            product(load8<DT>(row, v, cols, aligned), v, d);
            uint32_t q[kVec], h[kVec];
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const float t = fin ? fminf(fmaxf(d[e] * up * inv, -32639.f), 32639.f) : 0.f;
                q[e] = (uint32_t)__float2int_rn(t);
                h[e] = (uint32_t)(((int)q[e] - (int)(int8_t)(uint8_t)q[e]) >> 8);
            }
            store8(hi, v * kVec, cols, bytes4(h[0], h[1], h[2], h[3]), bytes4(h[4], h[5], h[6], h[7]));
            store8(lo, v * kVec, cols, bytes4(q[0], q[1], q[2], q[3]), bytes4(q[4], q[5], q[6], q[7]));
        }
        if (blockDim.x > 32) __syncthreads();
    }
}

// Columns of S[t][j] (rows t < R, columns j < r; 16-bit or fp32), optionally
// times f[t], in 24-bit fixed point with one step per column, as three digit
// planes transposed to planes[d][j][t] (rows of ld bytes, rp rows a plane).
// A step is max / 8355711: half of it is 6e-8 of the column's largest value.
// A cluster of 8 CTAs shares 16 columns: each finds the maxima of its rows,
// the cluster joins them over distributed shared memory.
constexpr int kColStrip = 16, kColTile = 128, kColCluster = 8, kColThreads = 256;
constexpr float kColMax = 8355711.f;   // 127 * (65536 + 256 + 1)

template <int DT>
__global__ void __cluster_dims__(1, kColCluster, 1) __launch_bounds__(kColThreads)
k_int8_col_digits(const void *S, int64_t R, int r, const float *__restrict__ f, int64_t per,
                  int8_t *planes, int64_t ld, int rp, float *steps) {
    namespace cg = cooperative_groups;
    __shared__ uint32_t cmax[kColStrip];
    __shared__ float stile[kColStrip][kColTile + 1];
    __shared__ float sinv[kColStrip], sup[kColStrip];
    cg::cluster_group cl = cg::this_cluster();
    const int j0 = blockIdx.x * kColStrip;
    const int64_t t0 = (int64_t)blockIdx.y * per;
    const int64_t t1 = t0 + per < R ? t0 + per : R;
    const int tid = threadIdx.x;
    auto value = [&](int64_t t, int j) -> float {
        if (t >= t1 || j >= r) return 0.f;
        const float v = DT == QLORA_DTYPE_FP32 ? __ldg(static_cast<const float *>(S) + t * r + j)
                                               : dec16(__ldg(static_cast<const uint16_t *>(S) + t * r + j),
                                                       DT == QLORA_DTYPE_FP16);
        return f ? __fmul_rn(v, __ldg(f + t)) : v;
    };
    if (tid < kColStrip) cmax[tid] = 0;
    __syncthreads();
    {
        const int j = tid % kColStrip;
        uint32_t m = 0;
        for (int64_t t = t0 + tid / kColStrip; t < t1; t += kColThreads / kColStrip) {
            const uint32_t b = __float_as_uint(fabsf(value(t, j0 + j)));
            m = b > m ? b : m;
        }
        const uint32_t o = __shfl_xor_sync(0xffffffffu, m, 16);
        m = o > m ? o : m;
        if ((tid & 16) == 0) atomicMax(&cmax[j], m);
    }
    cl.sync();
    if (tid < kColStrip) {
        uint32_t m = 0;
        for (int c = 0; c < kColCluster; ++c) {
            const uint32_t o = *cl.map_shared_rank(&cmax[tid], c);
            m = o > m ? o : m;
        }
        const bool fin = m < 0x7f800000u;
        const float up = m < 0x21800000u ? 0x1p64f : 1.f;
        const float a = __uint_as_float(m) * up;
        sup[tid] = up;
        sinv[tid] = fin && a > 0.f ? __fdiv_rn(kColMax, a) : 0.f;
        if (blockIdx.y == 0 && j0 + tid < rp)
            steps[j0 + tid] = fin ? __fdiv_rn(a, kColMax) / up : __uint_as_float(0x7fffffffu);
    }
    cl.sync();   // the maxima have been read before any CTA leaves
    for (int64_t tb = t0; tb < t1; tb += kColTile) {
        for (int i = tid; i < kColTile * kColStrip; i += kColThreads)
            stile[i % kColStrip][i / kColStrip] = value(tb + i / kColStrip, j0 + i % kColStrip);
        __syncthreads();
        const int j = tid / 16, tg = (tid % 16) * 8;   // 8 rows t of column j
        if (tb + tg < t1 && j0 + j < rp) {
            const float inv = sinv[j], up = sup[j];
            uint32_t d[3][2] = {};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float x = inv > 0.f ? fminf(fmaxf(stile[j][tg + e] * up * inv, -kColMax), kColMax) : 0.f;
                const int q = __float2int_rn(x);
                const int b0 = (int)(int8_t)(uint8_t)q;
                const int q1 = (q - b0) >> 8;
                const int b1 = (int)(int8_t)(uint8_t)q1;
                const int b2 = (q1 - b1) >> 8;
                d[0][e / 4] |= (uint32_t)(uint8_t)b2 << (8 * (e & 3));
                d[1][e / 4] |= (uint32_t)(uint8_t)b1 << (8 * (e & 3));
                d[2][e / 4] |= (uint32_t)(uint8_t)b0 << (8 * (e & 3));
            }
#pragma unroll
            for (int p = 0; p < 3; ++p)
                *reinterpret_cast<uint2 *>(planes + ((int64_t)p * rp + j0 + j) * ld + tb + tg) =
                    make_uint2(d[p][0], d[p][1]);
        }
        __syncthreads();
    }
}

// Pooled checkpoint: u[m][k'] = s[m] * (sum of 64 codes) / 64 as hi/lo terms of
// the compute dtype into [M][ld] buffers (columns past Da are zero).  The sum
// of codes is exact (at most 14 bits); the product is rounded once in fp32.
__global__ void k_int8_pool_split(const int8_t *__restrict__ codes, int64_t cld, const float *__restrict__ scales,
                                  int64_t M, int64_t Da, int64_t ld, uint16_t *__restrict__ hi,
                                  uint16_t *__restrict__ lo, bool f16) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= M * ld) return;
    const int64_t m = i / ld, k = i % ld;
    float v = 0.f;
    if (k < Da) {
        const uint4 *p = reinterpret_cast<const uint4 *>(codes + m * cld + k * 64);
        int sum = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint4 w = __ldg(p + e);
            sum = __dp4a((int)w.x, 0x01010101, sum);
            sum = __dp4a((int)w.y, 0x01010101, sum);
            sum = __dp4a((int)w.z, 0x01010101, sum);
            sum = __dp4a((int)w.w, 0x01010101, sum);
        }
        v = __fmul_rn((float)sum * 0.015625f, __ldg(scales + m));
    }
    const uint16_t h = enc16(v, f16);
    hi[i] = h;
    lo[i] = enc16(v - dec16(h, f16), f16);
}

// out[m][k] = RN_dt(code * s): 8 values a thread.
template <int DT>
__global__ void k_int8_dequantize(const int8_t *__restrict__ codes, int64_t ld, const float *__restrict__ scales,
                                  int64_t rows, int64_t cols, void *out, bool vec) {
    const int64_t nv = (cols + kVec - 1) / kVec;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < rows * nv;
         i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t m = i / nv, e0 = (i % nv) * kVec;
        const float s = __ldg(scales + m);
        const int8_t *src = codes + m * ld + e0;
        float v[kVec];
#pragma unroll
        for (int e = 0; e < kVec; ++e) v[e] = e0 + e < cols ? __fmul_rn((float)__ldg(src + e), s) : 0.f;
        if (DT == QLORA_DTYPE_FP32) {
            float *o = static_cast<float *>(out) + m * cols + e0;
            if (vec) {
                reinterpret_cast<float4 *>(o)[0] = make_float4(v[0], v[1], v[2], v[3]);
                reinterpret_cast<float4 *>(o)[1] = make_float4(v[4], v[5], v[6], v[7]);
            } else {
#pragma unroll
                for (int e = 0; e < kVec; ++e)
                    if (e0 + e < cols) o[e] = v[e];
            }
        } else {
            constexpr bool f16 = DT == QLORA_DTYPE_FP16;
            uint16_t *o = static_cast<uint16_t *>(out) + m * cols + e0;
            if (vec) {
                *reinterpret_cast<uint4 *>(o) = make_uint4(pack2(v[0], v[1], f16), pack2(v[2], v[3], f16),
                                                           pack2(v[4], v[5], f16), pack2(v[6], v[7], f16));
            } else {
#pragma unroll
                for (int e = 0; e < kVec; ++e)
                    if (e0 + e < cols) o[e] = enc16(v[e], f16);
            }
        }
    }
}

// Threads of a row's CTA: four steps of 8 values each keep a row of up to
// 32768 values in registers (fp32: two, 16384); longer ones are read a second
// time.
int row_threads(int64_t cols, int steps = 4) {
    const int64_t nv = (cols + kVec - 1) / kVec;
    int64_t t = (nv + steps - 1) / steps;
    t = (t + 31) / 32 * 32;
    return (int)(t > kMaxRowThreads ? kMaxRowThreads : t);
}
unsigned row_grid(int64_t rows) { return (unsigned)(rows < 0x7fffffff ? rows : 0x7fffffff); }

}  // namespace

int launch_int8_quantize(const void *X, int dtype, int64_t ldx, const int8_rows_t &q, uint32_t *d_status,
                         cudaStream_t st) {
    const int esize = dtype == QLORA_DTYPE_FP32 ? 4 : 2;
    const bool al = (reinterpret_cast<uintptr_t>(X) & 15u) == 0 && (ldx * esize) % 16 == 0;
    const int t = row_threads(q.cols, dtype == QLORA_DTYPE_FP32 ? 2 : 4);
    const unsigned g = row_grid(q.rows);
    if (dtype == QLORA_DTYPE_BF16)
        k_int8_quantize<QLORA_DTYPE_BF16><<<g, t, 0, st>>>(X, ldx, q.rows, q.cols, q.codes, q.ld, q.scales, al,
                                                            d_status);
    else if (dtype == QLORA_DTYPE_FP16)
        k_int8_quantize<QLORA_DTYPE_FP16><<<g, t, 0, st>>>(X, ldx, q.rows, q.cols, q.codes, q.ld, q.scales, al,
                                                            d_status);
    else
        k_int8_quantize<QLORA_DTYPE_FP32><<<g, t, 0, st>>>(X, ldx, q.rows, q.cols, q.codes, q.ld, q.scales, al,
                                                            d_status);
    QLORA_LAUNCH_CHECK();
    return QLORA_OK;
}

int launch_int8_row_digits(const uint16_t *Y, bool f16, int64_t rows, int64_t cols, const float *cscale,
                           int8_t *planes, int64_t ld, float *steps, cudaStream_t st) {
    const bool al = (reinterpret_cast<uintptr_t>(Y) & 15u) == 0 && cols % 8 == 0;
    const int t = row_threads(cols);
    if (f16)
        k_int8_row_digits<QLORA_DTYPE_FP16><<<row_grid(rows), t, 0, st>>>(Y, rows, cols, cscale, planes, ld, steps, al);
    else
        k_int8_row_digits<QLORA_DTYPE_BF16><<<row_grid(rows), t, 0, st>>>(Y, rows, cols, cscale, planes, ld, steps, al);
    QLORA_LAUNCH_CHECK();
    return QLORA_OK;
}

int launch_int8_col_digits(const void *S, int dtype, int64_t R, int r, const float *f, int8_t *planes, int64_t ld,
                           int rp, float *steps, cudaStream_t st) {
    const int64_t per = ((R + kColCluster - 1) / kColCluster + 15) / 16 * 16;
    const dim3 grid((unsigned)((rp + kColStrip - 1) / kColStrip), kColCluster);
    if (dtype == QLORA_DTYPE_FP32)
        k_int8_col_digits<QLORA_DTYPE_FP32><<<grid, kColThreads, 0, st>>>(S, R, r, f, per, planes, ld, rp, steps);
    else if (dtype == QLORA_DTYPE_FP16)
        k_int8_col_digits<QLORA_DTYPE_FP16><<<grid, kColThreads, 0, st>>>(S, R, r, f, per, planes, ld, rp, steps);
    else
        k_int8_col_digits<QLORA_DTYPE_BF16><<<grid, kColThreads, 0, st>>>(S, R, r, f, per, planes, ld, rp, steps);
    QLORA_LAUNCH_CHECK();
    return QLORA_OK;
}

int launch_int8_pool_split(const int8_rows_t &q, int64_t Da, int64_t ld, uint16_t *hi, uint16_t *lo,
                           cudaStream_t st, bool f16) {
    const int64_t n = q.rows * ld;
    if (n == 0) return QLORA_OK;
    k_int8_pool_split<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(q.codes, q.ld, q.scales, q.rows, Da, ld, hi, lo,
                                                                   f16);
    QLORA_LAUNCH_CHECK();
    return QLORA_OK;
}

int launch_int8_dequantize(const int8_rows_t &q, int dtype, void *out, cudaStream_t st) {
    const int64_t n = q.rows * ((q.cols + kVec - 1) / kVec);
    const int64_t want = (n + 255) / 256, most = (int64_t)device_sms() * 32;
    const unsigned g = (unsigned)(want < most ? want : most);
    const bool vec = q.cols % 8 == 0 && (reinterpret_cast<uintptr_t>(out) & 15u) == 0;
    if (dtype == QLORA_DTYPE_BF16)
        k_int8_dequantize<QLORA_DTYPE_BF16><<<g, 256, 0, st>>>(q.codes, q.ld, q.scales, q.rows, q.cols, out, vec);
    else if (dtype == QLORA_DTYPE_FP16)
        k_int8_dequantize<QLORA_DTYPE_FP16><<<g, 256, 0, st>>>(q.codes, q.ld, q.scales, q.rows, q.cols, out, vec);
    else
        k_int8_dequantize<QLORA_DTYPE_FP32><<<g, 256, 0, st>>>(q.codes, q.ld, q.scales, q.rows, q.cols, out, vec);
    QLORA_LAUNCH_CHECK();
    return QLORA_OK;
}

}  // namespace qlora
