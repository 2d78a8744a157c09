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

#include "int8_rows.cuh"

namespace qlora {
namespace {

constexpr int kMaxRowThreads = 1024;
constexpr int kDigitThreads = 512;

// One CTA per row; see launch_int8_quantize for its threads.  HBM-bound: the
// CTAs of an SM have to keep some 50 KB of loads in flight between them, so
// the variant for short rows holds its registers down for more CTAs.
template <int DT, int MOST>
__global__ void __launch_bounds__(MOST, MOST == kMaxRowThreads ? 1 : 1280 / MOST)
k_int8_quantize(const void *X, int64_t ldx, int cols, int8_t *codes, int64_t ld, float *scales,
                uint32_t *status) {
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    constexpr int esize = DT == QLORA_DTYPE_FP32 ? 4 : 2;
    constexpr int kSteps = kKeep<DT>;
    const int nv = (cols + kVec - 1) / kVec;
    const int64_t m = blockIdx.x;
    const char *row = static_cast<const char *>(X) + m * ldx * esize;
    Raw8<DT> keep[kSteps];
    uint32_t am = 0;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int v = i * blockDim.x + threadIdx.x;
        if (v < nv) keep[i] = load8<DT>(row, v, cols);
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
        if (i * (int)blockDim.x + (int)threadIdx.x < nv) am = absmax8<DT>(keep[i], am);
    for (int v = kSteps * blockDim.x + threadIdx.x; v < nv; v += blockDim.x)
        am = absmax8<DT>(load8<DT>(row, v, cols), am);
    am = block_max(absmax_bits<DT>(am));
    const bool fin = am < 0x7f800000u;
    const float a = __uint_as_float(am);
    const float s = fin ? __fdiv_rn(a, 127.f) : __uint_as_float(0x7fffffffu);
    if (threadIdx.x == 0) {
        scales[m] = s;
        if (!fin && status) atomicOr(status, QLORA_STATUS_NONFINITE);
    }
    int8_t *dst = codes + m * ld;
    const bool zero = !fin || s == 0.f;
    float inv = 0.f;
    const Decide how = zero ? kExact : decide<DT>(a, s, inv);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int v = i * blockDim.x + threadIdx.x;
        if (v < nv) {
            const uint2 c = zero ? make_uint2(0u, 0u) : encode8<DT>(keep[i], s, inv, how);
            store8(dst, v * kVec, cols, c.x, c.y);
        }
    }
    for (int v = kSteps * blockDim.x + threadIdx.x; v < nv; v += blockDim.x) {
        const uint2 c = zero ? make_uint2(0u, 0u) : encode8<DT>(load8<DT>(row, v, cols), s, inv, how);
        store8(dst, v * kVec, cols, c.x, c.y);
    }
}

// Rows of D = dY * scale[column] (RN32) in 16-bit fixed point, q = RN(D / step),
// step = a / 32639, as two digit planes.  A rounding is off by half a step,
// a / 65278, so a row by at most sqrt(cols) / 65278 of its norm whatever its
// values (about 4e-5 for normal ones): below the 16-bit output's own rounding.
template <int DT, int MOST>
__global__ void __launch_bounds__(MOST, MOST == kDigitThreads ? 2 : 1152 / MOST)
k_int8_row_digits(const void *Y, int64_t rows, int cols, const float *__restrict__ cscale,
                  int8_t *planes, int64_t ld, float *steps, bool vscale) {
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    constexpr int kSteps = 4;
    const int nv = (cols + kVec - 1) / kVec;
    const int64_t m = blockIdx.x;
    const char *row = static_cast<const char *>(Y) + m * cols * 2;
    // the scales come from L1 both times; the raw values alone stay in registers
    auto products = [&](const Raw8<DT> &r, int v, float (&d)[kVec]) {
        float f[kVec];
        if (vscale && v * kVec + kVec <= cols) {
            const float4 x = __ldg(reinterpret_cast<const float4 *>(cscale + v * kVec));
            const float4 y = __ldg(reinterpret_cast<const float4 *>(cscale + v * kVec) + 1);
            f[0] = x.x, f[1] = x.y, f[2] = x.z, f[3] = x.w, f[4] = y.x, f[5] = y.y, f[6] = y.z, f[7] = y.w;
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) f[e] = v * kVec + e < cols ? __ldg(cscale + v * kVec + e) : 0.f;
        }
#pragma unroll
        for (int e = 0; e < kVec; ++e) d[e] = __fmul_rn(val8(r, e), f[e]);
    };
    // NaN-keeping maximum of magnitudes, as integers
    auto join = [&](const Raw8<DT> &r, int v, uint32_t m) {
        float d[kVec];
        products(r, v, d);
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            const uint32_t b = __float_as_uint(d[e]) & 0x7fffffffu;
            m = b > m ? b : m;
        }
        return m;
    };
    Raw8<DT> keep[kSteps];
    uint32_t am = 0;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int v = i * blockDim.x + threadIdx.x;
        if (v < nv) keep[i] = load8<DT>(row, v, cols);
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int v = i * blockDim.x + threadIdx.x;
        if (v < nv) am = join(keep[i], v, am);
    }
    for (int v = kSteps * blockDim.x + threadIdx.x; v < nv; v += blockDim.x)
        am = join(load8<DT>(row, v, cols), v, am);
    am = block_max(am);
    const bool fin = am < 0x7f800000u;
    // magnitudes below 2^-60 are raised by 2^64 first, so that 1/step stays finite
    const float up = am < 0x21800000u ? 0x1p64f : 1.f;
    const float a = __uint_as_float(am) * up;
    const float inv = fin && a > 0.f ? __fdiv_rn(32639.f, a) : 0.f;
    if (threadIdx.x == 0) steps[m] = fin ? __fdiv_rn(a, 32639.f) / up : __uint_as_float(0x7fffffffu);
    int8_t *hi = planes + m * ld, *lo = planes + (rows + m) * ld;
    // |d * up * inv| <= 32639 (1 + 2^-23), so the magic addition rounds it to an
    // integer q in +-32639, whose 16 low bits are those of the sum's pattern;
    // the upper digit is the byte of q + 128 above its lower one.
    auto put = [&](const Raw8<DT> &r, int v) {
        float d[kVec];
        products(r, v, d);
        uint32_t q[kVec], h[kVec];
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            q[e] = fin ? __float_as_uint(__fmaf_rn(__fmul_rn(d[e], up), inv, kMagic)) : 0u;
            h[e] = q[e] + 128u;
        }
        auto second = [&](int e) {
            return __byte_perm(__byte_perm(h[e], h[e + 1], 0x0051), __byte_perm(h[e + 2], h[e + 3], 0x0051), 0x5410);
        };
        store8(hi, v * kVec, cols, second(0), second(4));
        store8(lo, v * kVec, cols, bytes4(q[0], q[1], q[2], q[3]), bytes4(q[4], q[5], q[6], q[7]));
    };
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int v = i * blockDim.x + threadIdx.x;
        if (v < nv) put(keep[i], v);
    }
    for (int v = kSteps * blockDim.x + threadIdx.x; v < nv; v += blockDim.x)
        put(load8<DT>(row, v, cols), v);
}

// Columns of S[t][j] (rows t < R, columns j < r; 16-bit or fp32), optionally
// times f[t], in 24-bit fixed point with one step per column, as three digit
// planes transposed to planes[d][j][t] (rows of ld bytes, rp rows a plane).
// A step is max / 8355711: half of it is 6e-8 of the column's largest value.
// A cluster of 8 CTAs shares 8 columns: each finds the maxima of its rows,
// keeping the values in shared memory (up to kColKeep rows; past them they are
// read again), and the cluster joins the maxima over distributed shared memory.
constexpr int kColStrip = 8, kColKeep = 1024, kColCluster = 8, kColThreads = 256;
constexpr int kColBatch = 16;          // loads in flight a thread
constexpr float kColMax = 8355711.f;   // 127 * (65536 + 256 + 1)

template <int DT>
__global__ void __cluster_dims__(1, kColCluster, 1) __launch_bounds__(kColThreads)
k_int8_col_digits(const void *S, int64_t R, int r, const float *__restrict__ f, int64_t per,
                  int8_t *planes, int64_t ld, int rp, float *steps) {
    namespace cg = cooperative_groups;
    __shared__ uint32_t cmax[kColStrip];
    __shared__ float tile[kColStrip][kColKeep + 1];
    cg::cluster_group cl = cg::this_cluster();
    const int j0 = blockIdx.x * kColStrip;
    const int64_t t0 = (int64_t)blockIdx.y * per;
    const int64_t t1 = t0 + per < R ? t0 + per : R;
    const int tid = threadIdx.x, j = tid % kColStrip, tr = tid / kColStrip;
    constexpr int kRows = kColThreads / kColStrip;      // rows a pass of the CTA
    auto value = [&](int64_t t) -> float {
        if (t >= t1 || j0 + j >= r) return 0.f;
        const float v = DT == QLORA_DTYPE_FP32 ? __ldg(static_cast<const float *>(S) + t * r + j0 + j)
                                               : dec16(__ldg(static_cast<const uint16_t *>(S) + t * r + j0 + j),
                                                       DT == QLORA_DTYPE_FP16);
        return f ? __fmul_rn(v, __ldg(f + t)) : v;
    };
    // values of rows [tb, tb + kColKeep) into the tile; their largest magnitude's bits
    auto fill = [&](int64_t tb) -> uint32_t {
        uint32_t m = 0;
        for (int k0 = 0; k0 < kColKeep && tb + k0 < t1; k0 += kRows * kColBatch) {
            float v[kColBatch];
#pragma unroll
            for (int i = 0; i < kColBatch; ++i) v[i] = value(tb + k0 + i * kRows + tr);
#pragma unroll
            for (int i = 0; i < kColBatch; ++i) {
                const uint32_t b = __float_as_uint(v[i]) & 0x7fffffffu;
                m = b > m ? b : m;
                tile[j][k0 + i * kRows + tr] = v[i];
            }
        }
        return m;
    };
    if (tid < kColStrip) cmax[tid] = 0;
    __syncthreads();
    uint32_t m = 0;
    for (int64_t tb = t0; tb < t1; tb += kColKeep) {
        const uint32_t o = fill(tb);
        m = o > m ? o : m;
    }
#pragma unroll
    for (int x = kColStrip; x < 32; x *= 2) {
        const uint32_t o = __shfl_xor_sync(0xffffffffu, m, x);
        m = o > m ? o : m;
    }
    if ((tid & 31) < kColStrip) atomicMax(&cmax[j], m);
    cl.sync();
    // every thread joins the maxima of the column that it converts
    const int jc = tid / kRows, tg = (tid % kRows) * 8;   // 8 rows of column jc at a time
    m = 0;
#pragma unroll
    for (int c = 0; c < kColCluster; ++c) {
        const uint32_t o = *cl.map_shared_rank(&cmax[jc], c);
        m = o > m ? o : m;
    }
    cl.sync();   // the maxima have been read before any CTA leaves
    const bool fin = m < 0x7f800000u;
    const float up = m < 0x21800000u ? 0x1p64f : 1.f;
    const float a = __uint_as_float(m) * up;
    const float inv = fin && a > 0.f ? __fdiv_rn(kColMax, a) : 0.f;
    if (blockIdx.y == 0 && tg == 0 && j0 + jc < rp)
        steps[j0 + jc] = fin ? __fdiv_rn(a, kColMax) / up : __uint_as_float(0x7fffffffu);
    const bool again = t1 - t0 > kColKeep;
    for (int64_t tb = t0; tb < t1; tb += kColKeep) {
        if (again) {
            __syncthreads();
            fill(tb);
            __syncthreads();
        }
        for (int k = tg; k < kColKeep && tb + k < t1; k += kRows * 8) {
            if (j0 + jc >= rp) break;
            uint32_t d[3][2] = {};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float x = inv > 0.f ? fminf(fmaxf(tile[jc][k + e] * up * inv, -kColMax), kColMax) : 0.f;
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
                *reinterpret_cast<uint2 *>(planes + ((int64_t)p * rp + j0 + jc) * ld + tb + k) =
                    make_uint2(d[p][0], d[p][1]);
        }
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

// Threads of a row's CTA, `steps` of 8 values each in registers; what a row
// has past most * steps * 8 values is read a second time.
int row_threads(int64_t cols, int steps, int most) {
    const int64_t nv = (cols + kVec - 1) / kVec;
    const int64_t t = ((nv + steps - 1) / steps + 31) / 32 * 32;
    return (int)(t > most ? most : t);
}

template <int DT>
auto pick_quantize(int threads) {
    return threads <= 256 ? k_int8_quantize<DT, 256> : k_int8_quantize<DT, kMaxRowThreads>;
}

template <int DT>
auto pick_row_digits(int threads) {
    return threads <= 384 ? k_int8_row_digits<DT, 384> : k_int8_row_digits<DT, kDigitThreads>;
}

}  // namespace

int launch_int8_quantize(const void *X, int dtype, int64_t ldx, const int8_rows_t &q, uint32_t *d_status,
                         cudaStream_t st) {
    const int t = row_threads(q.cols, dtype == QLORA_DTYPE_FP32 ? kKeep<QLORA_DTYPE_FP32> : kKeep<QLORA_DTYPE_BF16>,
                              kMaxRowThreads);
    auto *k = dtype == QLORA_DTYPE_BF16   ? pick_quantize<QLORA_DTYPE_BF16>(t)
              : dtype == QLORA_DTYPE_FP16 ? pick_quantize<QLORA_DTYPE_FP16>(t)
                                          : pick_quantize<QLORA_DTYPE_FP32>(t);
    k<<<(unsigned)q.rows, t, 0, st>>>(X, ldx, (int)q.cols, q.codes, q.ld, q.scales, d_status);
    QLORA_LAUNCH_CHECK();
    return QLORA_OK;
}

int launch_int8_row_digits(const uint16_t *Y, bool f16, int64_t rows, int64_t cols, const float *cscale,
                           int8_t *planes, int64_t ld, float *steps, cudaStream_t st) {
    const bool vscale = (reinterpret_cast<uintptr_t>(cscale) & 15u) == 0;
    const int t = row_threads(cols, 4, kDigitThreads);
    auto *k = f16 ? pick_row_digits<QLORA_DTYPE_FP16>(t) : pick_row_digits<QLORA_DTYPE_BF16>(t);
    k<<<(unsigned)rows, t, 0, st>>>(Y, rows, (int)cols, cscale, planes, ld, steps, vscale);
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
