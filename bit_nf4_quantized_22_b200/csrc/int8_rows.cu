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
//   .. in 32 bits, four digits (|q| <= 2^30)       those that 16 bits would take too much from
//   q = 65536 d2 + 256 d1 + d0 (|q| <= 8355711)   columns of A, of scale * G
// so that the integer tensor cores give the product of the full operand, as
// the digits' products added with their weights.
#include <cooperative_groups.h>

#include "int8_rows.cuh"

namespace qlora {
namespace {

// Most threads of a row's CTA: what the steps' registers leave room for.
constexpr int row_threads(int steps) { return steps >= 8 ? 512 : 1024; }

// A CTA (WARP: a warp, eight rows a CTA) per row, STEPS x 8 values a thread in
// registers between the maximum and the codes (what a longer row has past them
// is read again).  HBM-bound: many rows want few threads with many loads each
// (28672 x 8192 bf16: 8 steps 102 us, 6.9 TB/s; 4 steps 116, 1 step 204; rows
// brought through shared memory by bulk copies into persistent CTAs 119), short
// rows a warp each without a barrier (28672 x 1024: 15 us, a CTA 31).
template <int DT, bool FULL, int STEPS, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : row_threads(STEPS))
k_int8_quantize(const void *X, int64_t ldx, int64_t rows, int cols, int8_t *codes, int64_t ld, float *scales,
                uint32_t *status) {
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    constexpr int esize = DT == QLORA_DTYPE_FP32 ? 4 : 2;
    const int64_t m = WARP ? (int64_t)blockIdx.x * 8 + threadIdx.x / 32 : blockIdx.x;
    if (WARP && m >= rows) return;
    const int tid = WARP ? threadIdx.x & 31 : threadIdx.x, threads = WARP ? 32 : blockDim.x;
    const char *row = static_cast<const char *>(X) + m * ldx * esize;
    const uint32_t off = row_offset<FULL>(row);
    const RowSpan span = row_span<DT, FULL>(off, cols);
    const int first = span.v0 + tid;
    Raw8<DT> keep[STEPS], edge{};
    uint32_t am = 0;
    if (!FULL && tid < span.edges) edge = edge8<DT>(row, span.edge(tid));
    load_steps<DT, FULL, STEPS>(row, off, first, threads, span.v1, keep);
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
        if (first + i * threads < span.v1) am = absmax8<DT>(keep[i], am);
    for (int v = first + STEPS * threads; v < span.v1; v += threads) {
        Raw8<DT> x;
        load_steps<DT, FULL, 1>(row, off, v, threads, span.v1, &x);
        am = absmax8<DT>(x, am);
    }
    if (!FULL) am = absmax8<DT>(edge, am);
    am = absmax_bits<DT>(am);
    am = WARP ? __reduce_max_sync(0xffffffffu, am) : block_max(am);
    const RowCode rc = row_code<DT>(am);
    if (tid == 0) {
        scales[m] = rc.s;
        if (!rc.mask && status) atomicOr(status, QLORA_STATUS_NONFINITE);
    }
    int8_t *dst = codes + m * ld;
    float far = 0.f;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int v = first + i * threads;
        if (v < span.v1) {
            const uint2 c = encode8<DT>(keep[i], rc, far);
            store8<true>(dst, v * kVec, cols, c.x, c.y);
        }
    }
    for (int v = first + STEPS * threads; v < span.v1; v += threads) {
        Raw8<DT> x;
        load_steps<DT, FULL, 1>(row, off, v, threads, span.v1, &x);
        const uint2 c = encode8<DT>(x, rc, far);
        store8<true>(dst, v * kVec, cols, c.x, c.y);
    }
    if (!FULL && tid < span.edges) dst[span.edge(tid)] = (int8_t)(uint8_t)(encode8<DT>(edge, rc, far).x & 255u);
    if (rc.exact || far > kFar) {
        encode_exact<DT>(row, first, threads, cols, rc.s, dst, nullptr);
        if (!FULL && tid < span.edges) dst[span.edge(tid)] = (int8_t)code_exact<DT>(val8(edge, 0), rc.s);
    }
}

// Rows of D = dY * scale[column] (RN32) in 16-bit fixed point, q = RN(D / step),
// step = a / 32639, as two digit planes; a row that this would take too much from
// in 32 bits, step the power of two with a / step in [2^29, 2^30), as four
// (`deep`: its planes then hold those digits instead).
//
// What 16 bits take from a row is known once its digits are: with h half a step of
// the result's type (bf16 2^-8, fp16 2^-11) and ||D|| from the upper digits,
//   the roundings' noise, sqrt(cols / 12) step              <= h / 4 ||D||
//   the values under 8 steps, a quarter of a step each      <= h / 4 ||D||
//   the roundings' sum, which weights with a mean multiply  <= h / 2 ||D||
// Normal rows pass (4096 to 131072 columns: noise 3e-5 to 5e-5 of their norm), a
// loss's softmax - onehot does not: thousands of values under half a step, all of
// one sign, would be lost. The three are sums of integers, so a row's choice is its own
// whatever kernel, thread or batch makes it.  32 bits keep every value to
// max 2^-30: 131072 of them to 2^-13 of the largest, and D's own fp32 where a
// value is within 2^-6 of it.  Rows below 2^-111, whose 16-bit step would be subnormal
// (it would lose up to all of its own bits), are cut in 32 bits too.
//
// The scales of one vector's columns (from L1 the second time).
template <bool FULL>
__device__ __forceinline__ void digit_scales(const float *__restrict__ cscale, int v, float (&f)[kVec]) {
    if (FULL || (reinterpret_cast<uintptr_t>(cscale) & 15u) == 0) {
        const float4 x = __ldg(reinterpret_cast<const float4 *>(cscale + v * kVec));
        const float4 y = __ldg(reinterpret_cast<const float4 *>(cscale + v * kVec) + 1);
        f[0] = x.x, f[1] = x.y, f[2] = x.z, f[3] = x.w, f[4] = y.x, f[5] = y.y, f[6] = y.z, f[7] = y.w;
    } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e) f[e] = __ldg(cscale + v * kVec + e);
    }
}
template <int DT>
__device__ __forceinline__ void digit_products(const Raw8<DT> &r, const float (&f)[kVec], float (&d)[kVec]) {
#pragma unroll
    for (int e = 0; e < kVec; ++e) d[e] = __fmul_rn(val8(r, e), f[e]);
}
// Running maximum of magnitudes that keeps a NaN (the sign of m is of no account).
__device__ __forceinline__ float digit_max(const float (&d)[kVec], float m) {
#pragma unroll
    for (int e = 0; e < kVec; ++e) asm("max.NaN.xorsign.abs.f32 %0, %0, %1;\n" : "+f"(m) : "f"(d[e]));
    return m;
}
struct RowDigits {
    float step, up, inv;
    bool fin;
};
__device__ __forceinline__ RowDigits row_digits(uint32_t am) {
    RowDigits r;
    r.fin = am < 0x7f800000u;
    // magnitudes below 2^-60 are raised by 2^64 first, so that 1/step stays finite
    r.up = am < 0x21800000u ? 0x1p64f : 1.f;
    const float a = __uint_as_float(am) * r.up;
    r.inv = r.fin && a > 0.f ? __fdiv_rn(32639.f, a) : 0.f;
    r.step = r.fin ? __fdiv_rn(a, 32639.f) / r.up : __uint_as_float(0x7fffffffu);
    return r;
}
// What 16 bits take from a row: the upper digits' squares, 128 times the roundings'
// sum (mod 2^32, as bit patterns of magic numbers), the values under 8 steps.
struct DigitLoss {
    uint32_t squares, sum, small;
};
constexpr uint32_t kDigitZero = 0x4b408080u;   // kMagic + 32896.f: q = 0
// Each value adds (kMagic + 128 x)'s bits less 128 times those of q.
constexpr uint32_t kLossBase = 0x4b400000u - 128u * kDigitZero;

__device__ __forceinline__ void digit_loss(float d, float t, float inv128, DigitLoss &l) {
    // |128 x| <= 4177792.5 < 2^22: the magic addition rounds it to an integer too
    l.sum += __float_as_uint(__fmaf_rn(d, inv128, kMagic)) - 128u * __float_as_uint(t);
    l.small += __float_as_uint(t) - (kDigitZero - 7u) <= 14u ? 1u : 0u;
}
// |d up inv| <= 32639 (1 + 2^-23), so the magic addition rounds it to an integer
// q in +-32639.  With 32768 + 128 in the magic number, the sum's 16 low bits are
// 256 (d1 + 128) + (d0 + 128): both digits with their top bit flipped, each in
// a byte of its own.
__device__ __forceinline__ void put_digits(float (&d)[kVec], const RowDigits &r, int8_t *hi, int8_t *lo, DigitLoss &l) {
    uint32_t q[kVec / 2];
    if (r.up != 1.f) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) d[e] = __fmul_rn(d[e], r.up);
    }
    const float inv128 = r.inv * 128.f;
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
        const float t = __fmaf_rn(d[e], r.inv, kMagic + 32896.f);
        digit_loss(d[e], t, inv128, l);
        d[e] = t;
    }
    const uint32_t keep = r.fin ? 0xffffffffu : 0u;
#pragma unroll
    for (int i = 0; i < kVec / 2; ++i)
        q[i] = (__byte_perm(__float_as_uint(d[2 * i]), __float_as_uint(d[2 * i + 1]), 0x5410) ^ 0x80808080u) & keep;
    const uint2 upper = make_uint2(__byte_perm(q[0], q[1], 0x7531), __byte_perm(q[2], q[3], 0x7531));
    l.squares = __dp4a((int)upper.x, (int)upper.x, (int)l.squares);
    l.squares = __dp4a((int)upper.y, (int)upper.y, (int)l.squares);
    *reinterpret_cast<uint2 *>(hi) = upper;
    *reinterpret_cast<uint2 *>(lo) = make_uint2(__byte_perm(q[0], q[1], 0x6420), __byte_perm(q[2], q[3], 0x6420));
}
__device__ __forceinline__ void put_digit(float d, const RowDigits &r, int8_t *hi, int8_t *lo, DigitLoss &l) {
    d = __fmul_rn(d, r.up);
    const float t = __fmaf_rn(d, r.inv, kMagic + 32896.f);
    digit_loss(d, t, r.inv * 128.f, l);
    const uint32_t q = (__float_as_uint(t) ^ 0x8080u) & (r.fin ? 0xffffu : 0u);
    const int upper = (int8_t)(uint8_t)(q >> 8);
    l.squares += (uint32_t)(upper * upper);
    *hi = (int8_t)upper;
    *lo = (int8_t)(uint8_t)(q & 255u);
}

// Do 16 bits take too much?  squares counts ||D||^2 in steps of 256: with h^2 =
// 2^-16 (bf16) or 2^-22 the three bounds are 4 cols <= 3 squares (or their 2^-6),
// small^2 <= squares and sum^2 <= 2^12 squares.
__device__ __forceinline__ bool loss_matters(uint32_t squares, int sum, uint32_t small, int cols, bool f16) {
    const uint64_t s = f16 ? squares >> 6 : squares;
    return 4 * (uint64_t)cols > 3 * s || (uint64_t)small * small > s ||
           (uint64_t)((int64_t)sum * sum) > s << 12;
}

__device__ __forceinline__ uint32_t block_sum(uint32_t v, uint32_t *part) {   // part: 32 words, free before and after
    v = __reduce_add_sync(0xffffffffu, v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    return __reduce_add_sync(0xffffffffu, (threadIdx.x & 31) < blockDim.x >> 5 ? part[threadIdx.x & 31] : 0u);
}

// The power of two of a deep row's step, and values over it.  2^-149 is the unit
// of D itself: no smaller step is needed.
constexpr uint32_t kTinyRow = 0x08000000u;     // 2^-111, as bits
struct DeepStep {
    float step, mul0, mul1;
};
__device__ __forceinline__ DeepStep deep_step(uint32_t am) {
    int k = (int)(am >> 23) - 127 - 29;
    k = k < -149 ? -149 : k;
    const int a = -k / 2, b = -k - a;    // in two factors: 2^149 is past fp32's range
    DeepStep s;
    s.step = __uint_as_float(k >= -126 ? (uint32_t)(k + 127) << 23 : 1u << (k + 149));
    s.mul0 = __uint_as_float((uint32_t)(a + 127) << 23);
    s.mul1 = __uint_as_float((uint32_t)(b + 127) << 23);
    return s;
}

// A row that the whole CTA finds beyond 16 bits: zeros, which lose nothing, come out of the values under 8
// steps; if too much is still lost, the row's four planes.  Out of line: ordinary rows do not come here.
template <int DT>
__device__ __noinline__ bool deep_row(const char *row, int cols, const float *__restrict__ cscale, uint32_t am,
                                      uint32_t squares, int sum, uint32_t small, int8_t *planes, int64_t plane,
                                      uint32_t *part) {
    const int nv = (cols + kVec - 1) / kVec;
    uint32_t zeros = 0;
    for (int v = threadIdx.x; v < nv; v += blockDim.x) {
        const Raw8<DT> r = load8<DT, false>(row, v, cols);
#pragma unroll
        for (int e = 0; e < kVec; ++e) zeros += v * kVec + e < cols && val8(r, e) == 0.f;
    }
    zeros = block_sum(zeros, part);
    if (am >= kTinyRow && !loss_matters(squares, sum, small - zeros, cols - (int)zeros, DT == QLORA_DTYPE_FP16))
        return false;
    const DeepStep ds = deep_step(am);
    for (int v = threadIdx.x; v < nv; v += blockDim.x) {
        const Raw8<DT> r = load8<DT, false>(row, v, cols);
        uint32_t d[4][2] = {};
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            const float x = __fmul_rn(val8(r, e), __ldg(cscale + (v * kVec + e < cols ? v * kVec + e : cols - 1)));
            int q = __float2int_rn(x * ds.mul0 * ds.mul1);           // |q| <= 2^30
#pragma unroll
            for (int p = 3; p >= 0; --p) {
                const int b = (int)(int8_t)(uint8_t)q;
                q = (q - b) >> 8;
                d[p][e / 4] |= (uint32_t)(uint8_t)b << (8 * (e & 3));
            }
        }
#pragma unroll
        for (int p = 0; p < 4; ++p) store8<false>(planes + p * plane, v * kVec, cols, d[p][0], d[p][1]);
    }
    return true;
}

// ROWS rows a CTA: the scales, read for the maxima and again for the digits, are
// most of the traffic inside the SM, and two rows share them.  64 registers, for two
// CTAs an SM of long rows too.  4096 x 11008: 51 us, 127 where all rows take four planes;
// what DigitLoss sums costs 14 of them (37 us without, one row a CTA 41; 4258 x 14856: 66
// us, 46 without, 67 with 78 registers).
template <int DT, bool FULL, int STEPS, int ROWS>
__global__ void __launch_bounds__(STEPS == 4 ? 512 : 1024, STEPS == 4 ? 2 : 1)
k_int8_row_digits(const void *Y, int64_t rows, int cols, const float *__restrict__ cscale,
                  int8_t *planes, int64_t ld, float *steps, uint8_t *deep) {
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    __shared__ uint32_t part[ROWS][32], sums[ROWS][3][32];
    const int64_t m0 = (int64_t)blockIdx.x * ROWS;
    const int threads = blockDim.x;
    const char *row[ROWS];
    uint32_t off[ROWS];
    RowSpan span{0, 0x7fffffff, 0};     // the rows' common one: they share the scales of a vector
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {    // a last odd row stands in for its missing neighbour too
        row[i] = static_cast<const char *>(Y) + (m0 + i < rows ? m0 + i : m0) * (int64_t)cols * 2;
        off[i] = row_offset<FULL>(row[i]);
        const RowSpan one = row_span<DT, FULL>(off[i], cols);
        span.v0 = one.v0 > span.v0 ? one.v0 : span.v0;
        span.v1 = one.v1 < span.v1 ? one.v1 : span.v1;
    }
    if (span.v1 <= span.v0) span.v0 = span.v1 = 0;
    span.edges = cols - (span.v1 - span.v0) * kVec;
    const int first = span.v0 + threadIdx.x;
    const bool ends = !FULL && (int)threadIdx.x < span.edges;
    const int at = ends ? span.edge(threadIdx.x) : 0;
    Raw8<DT> keep[ROWS][STEPS];
    float top[ROWS] = {}, d[kVec], edge[ROWS] = {};
    if (ends) {
        const float f = __ldg(cscale + at);
#pragma unroll
        for (int i = 0; i < ROWS; ++i) edge[i] = __fmul_rn(val8(edge8<DT>(row[i], at), 0), f);
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) load_steps<DT, FULL, STEPS>(row[i], off[i], first, threads, span.v1, keep[i]);
#pragma unroll
    for (int j = 0; j < STEPS; ++j) {
        const int v = first + j * threads;
        if (v < span.v1) {
            float f[kVec];
            digit_scales<FULL>(cscale, v, f);
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                digit_products<DT>(keep[i][j], f, d);
                top[i] = digit_max(d, top[i]);
            }
        }
    }
    for (int v = first + STEPS * threads; v < span.v1; v += threads) {
        float f[kVec];
        digit_scales<FULL>(cscale, v, f);
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            Raw8<DT> x;
            load_steps<DT, FULL, 1>(row[i], off[i], v, threads, span.v1, &x);
            digit_products<DT>(x, f, d);
            top[i] = digit_max(d, top[i]);
        }
    }
    RowDigits r[ROWS];
    DigitLoss loss[ROWS] = {};
    uint32_t am[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        if (!FULL) asm("max.NaN.xorsign.abs.f32 %0, %0, %1;\n" : "+f"(top[i]) : "f"(edge[i]));
        const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(top[i]) & 0x7fffffffu);
        if ((threadIdx.x & 31) == 0) part[i][threadIdx.x >> 5] = m;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const uint32_t m = (threadIdx.x & 31) < blockDim.x >> 5 ? part[i][threadIdx.x & 31] : 0u;
        am[i] = __reduce_max_sync(0xffffffffu, m);
        r[i] = row_digits(am[i]);
    }
    auto put = [&](const Raw8<DT> &x, int i, int v, const float (&f)[kVec]) {
        if (m0 + i >= rows) return;
        digit_products<DT>(x, f, d);
        put_digits(d, r[i], planes + (m0 + i) * ld + v * kVec, planes + (rows + m0 + i) * ld + v * kVec, loss[i]);
    };
#pragma unroll
    for (int j = 0; j < STEPS; ++j) {
        const int v = first + j * threads;
        if (v < span.v1) {
            float f[kVec];
            digit_scales<FULL>(cscale, v, f);
#pragma unroll
            for (int i = 0; i < ROWS; ++i) put(keep[i][j], i, v, f);
        }
    }
    for (int v = first + STEPS * threads; v < span.v1; v += threads) {
        float f[kVec];
        digit_scales<FULL>(cscale, v, f);
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            Raw8<DT> x;
            load_steps<DT, FULL, 1>(row[i], off[i], v, threads, span.v1, &x);
            put(x, i, v, f);
        }
    }
    if (ends) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
            if (m0 + i < rows)
                put_digit(edge[i], r[i], planes + (m0 + i) * ld + at, planes + (rows + m0 + i) * ld + at, loss[i]);
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const uint32_t w[3] = {loss[i].squares, loss[i].sum, loss[i].small};
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const uint32_t t = __reduce_add_sync(0xffffffffu, w[k]);
            if ((threadIdx.x & 31) == 0) sums[i][k][threadIdx.x >> 5] = t;
        }
    }
    __syncthreads();
#pragma unroll 1
    for (int i = 0; i < ROWS && m0 + i < rows; ++i) {
        uint32_t w[3];
#pragma unroll
        for (int k = 0; k < 3; ++k)
            w[k] = __reduce_add_sync(0xffffffffu, (threadIdx.x & 31) < blockDim.x >> 5 ? sums[i][k][threadIdx.x & 31] : 0u);
        const int sum = (int)(w[1] - (uint32_t)cols * kLossBase);
        const uint32_t a = i == 0 ? am[0] : am[ROWS - 1];
        // the same for the whole CTA; a zero row and one that is not finite have no digits to lose
        const bool is_deep = a > 0 && a < 0x7f800000u &&
                             (a < kTinyRow || loss_matters(w[0], sum, w[2], cols, DT == QLORA_DTYPE_FP16)) &&
                             deep_row<DT>(i == 0 ? row[0] : row[ROWS - 1], cols, cscale, a, w[0], sum, w[2],
                                          planes + (m0 + i) * ld, rows * ld, part[0]);
        if (threadIdx.x == 0) {
            steps[m0 + i] = is_deep ? deep_step(a).step : i == 0 ? r[0].step : r[ROWS - 1].step;
            deep[m0 + i] = is_deep;
        }
    }
    if (m0 + ROWS >= rows)    // zeros up to whole tiles of 256 rows
        for (int64_t m = rows + threadIdx.x; m < (rows + 255) / 256 * 256; m += threads) deep[m] = 0;
}

// Columns of S[t][j] (rows t < R, columns j < r; 16-bit or fp32), optionally
// times f[t], in 24-bit fixed point with one step per column, as three digit
// planes transposed to planes[d][j][t] (rows of ld bytes, rp rows a plane).
// A step is max / 8355711, and a value its nearest multiple, within half of it (6e-8
// of the column's largest value): the product by the step's reciprocal, three
// roundings of up to half a step each near the maximum, is corrected by what it
// leaves of the value (1.7 steps at worst without).  Columns below 2^-100, whose step would
// be subnormal and lose bits of its own, take a power of two.
// rep = 64 writes each row's digits 64 times over (t -> 64 t .. 64 t + 63).
// A cluster of 8 CTAs shares 8 columns: each finds the maxima of its rows,
// keeping the values in shared memory (up to kColKeep rows; past them they are
// read again), and the cluster joins the maxima over distributed shared memory.
// Latency-bound: 5 us for 4096 rows of 64 columns, 1 MB (16 loads in flight a
// thread; one at a time took 20).
constexpr int kColStrip = 8, kColKeep = 1024, kColCluster = 8, kColThreads = 256;
constexpr int kColBatch = 16;          // loads in flight a thread
constexpr float kColMax = 8355711.f;   // 127 * (65536 + 256 + 1)

template <int DT>
__global__ void __cluster_dims__(1, kColCluster, 1) __launch_bounds__(kColThreads)
k_int8_col_digits(const void *S, int64_t R, int r, const float *__restrict__ f, int64_t per,
                  int8_t *planes, int64_t ld, int rp, int rep, float *steps) {
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
    // below 2^-100: the power of two with max / step in [2^21, 2^22), but no less than 2^-149
    const int tiny = (int)(m >> 23) - 127 - 21 < -149 ? -149 : (int)(m >> 23) - 127 - 21;
    const float unit = m < 0x0d800000u ? ldexpf(1.f, tiny + 64) : __fdiv_rn(a, kColMax);   // the step, times up
    const float inv = fin && a > 0.f ? __fdiv_rn(1.f, unit) : 0.f;
    if (blockIdx.y == 0 && tg == 0 && j0 + jc < rp) steps[j0 + jc] = fin ? unit / up : __uint_as_float(0x7fffffffu);
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
                const float v = tile[jc][k + e] * up;
                const float t = inv > 0.f ? rintf(v * inv) : 0.f;
                const float x = inv > 0.f ? t + rintf(__fmaf_rn(-t, unit, v) * inv) : 0.f;   // integers below 2^24: exact
                const int q = __float2int_rn(fminf(fmaxf(x, -kColMax), kColMax));
                const int b0 = (int)(int8_t)(uint8_t)q;
                const int q1 = (q - b0) >> 8;
                const int b1 = (int)(int8_t)(uint8_t)q1;
                const int b2 = (q1 - b1) >> 8;
                d[0][e / 4] |= (uint32_t)(uint8_t)b2 << (8 * (e & 3));
                d[1][e / 4] |= (uint32_t)(uint8_t)b1 << (8 * (e & 3));
                d[2][e / 4] |= (uint32_t)(uint8_t)b0 << (8 * (e & 3));
            }
#pragma unroll
            for (int p = 0; p < 3; ++p) {
                int8_t *row = planes + ((int64_t)p * rp + j0 + jc) * ld;
                if (rep == 1) {
                    *reinterpret_cast<uint2 *>(row + tb + k) = make_uint2(d[p][0], d[p][1]);
                    continue;
                }
                for (int e = 0; e < 8 && tb + k + e < t1; ++e) {
                    const uint32_t b = ((d[p][e / 4] >> (8 * (e & 3))) & 255u) * 0x01010101u;
                    for (int i = 0; i < 4; ++i)
                        reinterpret_cast<uint4 *>(row + (tb + k + e) * 64)[i] = make_uint4(b, b, b, b);
                }
            }
        }
    }
}

// out[m][k] = RN_dt(code * s): 8 values a thread.  Bound by the bytes written, as
// nf4_dequantize is (28672 x 8192 into bf16: 133 us, 5.3 TB/s).
template <int DT>
__global__ void k_int8_dequantize(const int8_t *__restrict__ codes, int64_t ld, const float *__restrict__ scales,
                                  int64_t rows, int64_t cols, void *out, bool vec) {
    const int64_t nv = (cols + kVec - 1) / kVec;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < rows * nv;
         i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t m = i / nv, e0 = (i % nv) * kVec;
        const float s = __ldg(scales + m);
        const int8_t *src = codes + m * ld + e0;
        uint2 c = make_uint2(0u, 0u);
        if (e0 + kVec <= cols) {
            c = __ldg(reinterpret_cast<const uint2 *>(src));
        } else {
            for (int e = 0; e0 + e < cols; ++e)
                (e < 4 ? c.x : c.y) |= (uint32_t)(uint8_t)__ldg(src + e) << (8 * (e & 3));
        }
        float v[kVec];
#pragma unroll
        for (int e = 0; e < kVec; ++e)
            v[e] = __fmul_rn((float)(int8_t)(uint8_t)((e < 4 ? c.x : c.y) >> (8 * (e & 3))), s);
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

// Steps of a row's CTA: one while every warp of every row has a place on the
// GPU at once, two up to six times that, eight past it (fp32, whose codes cost
// more instructions: two).
int row_steps(int64_t rows, int64_t cols, bool f32) {
    const int64_t nv = (cols + kVec - 1) / kVec, warps = rows * ((nv + 31) / 32), places = 32 * (int64_t)device_sms();
    if (nv <= row_threads(1) && warps <= places) return 1;
    if (f32 || (nv <= 2 * row_threads(2) && warps <= 6 * places)) return 2;
    return 8;
}
int row_cta(int64_t cols, int steps) {
    const int64_t nv = (cols + kVec - 1) / kVec, t = ((nv + steps - 1) / steps + 31) / 32 * 32;
    return (int)(t > row_threads(steps) ? row_threads(steps) : t);
}

template <int DT, bool FULL>
int launch_quantize(const void *X, int64_t ldx, const int8_rows_t &q, uint32_t *status, cudaStream_t st) {
    constexpr bool f32 = DT == QLORA_DTYPE_FP32;
    constexpr int kWarpSteps = f32 ? 2 : 4;
    const int cols = (int)q.cols;
    if (cols <= 32 * kVec * kWarpSteps && q.rows >= 2 * device_sms()) {
        k_int8_quantize<DT, FULL, kWarpSteps, true><<<(unsigned)((q.rows + 7) / 8), 256, 0, st>>>(
            X, ldx, q.rows, cols, q.codes, q.ld, q.scales, status);
    } else {
        const int steps = row_steps(q.rows, q.cols, f32);
        auto *k = steps == 1   ? k_int8_quantize<DT, FULL, 1, false>
                  : steps == 2 ? k_int8_quantize<DT, FULL, 2, false>
                               : k_int8_quantize<DT, FULL, f32 ? 2 : 8, false>;
        k<<<(unsigned)q.rows, row_cta(q.cols, steps), 0, st>>>(X, ldx, q.rows, cols, q.codes, q.ld, q.scales, status);
    }
    QLORA_LAUNCH_CHECK();
    return QLORA_OK;
}

template <int DT, bool FULL>
int launch_row_digits(const uint16_t *Y, int64_t rows, int64_t cols, const float *cscale, int8_t *planes, int64_t ld,
                      float *steps, uint8_t *deep, cudaStream_t st) {
    const int n = row_steps(rows, cols, false), per = n == 8 ? 2 : 1;
    auto *k = n == 1   ? k_int8_row_digits<DT, FULL, 1, 1>
              : n == 2 ? k_int8_row_digits<DT, FULL, 2, 1>
                       : k_int8_row_digits<DT, FULL, 4, 2>;
    const int t = n == 8 ? row_cta(cols, 4) : row_cta(cols, n);
    k<<<(unsigned)((rows + per - 1) / per), n == 8 && t > 512 ? 512 : t, 0, st>>>(Y, rows, (int)cols, cscale, planes, ld,
                                                                                steps, deep);
    QLORA_LAUNCH_CHECK();
    return QLORA_OK;
}

}  // namespace

int launch_int8_quantize(const void *X, int dtype, int64_t ldx, const int8_rows_t &q, uint32_t *d_status,
                         cudaStream_t st) {
    const int esize = dtype == QLORA_DTYPE_FP32 ? 4 : 2;
    const bool full = (reinterpret_cast<uintptr_t>(X) & 15u) == 0 && (ldx * esize) % 16 == 0 && q.cols % kVec == 0;
    auto *f = dtype == QLORA_DTYPE_BF16
                  ? (full ? launch_quantize<QLORA_DTYPE_BF16, true> : launch_quantize<QLORA_DTYPE_BF16, false>)
              : dtype == QLORA_DTYPE_FP16
                  ? (full ? launch_quantize<QLORA_DTYPE_FP16, true> : launch_quantize<QLORA_DTYPE_FP16, false>)
                  : (full ? launch_quantize<QLORA_DTYPE_FP32, true> : launch_quantize<QLORA_DTYPE_FP32, false>);
    return f(X, ldx, q, d_status, st);
}

int launch_int8_row_digits(const uint16_t *Y, bool f16, int64_t rows, int64_t cols, const float *cscale,
                           int8_t *planes, int64_t ld, float *steps, uint8_t *deep, cudaStream_t st) {
    const bool full = ((reinterpret_cast<uintptr_t>(Y) | reinterpret_cast<uintptr_t>(cscale)) & 15u) == 0 &&
                      cols % kVec == 0;
    auto *f = f16 ? (full ? launch_row_digits<QLORA_DTYPE_FP16, true> : launch_row_digits<QLORA_DTYPE_FP16, false>)
                  : (full ? launch_row_digits<QLORA_DTYPE_BF16, true> : launch_row_digits<QLORA_DTYPE_BF16, false>);
    return f(Y, rows, cols, cscale, planes, ld, steps, deep, st);
}

int launch_int8_col_digits(const void *S, int dtype, int64_t R, int r, const float *f, int8_t *planes, int64_t ld,
                           int rp, int rep, float *steps, cudaStream_t st) {
    const int64_t per = ((R + kColCluster - 1) / kColCluster + 15) / 16 * 16;
    const dim3 grid((unsigned)((rp + kColStrip - 1) / kColStrip), kColCluster);
    if (dtype == QLORA_DTYPE_FP32)
        k_int8_col_digits<QLORA_DTYPE_FP32><<<grid, kColThreads, 0, st>>>(S, R, r, f, per, planes, ld, rp, rep, steps);
    else if (dtype == QLORA_DTYPE_FP16)
        k_int8_col_digits<QLORA_DTYPE_FP16><<<grid, kColThreads, 0, st>>>(S, R, r, f, per, planes, ld, rp, rep, steps);
    else
        k_int8_col_digits<QLORA_DTYPE_BF16><<<grid, kColThreads, 0, st>>>(S, R, r, f, per, planes, ld, rp, rep, steps);
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
