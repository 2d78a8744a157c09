// int8_rows.cuh -- device helpers of the 8-bit row codec: loads of eight
// values, row maxima and the decision of a code (int8_rows.cu, int8_gemv.cu).
#pragma once
#include "int8_gemm.cuh"

namespace qlora {
namespace {

constexpr int kVec = 8;           // values per thread and step
constexpr float kMagic = 12582912.f;   // 1.5 * 2^23: adding it rounds to an integer, ties to even

// Eight consecutive values of a row as they were loaded.
template <int DT>
struct Raw8 {
    uint32_t w[DT == QLORA_DTYPE_FP32 ? 8 : 4];
};

// The 8 values that start off bytes into a run of words.
template <int DT>
__device__ __forceinline__ void shift8(const uint32_t *in, uint32_t off, Raw8<DT> &r) {
    constexpr int kWords = sizeof(r.w) / 4;
    uint32_t t[kWords + 1];
#pragma unroll
    for (int i = 0; i < kWords + 1; ++i) {
        t[i] = in[i];
        if (off >= 4 && i + 1 < kWords + 4) t[i] = in[i + 1];
        if (off >= 8 && i + 2 < kWords + 4) t[i] = in[i + 2];
        if (off >= 12 && i + 3 < kWords + 4) t[i] = in[i + 3];
    }
#pragma unroll
    for (int i = 0; i < kWords; ++i)
        r.w[i] = DT == QLORA_DTYPE_FP32 ? t[i] : __funnelshift_r(t[i], t[i + 1], 8 * (off & 3u));
}

// Values [8 v, 8 v + 8) of a row, zeros past its end.  FULL: rows start on
// 16-byte borders and hold a multiple of 8 values.  Otherwise a row that starts
// off a border is read in the aligned pieces around the values, where all lie
// inside the row, and shifted into place; what is left, at the
// row's ends, comes value by value (the addresses clamped, so that the eight
// loads do not wait for one another).
template <int DT, bool FULL>
__device__ __forceinline__ Raw8<DT> load8(const void *row, int v, int cols) {
    Raw8<DT> r;
    constexpr int kWords = sizeof(r.w) / 4;
    constexpr int kSize = kWords / 2;      // bytes a value
    const int e0 = v * kVec;
    const char *at = static_cast<const char *>(row) + (int64_t)e0 * kSize;
    const uint32_t off = FULL ? 0u : (uint32_t)(reinterpret_cast<uintptr_t>(row) & 15u);
    if (FULL || (off == 0 && e0 + kVec <= cols)) {
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) {
            const uint4 t = __ldg(reinterpret_cast<const uint4 *>(at) + i);
            r.w[4 * i] = t.x, r.w[4 * i + 1] = t.y, r.w[4 * i + 2] = t.z, r.w[4 * i + 3] = t.w;
        }
        return r;
    }
    if (v > 0 && e0 + kVec + 16 / kSize <= cols) {
        uint32_t in[kWords + 4];
#pragma unroll
        for (int i = 0; i < kWords / 4 + 1; ++i) {
            const uint4 x = __ldg(reinterpret_cast<const uint4 *>(at - off) + i);
            in[4 * i] = x.x, in[4 * i + 1] = x.y, in[4 * i + 2] = x.z, in[4 * i + 3] = x.w;
        }
        shift8<DT>(in, off, r);
        return r;
    }
    uint32_t one[kVec];
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
        const int i = e0 + e < cols ? e0 + e : cols - 1;
        one[e] = DT == QLORA_DTYPE_FP32 ? __ldg(static_cast<const uint32_t *>(row) + i)
                                        : (uint32_t)__ldg(static_cast<const uint16_t *>(row) + i);
    }
#pragma unroll
    for (int e = 0; e < kVec; ++e) one[e] = e0 + e < cols ? one[e] : 0u;
#pragma unroll
    for (int i = 0; i < kWords; ++i)
        r.w[i] = DT == QLORA_DTYPE_FP32 ? one[i % kVec] : one[2 * i % kVec] | (one[(2 * i + 1) % kVec] << 16);
    return r;
}

// A row as the whole vectors [v0, v1) whose (aligned) pieces lie inside it and
// `edges` <= 32 values around them, one a thread: so no load of a vector waits in
// a branch for another (bf16 of 8192 x 8191, rows on 16-byte borders: 32 us, with
// the ends among the vectors 41).
struct RowSpan {
    int v0, v1, edges;
    __device__ __forceinline__ int edge(int i) const { return i < v0 * kVec ? i : i + (v1 - v0) * kVec; }
};
template <int DT, bool FULL>
__device__ __forceinline__ RowSpan row_span(uint32_t off, int cols) {
    if (FULL) return RowSpan{0, cols / kVec, 0};
    constexpr int size = DT == QLORA_DTYPE_FP32 ? 4 : 2;
    RowSpan r{0, cols / kVec, 0};
    if (off) r.v0 = 1, r.v1 = (cols - (int)(16 - off) / size) / kVec;
    if (r.v1 <= r.v0) r.v0 = r.v1 = 0;
    r.edges = cols - (r.v1 - r.v0) * kVec;
    return r;
}
template <bool FULL>
__device__ __forceinline__ uint32_t row_offset(const void *row) {
    return FULL ? 0u : (uint32_t)(reinterpret_cast<uintptr_t>(row) & 15u);
}
template <int DT>
__device__ __forceinline__ Raw8<DT> edge8(const void *row, int e) {   // value e, then zeros
    Raw8<DT> r{};
    r.w[0] = DT == QLORA_DTYPE_FP32 ? __ldg(static_cast<const uint32_t *>(row) + e)
                                    : (uint32_t)__ldg(static_cast<const uint16_t *>(row) + e);
    return r;
}
// Vectors v, v + stride, .. of a row whose start lies off bytes past a border.
// Shifted ones are loaded four at a time: 8192 x 8192 in rows of 8196 take 33 us,
// two at a time 36, eight at a time (104 registers) 39, one by one 46.
constexpr int kShiftGroup = 4;
template <int DT, bool FULL, int STEPS>
__device__ __forceinline__ void load_steps(const char *row, uint32_t off, int v, int stride, int v1, Raw8<DT> *to) {
    if (FULL || off == 0) {
#pragma unroll
        for (int i = 0; i < STEPS; ++i)
            if (v + i * stride < v1) to[i] = load8<DT, true>(row, v + i * stride, 0);
        return;
    }
    constexpr int kWords = sizeof(Raw8<DT>) / 4, kGroup = STEPS < kShiftGroup ? STEPS : kShiftGroup;
#pragma unroll
    for (int g = 0; g < STEPS; g += kGroup) {
        uint32_t w[kGroup][kWords + 4];
#pragma unroll
        for (int i = 0; i < kGroup; ++i)
            if (v + (g + i) * stride < v1) {
                const uint4 *at = reinterpret_cast<const uint4 *>(row + (int64_t)(v + (g + i) * stride) * (kWords * 4) - off);
#pragma unroll
                for (int j = 0; j < kWords / 4 + 1; ++j) {
                    const uint4 t = __ldg(at + j);
                    w[i][4 * j] = t.x, w[i][4 * j + 1] = t.y, w[i][4 * j + 2] = t.z, w[i][4 * j + 3] = t.w;
                }
            }
#pragma unroll
        for (int i = 0; i < kGroup; ++i) shift8<DT>(w[i], off, to[g + i]);
    }
}

template <int DT>
__device__ __forceinline__ float val8(const Raw8<DT> &r, int e) {
    if (DT == QLORA_DTYPE_FP32) return __uint_as_float(r.w[e % (sizeof(r.w) / 4)]);
    const uint32_t w = r.w[e / 2];
    return (e & 1) ? hi16(w, DT == QLORA_DTYPE_FP16) : lo16(w, DT == QLORA_DTYPE_FP16);
}

// Running maximum of the magnitudes' bit patterns (two 16-bit patterns a word,
// or one of fp32): they order as the magnitudes do, infinities and NaNs above
// every finite value.
template <int DT>
__device__ __forceinline__ uint32_t absmax8(const Raw8<DT> &r, uint32_t m) {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(r.w) / 4); ++i) {
        if (DT == QLORA_DTYPE_FP32) {
            const uint32_t b = r.w[i] & 0x7fffffffu;
            m = b > m ? b : m;
        } else {
            m = __vmaxu2(m, r.w[i] & 0x7fff7fffu);
        }
    }
    return m;
}
// The maximum as fp32 bits.
template <int DT>
__device__ __forceinline__ uint32_t absmax_bits(uint32_t m) {
    if (DT == QLORA_DTYPE_FP32) return m;
    const uint32_t a = m & 0xffffu, b = m >> 16;
    return __float_as_uint(dec16((uint16_t)(a > b ? a : b), DT == QLORA_DTYPE_FP16));
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

// Store 8 code bytes at element e0 of a row (16-byte aligned start).
template <bool FULL>
__device__ __forceinline__ void store8(int8_t *row, int e0, int cols, uint32_t lo, uint32_t hi) {
    if (FULL || e0 + kVec <= cols) {
        *reinterpret_cast<uint2 *>(row + e0) = make_uint2(lo, hi);
        return;
    }
    for (int e = 0; e < kVec && e0 + e < cols; ++e)
        row[e0 + e] = (int8_t)(uint8_t)((e < 4 ? lo >> (8 * e) : hi >> (8 * (e - 4))) & 255u);
}

__device__ __forceinline__ uint32_t bytes4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// How a row's codes are decided: fma(x, inv, magic) rounds x * inv to the
// nearest integer in its low bits, with inv chosen for the row.
//   16 bits: x and a have at most 11 significant bits, so the quotient by the
// unrounded a / 127 either lies on a border between two codes or differs from
// it by at least 1 / (254 * 2^11) > 2^-19 of itself.  Only border values need
// the direction in which s was rounded, and a reciprocal moved by 2^-21 of
// itself that way decides them: the other codes keep their side, as
// 2^-21 + 3 * 2^-24 < 2^-19.  Where s = a / 127 exactly, a power of two has an
// exact reciprocal (true ties, to even); other scales (0.7% of fp16 rows, no
// bf16 one) take code_exact.
//   fp32: inv = RN(1/s) puts the quotient at most 127 * 2^-23 < 1.6e-5 off, so a
// code is decided unless the quotient lies within 2e-5 of a border; a thread
// that met such a one (`far`) does its part again by code_exact.
//   1/s near the ends of fp32's range: code_exact.
// Rows whose codes are all 0 (s = 0, or a NaN or an infinity in them): inv = 0
// and a mask, since a NaN has no code.
struct RowCode {
    float s, inv;
    uint32_t mask;
    bool exact;
};

template <int DT>
__device__ __forceinline__ RowCode row_code(uint32_t am) {
    RowCode r;
    const bool fin = am < 0x7f800000u;
    const float a = __uint_as_float(am);
    r.s = fin ? __fdiv_rn(a, 127.f) : __uint_as_float(0x7fffffffu);
    r.mask = fin ? 0xffffffffu : 0u;
    r.inv = 0.f;
    r.exact = false;
    if (!fin || r.s == 0.f) return r;
    if (r.s < 0x1p-120f) {
        r.exact = true;
        return r;
    }
    r.inv = __frcp_rn(r.s);
    if (DT == QLORA_DTYPE_FP32) return r;
    const float over = __fmaf_rn(r.s, 127.f, -a);   // > 0: s was rounded up
    if (over == 0.f) r.exact = (__float_as_uint(r.s) & 0x7fffffu) != 0;
    else r.inv = __fmaf_rn(over > 0.f ? -0x1p-21f : 0x1p-21f, r.inv, r.inv);
    return r;
}

template <int DT>
__device__ __forceinline__ uint2 encode8(const Raw8<DT> &r, const RowCode &rc, float &far) {
    uint32_t c[kVec];
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
        const float x = val8(r, e);
        const float t = __fmaf_rn(x, rc.inv, kMagic);
        c[e] = __float_as_uint(t);
        if (DT == QLORA_DTYPE_FP32) far = fmaxf(far, fabsf(__fmaf_rn(x, rc.inv, -(t - kMagic))));
    }
    return make_uint2(bytes4(c[0], c[1], c[2], c[3]) & rc.mask, bytes4(c[4], c[5], c[6], c[7]) & rc.mask);
}
constexpr float kFar = 0.49998f;

// Code of x by division.  fp16 (s = a / 127 exactly): a rounded fp32 quotient
// is on a border only if the quotient is.  Else in fp64, where the quotient of
// two numbers of 24 bits is never within 2^-33 (relative) of a border without
// lying on it.
template <int DT>
__device__ __forceinline__ int code_exact(float x, float s) {
    if (DT == QLORA_DTYPE_FP16) return __float2int_rn(__fdiv_rn(x, s));
    const double q = (double)x / (double)s;
    return __double2int_rn(q > 127.0 ? 127.0 : (q < -127.0 ? -127.0 : q));
}

// A thread's part of a row (vectors v0, v0 + stride, ...) by code_exact, to dst
// and, if it is not NULL, to also.  Out of line: few rows come here.
template <int DT>
__device__ __noinline__ void encode_exact(const void *row, int v0, int stride, int cols, float s, int8_t *dst,
                                          int8_t *also) {
#pragma unroll 1
    for (int v = v0; v * kVec < cols; v += stride) {
        const Raw8<DT> r = load8<DT, false>(row, v, cols);
        uint32_t c[kVec];
#pragma unroll
        for (int e = 0; e < kVec; ++e) c[e] = (uint32_t)code_exact<DT>(val8(r, e), s);
        const uint32_t lo = bytes4(c[0], c[1], c[2], c[3]), hi = bytes4(c[4], c[5], c[6], c[7]);
        store8<false>(dst, v * kVec, cols, lo, hi);
        if (also) store8<false>(also, v * kVec, cols, lo, hi);
    }
}

}  // namespace
}  // namespace qlora
