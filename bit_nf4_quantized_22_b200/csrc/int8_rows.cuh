// int8_rows.cuh -- device helpers of the 8-bit row codec: loads of eight
// values, row maxima and the decision of a code (int8_rows.cu, int8_gemv.cu).
#pragma once
#include "int8_gemm.cuh"

namespace qlora {
namespace {

constexpr int kVec = 8;           // values per thread and step
constexpr float kMagic = 12582912.f;   // 1.5 * 2^23: adding it rounds to an integer, ties to even
// steps whose values stay in registers between the maximum and the codes
template <int DT> constexpr int kKeep = DT == QLORA_DTYPE_FP32 ? 2 : 4;

// Eight consecutive values of a row as they were loaded.
template <int DT>
struct Raw8 {
    uint32_t w[DT == QLORA_DTYPE_FP32 ? 8 : 4];
};

// Values [8 v, 8 v + 8) of a row, zeros past its end.  A 16-bit row that starts
// off a 16-byte border is read in the two aligned pieces around the values,
// where both lie inside the row, and shifted into place.
template <int DT>
__device__ __forceinline__ Raw8<DT> load8(const void *row, int v, int cols) {
    Raw8<DT> r;
    constexpr int kWords = sizeof(r.w) / 4;
    constexpr int kSize = kWords / 2;      // bytes a value
    const int e0 = v * kVec;
    const char *at = static_cast<const char *>(row) + (int64_t)e0 * kSize;
    const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(row) & 15u);
    if (off == 0 && e0 + kVec <= cols) {
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) {
            const uint4 t = __ldg(reinterpret_cast<const uint4 *>(at) + i);
            r.w[4 * i] = t.x, r.w[4 * i + 1] = t.y, r.w[4 * i + 2] = t.z, r.w[4 * i + 3] = t.w;
        }
        return r;
    }
    if (DT != QLORA_DTYPE_FP32 && v > 0 && e0 + 2 * kVec <= cols) {
        const uint4 x = __ldg(reinterpret_cast<const uint4 *>(at - off));
        const uint4 y = __ldg(reinterpret_cast<const uint4 *>(at - off) + 1);
        const uint32_t in[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
        uint32_t t[5];
#pragma unroll
        for (int i = 0; i < 5; ++i) {
            t[i] = in[i];
            if (off >= 4 && i + 1 < 8) t[i] = in[i + 1];
            if (off >= 8 && i + 2 < 8) t[i] = in[i + 2];
            if (off >= 12 && i + 3 < 8) t[i] = in[i + 3];
        }
#pragma unroll
        for (int i = 0; i < kWords; ++i) r.w[i] = __funnelshift_r(t[i % 4], t[i % 4 + 1], 8 * (off & 3u));
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

// Code of x exactly: the quotient in fp64 is never within 2^-33 (relative) of
// a border between two codes without lying on it, since x and s have 24 bits.
__device__ __noinline__ int code_exact(float x, float s) {
    const double q = (double)x / (double)s;
    const int c = __double2int_rn(q > 127.0 ? 127.0 : (q < -127.0 ? -127.0 : q));
    return c;
}

// Store 8 code bytes at element e0 of a row (16-byte aligned start).
__device__ __forceinline__ void store8(int8_t *row, int e0, int cols, uint32_t lo, uint32_t hi) {
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

// How a row's codes are decided.
//   fp32: fma(x, 1/s, magic) rounds x * RN(1/s) to the nearest integer in its
// low bits.  The rounded reciprocal puts the quotient at most 127 * 2^-23 off,
// so a code is decided unless the quotient lies within 1e-4 of a border, where
// code_exact decides (kNear).
//   16 bits: x and a have at most 11 significant bits, so the quotient by the
// unrounded a / 127 either lies on a border or differs from it by at least
// 1 / (254 * 2^11) > 2^-19 of itself.  Only border values need the direction
// in which s was rounded, and a reciprocal moved by 2^-21 of itself that way
// decides them: the other codes keep their side, 2^-21 + 3 * 2^-24 < 2^-19
// (kSure).  Where s = a / 127 exactly, a power of two has an exact reciprocal
// (true ties, to even), and other scales take the fp32 way.
//   1/s near the ends of fp32's range: every code by code_exact (kExact).
enum Decide { kSure, kNear, kExact };

template <int DT>
__device__ __forceinline__ Decide decide(float a, float s, float &inv) {
    inv = 0.f;
    if (s < 0x1p-120f) return kExact;
    inv = __frcp_rn(s);
    if (DT == QLORA_DTYPE_FP32) return kNear;
    const float over = __fmaf_rn(s, 127.f, -a);   // > 0: s was rounded up
    if (over == 0.f) return (__float_as_uint(s) & 0x7fffffu) == 0 ? kSure : kNear;
    inv = __fmaf_rn(over > 0.f ? -0x1p-21f : 0x1p-21f, inv, inv);
    return kSure;
}

template <int DT>
__device__ __forceinline__ uint2 encode8(const Raw8<DT> &r, float s, float inv, Decide how) {
    uint32_t c[kVec];
    if (how == kSure) {
#pragma unroll
        for (int e = 0; e < kVec; e += 2) {
            float t0, t1;
            fma2_rn(inv, val8(r, e), val8(r, e + 1), kMagic, kMagic, t0, t1);
            c[e] = __float_as_uint(t0), c[e + 1] = __float_as_uint(t1);
        }
    } else {
        float far = how == kExact ? 1.f : 0.f;
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            const float x = val8(r, e);
            const float t = __fmaf_rn(x, inv, kMagic);
            c[e] = __float_as_uint(t);
            far = fmaxf(far, fabsf(__fmaf_rn(x, inv, -(t - kMagic))));
        }
        if (far > 0.4999f) {
#pragma unroll
            for (int e = 0; e < kVec; ++e) c[e] = (uint32_t)code_exact(val8(r, e), s);
        }
    }
    return make_uint2(bytes4(c[0], c[1], c[2], c[3]), bytes4(c[4], c[5], c[6], c[7]));
}

}  // namespace
}  // namespace qlora
