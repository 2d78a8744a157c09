// int8_gemv.cu -- the product of a few tokens (M <= 4) with a weight of 8-bit
// rows, bound by the weight's bytes:
//
//   y[m][n] = (sum_k cx[m][k] cw[n][k]) * sx[m] * sw[n] + bias[n]
//
// A warp takes a row (short rows: two) at a time, its lanes 16 codes each of
// every 512; the tokens' codes lie in shared memory and four-way integer dot
// products (exact) do the sums.  Warp w of all takes rows w, w + warps, ...: one
// wave of CTAs whose rows differ by one at most.  Four CTAs an SM with eight
// loads a lane keep up to 128 KB in flight; a warp's first loads are issued
// before anything that depends on the tokens.
// FUSED: the CTA also quantizes the tokens itself (each CTA all of them: a few
// KB from L2), which saves a launch where the tokens are short; CTA 0 writes
// their codes and scales out.
#include "int8_rows.cuh"

namespace qlora {
namespace {

constexpr int kGThreads = 256, kGWarps = kGThreads / 32;
constexpr int kGBatch = 8;                 // 16-byte loads a lane has in flight

struct GemvParams {
    const int8_t *w;
    int64_t ldw, N;
    int K, M, kp;              // kp: K rounded up to whole steps (codes of a token in shared memory)
    const float *wscale;
    const void *x;             // FUSED: the tokens and their dtype
    int64_t ldx;
    int x_dtype;
    int8_t *codes;             // X8: read, or written when FUSED
    int64_t ldc;
    float *xscale;
    const void *bias;
    void *y;
    int dtype, pdl;
    uint32_t *status;
};

// Codes and scales of the M tokens into shared memory, by the whole CTA.
template <int DT, int MT>
__device__ __forceinline__ void quantize_tokens(const GemvParams &p, int8_t *xs, float *sx, uint32_t *part) {
    constexpr int esize = DT == QLORA_DTYPE_FP32 ? 4 : 2;
    const int nv = (p.K + kVec - 1) / kVec;
    uint32_t am[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        am[m] = 0;
        const char *row = static_cast<const char *>(p.x) + m * p.ldx * esize;
        if (m < p.M)
            for (int v = threadIdx.x; v < nv; v += kGThreads) am[m] = absmax8<DT>(load8<DT, false>(row, v, p.K), am[m]);
        am[m] = __reduce_max_sync(0xffffffffu, absmax_bits<DT>(am[m]));
        if ((threadIdx.x & 31) == 0) part[m * kGWarps + threadIdx.x / 32] = am[m];
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        if (m >= p.M) break;
        uint32_t b = 0;
#pragma unroll
        for (int i = 0; i < kGWarps; ++i) b = part[m * kGWarps + i] > b ? part[m * kGWarps + i] : b;
        const RowCode rc = row_code<DT>(b);
        if (threadIdx.x == 0) {
            sx[m] = rc.s;
            if (blockIdx.x == 0) {
                p.xscale[m] = rc.s;
                if (!rc.mask && p.status) atomicOr(p.status, QLORA_STATUS_NONFINITE);
            }
        }
        const char *row = static_cast<const char *>(p.x) + m * p.ldx * esize;
        int8_t *dst = xs + (int64_t)m * p.kp, *out = p.codes + m * p.ldc;
        float far = 0.f;
        for (int v = threadIdx.x; v < p.kp / kVec; v += kGThreads) {
            uint2 c = make_uint2(0u, 0u);
            if (v < nv) c = encode8<DT>(load8<DT, false>(row, v, p.K), rc, far);
            *reinterpret_cast<uint2 *>(dst + v * kVec) = c;
            if (blockIdx.x == 0 && v < nv) store8<false>(out, v * kVec, p.K, c.x, c.y);
        }
        if (rc.exact || far > kFar)
            encode_exact<DT>(row, threadIdx.x, kGThreads, p.K, rc.s, dst, blockIdx.x == 0 ? out : nullptr);
    }
}

// 16 codes of a row from value k on; codes past the row's K count as zero.
__device__ __forceinline__ uint4 load_codes(const int8_t *row, int k, int K) {
    if (k + 16 <= K) return __ldcg(reinterpret_cast<const uint4 *>(row + k));
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 16; ++e)
        if (k + e < K) w[e / 4] |= (uint32_t)(uint8_t)__ldcg(row + k + e) << (8 * (e & 3));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// RW * ST = kGBatch: rows at a time and 512-value steps of each in a batch.
template <int MT, int RW, bool FUSED>
__global__ void __launch_bounds__(kGThreads, 4)
k_int8_gemv(const GemvParams p) {
    constexpr int ST = kGBatch / RW;
    extern __shared__ __align__(16) int8_t xs[];     // [MT][kp]
    __shared__ float sx[MT];
    __shared__ uint32_t part[MT * kGWarps];
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * kGWarps;
    const int64_t w0 = (int64_t)blockIdx.x * kGWarps + threadIdx.x / 32;
    uint4 buf[RW][ST];
    auto load = [&](int64_t n, int s0) {
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            const int64_t row = n + i * warps;
            const int8_t *at = p.w + row * p.ldw;
#pragma unroll
            for (int j = 0; j < ST; ++j) {
                const int k = (s0 + j) * 512 + lane * 16;
                buf[i][j] = row < p.N && k < p.K ? load_codes(at, k, p.K) : make_uint4(0, 0, 0, 0);
            }
        }
    };
    load(w0, 0);
    if (FUSED) {
        if (p.x_dtype == QLORA_DTYPE_BF16) quantize_tokens<QLORA_DTYPE_BF16, MT>(p, xs, sx, part);
        else if (p.x_dtype == QLORA_DTYPE_FP16) quantize_tokens<QLORA_DTYPE_FP16, MT>(p, xs, sx, part);
        else quantize_tokens<QLORA_DTYPE_FP32, MT>(p, xs, sx, part);
    } else {
        if (p.pdl) asm volatile("griddepcontrol.wait;\n" ::: "memory");
        if (threadIdx.x < MT) sx[threadIdx.x] = (int)threadIdx.x < p.M ? __ldcg(p.xscale + threadIdx.x) : 0.f;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            if (m >= p.M) break;
            for (int k = threadIdx.x * 16; k < p.kp; k += kGThreads * 16)
                *reinterpret_cast<uint4 *>(xs + (int64_t)m * p.kp + k) =
                    k < p.K ? load_codes(p.codes + m * p.ldc, k, p.K) : make_uint4(0, 0, 0, 0);
        }
    }
    for (int m = p.M; m < MT; ++m)
        for (int k = threadIdx.x * 16; k < p.kp; k += kGThreads * 16)
            *reinterpret_cast<uint4 *>(xs + (int64_t)m * p.kp + k) = make_uint4(0, 0, 0, 0);
    __syncthreads();
    const int steps = p.kp / 512;
    bool loaded = true;
    for (int64_t n = w0; n < p.N; n += RW * warps) {
        int acc[RW][MT];
#pragma unroll
        for (int i = 0; i < RW; ++i)
#pragma unroll
            for (int m = 0; m < MT; ++m) acc[i][m] = 0;
        for (int s0 = 0; s0 < steps; s0 += ST) {
            if (!loaded) load(n, s0);
            loaded = false;
#pragma unroll
            for (int j = 0; j < ST; ++j) {
                if (s0 + j >= steps) break;
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const uint4 x =
                        *reinterpret_cast<const uint4 *>(xs + (int64_t)m * p.kp + (s0 + j) * 512 + lane * 16);
#pragma unroll
                    for (int i = 0; i < RW; ++i) {
                        acc[i][m] = __dp4a((int)buf[i][j].x, (int)x.x, acc[i][m]);
                        acc[i][m] = __dp4a((int)buf[i][j].y, (int)x.y, acc[i][m]);
                        acc[i][m] = __dp4a((int)buf[i][j].z, (int)x.z, acc[i][m]);
                        acc[i][m] = __dp4a((int)buf[i][j].w, (int)x.w, acc[i][m]);
                    }
                }
            }
        }
        int mine = 0;
#pragma unroll
        for (int i = 0; i < RW; ++i)
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const int t = __reduce_add_sync(0xffffffffu, acc[i][m]);
                if (lane == i * MT + m) mine = t;
            }
        const int m = lane % MT;
        const int64_t row = n + (lane / MT) * warps;
        if (lane < RW * MT && m < p.M && row < p.N) {
            const float bs = p.bias ? load_any(p.bias, row, p.dtype) : 0.f;
            const float v = __fmaf_rn(__fmul_rn(sum_float((uint32_t)mine), sx[m]), __ldg(p.wscale + row), bs);
            const int64_t at = m * p.N + row;
            if (p.dtype == QLORA_DTYPE_FP32) static_cast<float *>(p.y)[at] = v;
            else static_cast<uint16_t *>(p.y)[at] = enc16(v, p.dtype == QLORA_DTYPE_FP16);
        }
    }
}

template <int MT, int RW>
int launch_gemv(const GemvParams &p, bool fused, cudaStream_t st) {
    const int smem = MT * p.kp;
    void (*k)(GemvParams) = fused ? k_int8_gemv<MT, RW, true> : k_int8_gemv<MT, RW, false>;
    if (set_max_smem(reinterpret_cast<const void *>(k), smem) != cudaSuccess) return QLORA_ECUDA;
    const int64_t want = (p.N + kGWarps * RW - 1) / (kGWarps * RW), most = 4 * device_sms();
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(want < most ? want : most));
    cfg.blockDim = dim3(kGThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.pdl ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, k, p) != cudaSuccess) return QLORA_ECUDA;
    QLORA_LAUNCH_CHECK();
    return QLORA_OK;
}

template <int MT>
int pick_rows(const GemvParams &p, bool fused, cudaStream_t st) {
    if (p.kp <= 2048) return launch_gemv<MT, 2>(p, fused, st);   // a batch of 4 steps holds a row: two rows at a time
    return launch_gemv<MT, 1>(p, fused, st);
}

}  // namespace

// Against the tall kernel at 16 tokens (one MMA width serves them all): one and
// two tokens are faster here at every size (rows given, cold weights, 4096 x 4096:
// 5.5 and 6.2 us, there 8.0; 8192 x 28672: 37.9 and 38.6, there 41.7), three and four
// on small weights alone (1024 x 1024: 3.6, there 4.9; 4096 x 11008: 15.6, there 11.4).
bool int8_gemv_takes(int64_t M, int64_t N, int64_t K) {
    return M * ((K + 511) / 512 * 512) <= kGemvTokenBytes && (M <= 2 || (M <= 4 && N * K <= (int64_t)8 << 20));
}

int launch_int8_gemv(const void *X, int x_dtype, int64_t ldx, const int8_rows_t &X8, const int8_rows_t &W,
                     const void *bias, void *Y, int dtype, uint32_t *d_status, cudaStream_t st) {
    const int M = (int)X8.rows;
    // quantizing in every CTA costs about 0.5 us for 2048 values, a launch of its own 1 us (and the host's 2)
    const bool fused = X && M * W.cols <= 4096;
    if (X && !fused) {
        const int rc = launch_int8_quantize(X, x_dtype, ldx, X8, d_status, st);
        if (rc) return rc;
    }
    GemvParams p{};
    p.w = W.codes, p.ldw = W.ld, p.N = W.rows;
    p.K = (int)W.cols, p.M = M;
    p.kp = (int)((W.cols + 511) / 512 * 512);
    p.wscale = W.scales;
    p.x = X, p.ldx = ldx, p.x_dtype = x_dtype;
    p.codes = X8.codes, p.ldc = X8.ld, p.xscale = X8.scales;
    p.bias = bias, p.y = Y, p.dtype = dtype;
    p.pdl = X && !fused;
    p.status = d_status;
    if (M == 1) return pick_rows<1>(p, fused, st);
    if (M == 2) return pick_rows<2>(p, fused, st);
    return pick_rows<4>(p, fused, st);
}

}  // namespace qlora
