// int8_gemm.cu -- products of int8 operands on the 5th-gen tensor cores
// (tcgen05 kind::i8, exact int32 sums in TMEM).
//
//   acc_d(p, q) = sum_t A(p, t) * B_d(q, t),      d = 0 .. planes - 1
//   out(p, q)   = (sum_d 256^(planes-1-d) acc_d(p, q)) * qscale[q] * pscale[p] + bias[p]
//
// A, the tall operand, is read in place, K-major (the reduction t contiguous)
// or MN-major (p contiguous); B holds `planes` signed base-256 digits of the
// other operand (int8_rows.cu), K-major.  The products built on it:
//   y  = x . W^T        p = output channel, q = token, A = W's codes, 1 plane
//   dX = dY . W         p = input feature,  q = token, A = W's codes (MN-major), 2 planes,
//                       4 for the tokens whose digits need them
//   T  = u . A          p = token, q = rank column, A = u's codes, 3 planes
//   dA = u^T . G        p = input feature, q = rank column, A = u's codes (MN-major), 3 planes
#include <cuda.h>
#include <cudaTypedefs.h>

#include <type_traits>

#include "int8_gemm.cuh"
#include "tcgen05_epilogue.cuh"

namespace qlora {
namespace {
using namespace tc;

constexpr int kTK = 128;                       // reduction values (bytes) per k-tile: one swizzle row
constexpr int kTP = 128;                       // rows of A per tile = TMEM lanes
constexpr int kTABytes = kTP * kTK;            // 16 KB
constexpr int kTThreads = 192;
constexpr int kTMaxStages = 8;
constexpr int kTMaxSplits = 8;                 // portable cluster size
constexpr int kTTwoN = 128;                    // UMMA N up to which two CTAs share an SM
constexpr int kTSmemTwo = 110 * 1024;
constexpr int kTSmemOne = 220 * 1024;

// 256 * (a rounded upper sum) + the lower sum, in fp32: off by 2^-23 of the larger of the two terms
__device__ __forceinline__ float join_digits(float upper, float lower) { return __fmaf_rn(upper, 256.f, lower); }
// The same of the joined upper and lower pair of four digits.
__device__ __forceinline__ float join_pairs(float upper, float lower) { return __fmaf_rn(upper, 65536.f, lower); }

// kind::i8 instruction descriptor: signed 8-bit A and B, s32 accumulator.
__host__ __device__ constexpr uint32_t idesc_i8(uint32_t m, uint32_t n, uint32_t a_mn, uint32_t b_mn) {
    return (2u << 4) | (1u << 7) | (1u << 10) | (a_mn << 15) | (b_mn << 16) | ((n >> 3) << 17) | ((m >> 4) << 24);
}
// The warp's index and its elected lane, in forms that the compiler knows to be
// the same for all lanes: the MMAs' descriptors then stay in uniform registers.
// (Issued from inside `if (lane == 0)` each MMA took some 175 cycles whatever
// its size, which bounded both kernels below.)
__device__ __forceinline__ int warp_index() { return __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0); }
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(e));
    return e != 0;
}
// One k-tile of 128 reduction values: four MMAs, by one elected lane of a
// converged warp; the first adds to the accumulator only if acc.
__device__ __forceinline__ void umma_i8_ktile(uint32_t d_tmem, uint64_t a, uint64_t b, uint64_t astep, uint64_t bstep,
                                              uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred e, p, q;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %10, 0;\n\t"
        "setp.eq.b32 q, %10, %10;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %9, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::i8 [%0], %3, %4, %9, q;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::i8 [%0], %5, %6, %9, q;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::i8 [%0], %7, %8, %9, q;\n\t}\n" ::"r"(d_tmem),
        "l"(a), "l"(b), "l"(a + astep), "l"(b + bstep), "l"(a + 2 * astep), "l"(b + 2 * bstep), "l"(a + 3 * astep),
        "l"(b + 3 * bstep), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void umma_commit_elect(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(bar)
        : "memory");
}
// 32 TMEM columns without the wait, and the wait for all loads before it, which
// the values pass through so that nothing reads them earlier.
__device__ __forceinline__ void tmem_ld32_issue(uint32_t taddr, uint32_t *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr));
}
#define QLORA_TIE16(v, o)                                                                                          \
    "+r"((v)[o]), "+r"((v)[(o) + 1]), "+r"((v)[(o) + 2]), "+r"((v)[(o) + 3]), "+r"((v)[(o) + 4]),                  \
        "+r"((v)[(o) + 5]), "+r"((v)[(o) + 6]), "+r"((v)[(o) + 7]), "+r"((v)[(o) + 8]), "+r"((v)[(o) + 9]),        \
        "+r"((v)[(o) + 10]), "+r"((v)[(o) + 11]), "+r"((v)[(o) + 12]), "+r"((v)[(o) + 13]), "+r"((v)[(o) + 14]),   \
        "+r"((v)[(o) + 15])
template <int N>
__device__ __forceinline__ void tmem_wait(uint32_t (&v)[N]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
#pragma unroll
    for (int o = 0; o < N; o += 16) asm volatile("" : QLORA_TIE16(v, o));
}
#undef QLORA_TIE16
__device__ __forceinline__ uint4 ld_cluster_uint4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared::cluster.v4.u32 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr));
    return v;
}

struct TallParams {
    int64_t P, Q;
    int planes, nt;        // B rows per plane and tile; UMMA N = planes * nt
    int64_t plane_rows;    // rows from one plane of B to the next
    int nk, per;           // k-tiles, and per split
    int a_mn;              // A is MN-major
    int stages;
    uint32_t stage_bytes, tmem_cols;
    const float *qscale, *pscale;
    float mul;
    const void *bias;      // per p, in the output's dtype
    void *out;
    int64_t ldo;
    int q_inner;           // out[p * ldo + q], else out[q * ldo + p]
    int pool;              // q_inner: the 64 rows of each group summed
    int dtype, vec;
    int pdl;               // B and the scales come from the kernel before (programmatic launch)
    const uint8_t *deep;   // planes == 4: the columns q with all of them; the others have two (the first ones)
    int64_t tiles_q;       // DEEP: tiles of columns
    uint32_t *status;
};

// Is any of flags[at .. at + n) set?  All threads of the CTA; the first form for all Q columns.
__device__ __forceinline__ bool any_deep(const uint8_t *flags, int64_t Q) {
    uint32_t any = 0;
    const int64_t whole = Q / 16;
    for (int64_t i = threadIdx.x; i < whole; i += kTThreads) {
        const uint4 v = __ldcg(reinterpret_cast<const uint4 *>(flags) + i);
        any |= v.x | v.y | v.z | v.w;
    }
    if (threadIdx.x < Q % 16) any |= __ldcg(flags + whole * 16 + threadIdx.x);
    return __syncthreads_or((int)any) != 0;
}
__device__ __forceinline__ bool any_deep(const uint8_t *flags, int64_t at, int n, int64_t Q) {
    const int64_t q = at + threadIdx.x;
    return __syncthreads_or((int)threadIdx.x < n && q < Q ? (int)__ldcg(flags + q) : 0) != 0;   // n <= 64
}

// CTA (x, y, z): rows [128 x, +128) of A, rows [nt y, +nt) of each plane of B,
// k-tiles [per z, +per).  Warp 0 loads by TMA into a ring of stages, warp 1
// issues the MMAs, all warps share the epilogue.  The CTAs of a cluster (all
// z) hold the splits of one tile: each leaves its int32 sums in its own shared
// memory and finishes every gridDim.z-th column, reading its peers' sums over
// distributed shared memory -- integer sums, so the split changes no result.
// For few tokens it is bound by the weight's bytes (16 on 8192 x 28672: 41.8 us,
// 5.6 TB/s), for some by what an SM takes in (an MMA of M = 128 rows re-reads
// its A for every tile of columns): 256 on 4096 x 4096 take 13 us, 1024 take 27.
//
// DEEP: the second launch of an input gradient, for the tiles with a token of
// four planes among them.  It leaves at once where there is none; else CTA y takes
// tiles y, y + gridDim.y, .. and stores those tokens' columns alone.  Its ring
// and accumulator run on from tile to tile (512 x 4096 x 32000, 115 us for two
// planes: none 2.7 us, one token 37, all 269, most of it the exchange of sums).
// FOUR: all tokens with four planes, in one launch. Both are kernels of their own: their
// columns' registers (188 for 126) would leave one CTA an SM to every product.
template <bool FOUR, bool DEEP>
__global__ void __launch_bounds__(kTThreads)
k_int8_tall(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const TallParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t *gen_base = smem_raw + (base - raw_addr);
    const int S = p.stages;
    const uint32_t bar0 = base + S * p.stage_bytes;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (kTMaxStages + s); };
    const uint32_t acc_bar = bar0 + 8u * (2 * kTMaxStages);
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(gen_base + S * p.stage_bytes + 160);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(gen_base + S * p.stage_bytes + 192);
    float *qs = reinterpret_cast<float *>(gen_base + S * p.stage_bytes + 256);   // [nt <= 256]
    float *qdeep = qs + 64;                        // planes == 4, nt <= 64: columns with all of them

    if (DEEP && !any_deep(p.deep, p.Q)) return;    // the same for all CTAs
    const int warp = warp_index(), lane = threadIdx.x & 31;
    const int64_t p0 = (int64_t)blockIdx.x * kTP;
    int64_t q0 = (int64_t)blockIdx.y * p.nt;
    const int kbeg = blockIdx.z * p.per;
    const int kend = kbeg + p.per < p.nk ? kbeg + p.per : p.nk;
    const int nloc = kend - kbeg;                  // >= 1 by construction
    const int N = p.planes * p.nt;
    const uint32_t rank = blockIdx.z, splits = gridDim.z;

    bool ok = true;
    const int head = DEEP ? 0 : nloc < S ? nloc : S;   // k-tiles that find their stage free, loaded ahead
    // tile i of this CTA into stage s
    auto load_a = [&](int i, int s) {
        const uint32_t sa = base + s * p.stage_bytes;
        const int t0 = (kbeg + i) * kTK;
        mbar_expect_tx(full_bar(s), p.stage_bytes);
        if (p.a_mn) tma_load_2d(sa, &tmA, (int)p0, t0, full_bar(s));
        else tma_load_2d(sa, &tmA, t0, (int)p0, full_bar(s));
    };
    auto load_b = [&](int i, int s) {
        const uint32_t sb = base + s * p.stage_bytes + kTABytes;
        const int t0 = (kbeg + i) * kTK;
        for (int d = 0; d < p.planes; ++d)
            tma_load_2d(sb + d * p.nt * kTK, &tmB, t0, (int)(d * p.plane_rows + q0), full_bar(s));
    };
    const bool leader = elect_one();               // one lane of each warp
    if (warp == 0 && leader) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        mbar_init(acc_bar, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
        fence_proxy_async();
        // A fills the ring at once; with pdl it is all that does not depend on the kernel before
        for (int i = 0; i < head; ++i) load_a(i, i);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(tmem_holder)),
                     "r"(p.tmem_cols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
    }
    if (warp == 0 && leader) {
        if (p.pdl) asm volatile("griddepcontrol.wait;\n" ::: "memory");
        for (int i = 0; i < head; ++i) load_b(i, i);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;

    // stage and round of the ring: of the loads in warp 0, of the MMAs in warp 1
    int s = warp == 0 ? head % S : 0;
    uint32_t round = warp == 0 && head == S ? 1u : 0u;
    uint32_t tile = 0;                             // tiles before this one
#pragma unroll 1
    for (int64_t y = blockIdx.y; !DEEP || y < p.tiles_q; y += gridDim.y) {
        if (DEEP) {
            q0 = y * p.nt;
            if (!any_deep(p.deep, q0, p.nt, p.Q)) continue;   // the same for all CTAs of the cluster
        }
        if (warp == 0) {
            if (leader) {
                for (int i = head; i < nloc && ok; ++i) {
                    if (!DEEP || round > 0) ok = mbar_wait(empty_bar(s), (round & 1) ^ 1, abort_flag);
                    if (!ok) break;
                    load_a(i, s);
                    load_b(i, s);
                    if (++s == S) s = 0, ++round;
                }
                if (!ok) *abort_flag = 1;
            }
        } else if (warp == 1) {
            const uint32_t idesc = idesc_i8(kTP, (uint32_t)N, p.a_mn ? 1u : 0u, 0u);
            // K-major: rows of 128 t, 8-row groups 1 KB apart, a step of 32 t
            // advances 32 B.  MN-major: rows of 128 p, 8 t a 1 KB group, a step
            // of 32 t advances 4 KB (one 128-wide atom, so no leading stride).
            const uint64_t astep = p.a_mn ? 256u : 2u;
            const uint64_t bdiff = kTABytes >> 4, sdiff = p.stage_bytes >> 4;
            uint64_t ad = sdesc(base, 16, 1024) + s * sdiff;
            for (int i = 0; i < nloc && ok; ++i) {
                ok = __all_sync(0xffffffffu, mbar_wait(full_bar(s), round & 1, abort_flag));   // the warp stays together
                if (!ok) break;
                tc_fence_after();
                umma_i8_ktile(tmem, ad, ad + bdiff, astep, 2, idesc, i > 0 ? 1u : 0u);
                umma_commit_elect(empty_bar(s));
                ad += sdiff;
                if (++s == S) s = 0, ++round, ad = sdesc(base, 16, 1024);
            }
            if (ok) umma_commit_elect(acc_bar);
            else *abort_flag = 1;
        } else {
            if (p.pdl) asm volatile("griddepcontrol.wait;\n" ::: "memory");
            for (int c = threadIdx.x - 64; c < p.nt; c += kTThreads - 64)   // not the read-only path: may be the kernel before's
                qs[c] = q0 + c < p.Q ? __ldcg(p.qscale + q0 + c) * p.mul : 0.f;
            if (FOUR)
                for (int c = threadIdx.x - 64; c < p.nt; c += kTThreads - 64)
                    qdeep[c] = q0 + c < p.Q && __ldcg(p.deep + q0 + c) ? 1.f : 0.f;
            ok = __all_sync(0xffffffffu, ok && mbar_wait(acc_bar, tile & 1, abort_flag));
            if (ok) {
                // TMEM -> the idle ring, as int32 [column][128 rows]
                tc_fence_after();
                const int qt = warp & 3;
                for (int c = 0; c < N; c += 16) {
                    uint32_t v[16];
                    tmem_ld16(tmem + ((uint32_t)(32 * qt) << 16) + c, v);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        *reinterpret_cast<uint32_t *>(gen_base + ((c + i) * kTP + 32 * qt + lane) * 4) = v[i];
                }
            } else {
                *abort_flag = 1;
            }
        }

        if (!ok && p.status) atomicOr(p.status, QLORA_STATUS_TIMEOUT);
        __syncwarp();
        tc_fence_before();
        __syncthreads();
        if (DEEP && warp == 0 && lane == 0 && *abort_flag) {
            // a wait gave up: time (tens of milliseconds) for this CTA's copies to land
            for (uint32_t i = 0; i < 20000; ++i) __nanosleep(1000);
        } else if (!DEEP && warp == 0 && lane == 0 && *abort_flag) {
            // a wait gave up: let this CTA's copies land before its shared memory is released
            for (int s = 0; s < S && s < nloc; ++s) {
                const int last = ((nloc - 1 - s) / S) * S + s;
                for (uint32_t i = 0; i < kWaitLimit; ++i)
                    if (mbar_try_wait(full_bar(s), (last / S) & 1)) break;
            }
        }
        __syncwarp();
        const int64_t prow = p0 + 4 * lane;
        float ps[4], bs[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool in = prow + e < p.P;
            ps[e] = in && p.pscale ? __ldg(p.pscale + prow + e) : 1.f;
            bs[e] = in && p.bias ? load_any(p.bias, prow + e, p.dtype) : 0.f;
        }
        cluster_sync();   // the cluster's sums are in shared memory
        {
            // column c of plane d over the splits, 4 rows
            auto column = [&](int d, int c) {
                uint4 t = make_uint4(0, 0, 0, 0);
                const uint32_t at = base + ((d * p.nt + c) * kTP + 4 * lane) * 4;
                uint4 v[kTMaxSplits];                 // all in flight: a peer's memory is far
#pragma unroll
                for (uint32_t z = 0; z < kTMaxSplits; ++z)
                    if (z < splits) v[z] = ld_cluster_uint4(mapa_shared(at, z));
#pragma unroll
                for (uint32_t z = 0; z < kTMaxSplits; ++z)
                    if (z < splits) t.x += v[z].x, t.y += v[z].y, t.z += v[z].z, t.w += v[z].w;   // mod 2^32
                return t;
            };
#pragma unroll 4
            for (int c = (int)rank + warp * (int)splits; c < p.nt; c += (kTThreads / 32) * (int)splits) {
                const int64_t q = q0 + c;
                if (q >= p.Q) break;
                uint4 t = column(0, c);
                float v[4] = {sum_float(t.x), sum_float(t.y), sum_float(t.z), sum_float(t.w)};
                const bool four = FOUR && qdeep[c] != 0.f;
                if (DEEP && !four) continue;
                if (FOUR || p.planes == 2) {
                    // as k_int8_wide does, so that a token's gradient does not depend on its batch
                    auto join = [&](float *u, uint4 l) {
                        u[0] = join_digits(u[0], sum_float(l.x)), u[1] = join_digits(u[1], sum_float(l.y));
                        u[2] = join_digits(u[2], sum_float(l.z)), u[3] = join_digits(u[3], sum_float(l.w));
                    };
                    join(v, column(1, c));
                    if (four) {
                        t = column(2, c);
                        float low[4] = {sum_float(t.x), sum_float(t.y), sum_float(t.z), sum_float(t.w)};
                        join(low, column(3, c));
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[e] = join_pairs(v[e], low[e]);
                    }
                } else if (p.planes > 2) {
                    int64_t sum[4] = {sum_int64(t.x), sum_int64(t.y), sum_int64(t.z), sum_int64(t.w)};
                    for (int d = 1; d < p.planes; ++d) {
                        t = column(d, c);
                        sum[0] = sum[0] * 256 + sum_int64(t.x), sum[1] = sum[1] * 256 + sum_int64(t.y);
                        sum[2] = sum[2] * 256 + sum_int64(t.z), sum[3] = sum[3] * 256 + sum_int64(t.w);
                    }
                    if (p.pool == 64) {
                        int64_t all = sum[0] + sum[1] + sum[2] + sum[3];
#pragma unroll
                        for (int x = 8; x > 0; x /= 2) all += __shfl_xor_sync(0xffffffffu, all, x);
                        if ((lane & 15) == 0 && prow < p.P)
                            static_cast<float *>(p.out)[prow / 64 * p.ldo + q] = __fmul_rn(__ll2float_rn(all), qs[c]);
                        continue;
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = __ll2float_rn(sum[e]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = __fmaf_rn(__fmul_rn(v[e], qs[c]), ps[e], bs[e]);
                if (p.q_inner) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (prow + e < p.P) static_cast<float *>(p.out)[(prow + e) * p.ldo + q] = v[e];
                } else if (p.dtype == QLORA_DTYPE_FP32) {
                    float *o = static_cast<float *>(p.out) + q * p.ldo + prow;
                    if (p.vec && prow + 4 <= p.P) {
                        *reinterpret_cast<float4 *>(o) = make_float4(v[0], v[1], v[2], v[3]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (prow + e < p.P) o[e] = v[e];
                    }
                } else {
                    const bool f16 = p.dtype == QLORA_DTYPE_FP16;
                    uint16_t *o = static_cast<uint16_t *>(p.out) + q * p.ldo + prow;
                    if (p.vec && prow + 4 <= p.P) {
                        *reinterpret_cast<uint2 *>(o) = make_uint2(pack2(v[0], v[1], f16), pack2(v[2], v[3], f16));
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (prow + e < p.P) o[e] = enc16(v[e], f16);
                    }
                }
            }
        }
        __syncwarp();
        if (DEEP) fence_proxy_async();                 // the ring's next copies come after these reads
        cluster_sync();   // no CTA leaves, or fills its ring again, while a peer reads its sums
        if (!DEEP) break;
        ++tile;
    }
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(p.tmem_cols));
    }
}


// ---------------------------------------------------------------- many tokens
// A persistent kernel of CTA pairs for the products with tokens (y and dX):
// tcgen05 cta_group::2, M = 256 token rows x N = 256 weight columns per MMA,
// two accumulators a pair.  With one plane they hold two row blocks of a
// 512 x 256 tile, with two the digits of one 256 x 256 tile.  DEEP: a tile with a row
// of four planes among its 256 goes through in two passes, the upper pair of planes
// and the lower; the upper sums wait in the epilogue's registers (4096 x 4096 x 11008
// without such a row 225 us, one among them 282, all 469).
// CTA r of the pair holds rows [128 r, +128) of each block and 128 of the
// columns.  Warp 0 loads (its ring runs on into the next tile), warp 1 of CTA
// 0 issues the MMAs, warps 4..11 take the sums out of TMEM, scale and store.
// The MMAs of the next tile start on an accumulator as soon as it is read:
// its first four k-tiles go to accumulator 0 before accumulator 1 is needed.
// 4096 x 4096 x 11008: 118 us (3.1e15 op/s), two digits of it 232 us (3.2e15).
// The MMAs bound it: 1024 cycles a k-tile at the full rate of the tensor cores,
// 164000 of the 182000 cycles of the pairs with five tiles (344 tiles on 74 pairs);
// a change of tiles idles them for about 3000, the last tile's 256 KB of results
// take 10000 to leave the pair.  L2 and its links are a third busy.
constexpr int kWStages = 4;
constexpr int kWSlab = 128 * kTK;                  // 16 KB: 128 rows of one operand
constexpr int kWStageBytes = 3 * kWSlab;           // two token slabs, one weight slab
constexpr int kWThreads = 384, kWEpiThreads = 256;   // warps: loads, MMAs, two idle; eight for the sums
constexpr int kWTurnPitch = 66;                    // words: 8 rows of 64 words a warp
constexpr int kWTurnBytes = 2560;                  // or a 2 KB block for TMA; a multiple of the swizzle's 512
constexpr int kWSmemBytes = kWStages * kWStageBytes + 1024 + (kWEpiThreads / 32) * kWTurnBytes + 256 + 2 * 2 * 256 * 4;
constexpr int kWGroup = 8;                         // row tiles that share a column tile's pass through L2

struct WideParams {
    int64_t M, N;
    int nk, mt, nt;            // k-tiles; row and column tiles
    int digits;                // two planes: one 256-row block, else two of them
    int64_t plane_rows;
    int b_mn;                  // the weight is MN-major
    const float *rscale, *cscale;
    float mul;
    const void *bias;
    void *out;
    int64_t ldo;
    int dtype, aligned;        // rows of the output start on 16-byte borders: TMA stores
    int pdl;
    const uint8_t *deep;       // digits: rows with four planes have a 1 (zeros up to a multiple of 256)
    uint32_t *status;
};

// One k-tile (four MMAs of the CTA pair) on one accumulator, as umma_i8_ktile.
__device__ __forceinline__ void umma_i8_pair_ktile(uint32_t d_tmem, uint64_t a, uint64_t b, uint64_t bstep,
                                                   uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred e, p, q;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %10, 0;\n\t"
        "setp.eq.b32 q, %10, %10;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %9, p;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::i8 [%0], %3, %4, %9, q;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::i8 [%0], %5, %6, %9, q;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::i8 [%0], %7, %8, %9, q;\n\t}\n" ::"r"(d_tmem),
        "l"(a), "l"(b), "l"(a + 2), "l"(b + bstep), "l"(a + 4), "l"(b + 2 * bstep), "l"(a + 6), "l"(b + 3 * bstep),
        "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void umma_commit_pair_elect(uint32_t bar, uint16_t mask) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}\n" ::"r"(bar),
        "h"(mask)
        : "memory");
}
// Row and column tile of tile t: groups of kWGroup row tiles, columns within a group.
__device__ __forceinline__ void tile_at(const WideParams &p, int t, int &tm, int &tn) {
    const int per = kWGroup * p.nt, g = t / per, in = t % per;
    const int rows = p.mt - g * kWGroup < kWGroup ? p.mt - g * kWGroup : kWGroup;
    tm = g * kWGroup + in % rows;
    tn = in / rows;
}

// A warp's block of 32 rows x 64 bytes of finished values, lane l with 16 words of
// row l, goes out as a TMA store from `turn` (the warp's own 2 KB, swizzled): it
// leaves while the next block is converted (926 x 212 x 10448: 15 us, stored by the
// lanes 20).  Products of short reductions wait for their results (7253 x 560 x
// 12160: 76 us for 176 MB of them, about 8 bytes a cycle and SM; what holds them
// at half of what the memory takes is not known).
__device__ __forceinline__ void store_tile(const CUtensorMap *tm, int x, int y, const uint32_t *w, uint32_t turn) {
    const int lane = threadIdx.x & 31;
    if (lane == 0) bulk_wait_read();                 // the block before is out of `turn`
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(turn + lane * 64 + ((i ^ (lane >> 1 & 3)) << 4)),
                     "r"(w[4 * i]), "r"(w[4 * i + 1]), "r"(w[4 * i + 2]), "r"(w[4 * i + 3])
                     : "memory");
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) {
        tma_store_2d(tm, turn, x, y);
        bulk_commit();
    }
}
// 32 rows x 256 bytes, 64 words a lane, of rows off 16-byte borders: turned in
// shared memory, 16-byte pieces from the offset there that makes their stores
// aligned, then the values around them.
// Two-byte stores to 32 rows at once took longer than the product (an input
// gradient of 2143 x 10158 x 2222: 289 us, so 77); 1131 x 1429 x 27441 takes 68 us,
// two bytes a lane along a row 101, and 1131 x 1429 x 27440, on borders, 58.
template <bool F32>
__device__ __forceinline__ void store_ragged(const WideParams &p, int64_t m0, int64_t n, const uint32_t *w,
                                             uint32_t *turn) {
    if (n >= p.N || m0 >= p.M) return;               // the same for all lanes
    constexpr int kSize = F32 ? 4 : 2;
    constexpr int kLanes = F32 ? 8 : 16, kRows = 32 / kLanes;      // a row's values around its pieces, rows a store
    const int lane = threadIdx.x & 31;
    const int bytes = p.N - n < 256 / kSize ? (int)(p.N - n) * kSize : 256;
    const int64_t pitch = p.ldo * kSize;
    const int rows = p.M - m0 < 32 ? (int)(p.M - m0) : 32;
    uint8_t *const out = static_cast<uint8_t *>(p.out) + m0 * pitch + n * kSize;
#pragma unroll 1
    for (int g = 0; g < 32; g += 8) {
        __syncwarp();
        if ((lane & 24) == g)
#pragma unroll
            for (int j = 0; j < 32; ++j)
                *reinterpret_cast<uint2 *>(turn + (lane & 7) * kWTurnPitch + 2 * j) = make_uint2(w[2 * j], w[2 * j + 1]);
        __syncwarp();
        int r = lane >> 4;
        uint8_t *o = out + (g + r) * pitch;
#pragma unroll
        for (int i = 0; i < 4; ++i, r += 2, o += 2 * pitch) {
            const int b = (int)(-reinterpret_cast<uintptr_t>(o) & 15u) + 16 * (lane & 15);
            if (g + r < rows && b + 16 <= bytes) {
                const uint32_t *from = turn + r * kWTurnPitch + (b >> 2);
                uint32_t v[5];
#pragma unroll
                for (int j = 0; j < 5; ++j) v[j] = from[j];
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = F32 ? v[j] : __funnelshift_r(v[j], v[j + 1], 8 * (b & 3));
                *reinterpret_cast<uint4 *>(o + b) = make_uint4(v[0], v[1], v[2], v[3]);
            }
        }
        r = lane / kLanes;
        o = out + (g + r) * pitch;
#pragma unroll
        for (int i = 0; i < 8 / kRows; ++i, r += kRows, o += kRows * pitch) {
            const int head = (int)(-reinterpret_cast<uintptr_t>(o) & 15u);
            const int around = head < bytes ? (bytes - head) & ~15 : bytes;      // bytes of pieces from head on
            int b = (lane & (kLanes - 1)) * kSize;
            if (b >= head) b += around;
            if (g + r < rows && b < bytes) {
                const uint8_t *from = reinterpret_cast<const uint8_t *>(turn + r * kWTurnPitch) + b;
                if (F32) *reinterpret_cast<uint32_t *>(o + b) = *reinterpret_cast<const uint32_t *>(from);
                else *reinterpret_cast<uint16_t *>(o + b) = *reinterpret_cast<const uint16_t *>(from);
            }
        }
    }
}
// Is one of the 256 rows of a tile deep?  Eight flags a lane, loaded a tile ahead.
__device__ __forceinline__ uint2 deep_flags(const WideParams &p, int t) {
    if (t >= p.mt * p.nt) return make_uint2(0, 0);
    int tm, tn;
    tile_at(p, t, tm, tn);
    return __ldcg(reinterpret_cast<const uint2 *>(p.deep + (int64_t)tm * 256) + (threadIdx.x & 31));
}
__device__ __forceinline__ bool any_flag(uint2 f) { return __any_sync(0xffffffffu, (f.x | f.y) != 0); }

template <bool DEEP>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWThreads, 1)
k_int8_wide(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
            const __grid_constant__ CUtensorMap tmY, const WideParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t *gen_base = smem_raw + (base - raw_addr);
    const uint32_t turns = base + kWStages * kWStageBytes, bar0 = turns + (kWEpiThreads / 32) * kWTurnBytes;
    uint8_t *bars = gen_base + (bar0 - base);
    auto full = [&](int s) { return bar0 + 8u * s; };                   // CTA 0: both CTAs' bytes landed
    auto empty = [&](int s) { return bar0 + 8u * (kWStages + s); };     // stage free (in both CTAs)
    const uint32_t acc_full = bar0 + 8u * (2 * kWStages);               // a tile's sums are complete (both)
    auto acc_free = [&](int h) { return bar0 + 8u * (2 * kWStages + 1 + h); };   // CTA 0: accumulator h read
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + 208);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + 240);
    float *cbuf = reinterpret_cast<float *>(bars + 256);   // [2][2][256]

    const int warp = warp_index(), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pairs = gridDim.x >> 1, pair = blockIdx.x >> 1;
    const int tiles = p.mt * p.nt;
    const int mrows = p.digits ? 256 : 512;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kWStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        mbar_init(acc_full, 1);
        for (int h = 0; h < 2; ++h) mbar_init(acc_free(h), 2 * (kWEpiThreads / 32));
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
        fence_proxy_async();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(tmem_holder)),
                     "r"(512u));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // both CTAs' barriers initialised before any cross-CTA use
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    bool ok = true;
    // 384 x 168 registers at launch = 128 x 40 + 256 x 232
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;\n");
        if (warp == 0) {
            {
                const bool leader = elect_one();
                auto load_w = [&](int s, int t0, int tn) {
                    const uint32_t fa0 = mapa_shared(full(s), 0);
                    const int c0 = tn * 256 + 128 * (int)rank;
                    if (rank == 0) mbar_expect_tx(full(s), 2 * kWStageBytes);
                    const uint32_t sb = base + s * kWStageBytes + 2 * kWSlab;
                    if (p.b_mn) tma_load_2d_pair(sb, &tmW, c0, t0, fa0);
                    else tma_load_2d_pair(sb, &tmW, t0, c0, fa0);
                };
                auto load_x = [&](int s, int t0, int tm, int pass) {
                    const uint32_t fa0 = mapa_shared(full(s), 0);
                    const uint32_t sa = base + s * kWStageBytes;
                    const int r0 = tm * mrows + 128 * (int)rank + (DEEP ? pass * 2 * (int)p.plane_rows : 0);
                    tma_load_2d_pair(sa, &tmX, t0, r0, fa0);
                    tma_load_2d_pair(sa + kWSlab, &tmX, t0, r0 + (p.digits ? (int)p.plane_rows : 256), fa0);
                };
                int it = 0, head = 0;
                uint2 flags = make_uint2(0, 0);
                for (int t = pair; t < tiles && ok; t += pairs) {
                    int tm, tn;
                    tile_at(p, t, tm, tn);
                    if (it == 0 && p.pdl) {
                        // the weight does not depend on the kernel before
                        head = p.nk < kWStages ? p.nk : kWStages;
                        if (leader)
                            for (int k = 0; k < head; ++k) load_w(k, k * kTK, tn);
                        asm volatile("griddepcontrol.wait;\n" ::: "memory");
                    }
                    int passes = 1;
                    if (DEEP) {
                        if (it == 0) flags = deep_flags(p, t);
                        passes = any_flag(flags) ? 2 : 1;
                        flags = deep_flags(p, t + pairs);
                    }
                    if (leader) {
                        int i = it;
                        for (int pass = 0; pass < passes && ok; ++pass)
                            for (int k = 0; k < p.nk && ok; ++k, ++i) {
                                const int s = i % kWStages;
                                if (i >= kWStages) ok = mbar_wait(empty(s), ((i / kWStages) & 1) ^ 1, abort_flag);
                                if (!ok) break;
                                if (i >= head) load_w(s, k * kTK, tn);
                                load_x(s, k * kTK, tm, pass);
                            }
                    }
                    it += passes * p.nk;
                    ok = __all_sync(0xffffffffu, ok);
                }
                if (!ok) *abort_flag = 1;
            }
        } else if (warp == 1) {
            if (rank == 0) {
                const uint32_t idesc = idesc_i8(256, 256, 0, p.b_mn ? 1u : 0u);
                const uint64_t bstep = p.b_mn ? 256u : 2u;
                const uint64_t dX = sdesc(base, 16, 1024), dW = sdesc(base + 2 * kWSlab, 16, 1024);
                constexpr uint32_t kStageD = kWStageBytes >> 4, kSlabD = kWSlab >> 4;
                auto mma = [&](uint32_t s, uint32_t h, uint32_t acc) {
                    umma_i8_pair_ktile(tmem + h * 256, dX + s * kStageD + h * kSlabD, dW + s * kStageD, bstep, idesc, acc);
                };
                static_assert((kWStages & (kWStages - 1)) == 0, "stage and parity from the running k-tile's bits");
                uint32_t it = 0, i = 0;                // k-tiles and passes before
                uint2 flags = make_uint2(0, 0);
                if (DEEP) {
                    if (p.pdl) asm volatile("griddepcontrol.wait;\n" ::: "memory");
                    flags = deep_flags(p, pair);
                }
                for (int t = pair; t < tiles && ok; t += pairs) {
                    int passes = 1;
                    if (DEEP) {
                        passes = any_flag(flags) ? 2 : 1;
                        flags = deep_flags(p, t + pairs);
                    }
                    for (int pass = 0; pass < passes && ok; ++pass, ++i) {
                        const uint32_t nk = p.nk, lead = nk < kWStages ? nk : kWStages;
                        if (i > 0) ok = __all_sync(0xffffffffu, mbar_wait_cluster(acc_free(0), (i - 1) & 1, abort_flag));
                        for (uint32_t k = 0; k < lead && ok; ++k) {
                            const uint32_t s = (it + k) % kWStages;
                            ok = __all_sync(0xffffffffu, mbar_wait_cluster(full(s), ((it + k) / kWStages) & 1, abort_flag));
                            if (!ok) break;
                            tc_fence_after();
                            mma(s, 0, k > 0 ? 1u : 0u);
                        }
                        if (ok && i > 0) ok = __all_sync(0xffffffffu, mbar_wait_cluster(acc_free(1), (i - 1) & 1, abort_flag));
                        if (!ok) break;
                        tc_fence_after();
                        for (uint32_t k = 0; k < lead; ++k) {
                            const uint32_t s = (it + k) % kWStages;
                            mma(s, 1, k > 0 ? 1u : 0u);
                            umma_commit_pair_elect(empty(s), 0x3);
                        }
                        for (uint32_t k = lead; k < nk; ++k) {
                            const uint32_t s = (it + k) % kWStages;
                            ok = __all_sync(0xffffffffu, mbar_wait_cluster(full(s), ((it + k) / kWStages) & 1, abort_flag));
                            if (!ok) break;
                            tc_fence_after();
                            mma(s, 0, 1u);
                            mma(s, 1, 1u);
                            umma_commit_pair_elect(empty(s), 0x3);
                        }
                        if (ok) umma_commit_pair_elect(acc_full, 0x3);
                        it += nk;
                    }
                }
                if (!ok) *abort_flag = 1;
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 232;\n");
        if (p.pdl) asm volatile("griddepcontrol.wait;\n" ::: "memory");
        const int e = threadIdx.x - 128;
        const int qt = warp & 3, cg = (warp - 4) >> 2;     // TMEM lane quarter, column half
        const uint32_t lanes = (uint32_t)(32 * qt) << 16;
        const uint32_t free0 = mapa_shared(acc_free(0), 0);
        int i = 0;
        uint32_t full_turns = 0;                               // DEEP: passes before
        uint2 flags = make_uint2(0, 0);
        if (DEEP) flags = deep_flags(p, pair);
        for (int t = pair; t < tiles; t += pairs, ++i) {   // all of them, also once a wait has given up
            int tm, tn;
            tile_at(p, t, tm, tn);
            bool two = false;
            if (DEEP) {
                two = any_flag(flags);
                flags = deep_flags(p, t + pairs);
            }
            const int64_t n0 = (int64_t)tn * 256;
            float *cs = cbuf + (i & 1) * 512, *cb = cs + 256;
            cs[e] = p.cscale && n0 + e < p.N ? __ldg(p.cscale + n0 + e) : 1.f;
            cb[e] = p.bias && n0 + e < p.N ? load_any(p.bias, n0 + e, p.dtype) : 0.f;
            const int64_t mblk = (int64_t)tm * mrows + 128 * rank + 32 * qt, mrow = mblk + lane;
            const uint32_t turn = turns + (warp - 4) * kWTurnBytes;
            uint32_t *turn_words = reinterpret_cast<uint32_t *>(gen_base + (turn - base));
            float rs[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t m = mrow + 256 * h;
                rs[h] = m < p.M && (h == 0 || !p.digits) ? __ldcg(p.rscale + m) * p.mul : 0.f;
            }
            ok = mbar_wait_turn<1, kWEpiThreads>(ok, acc_full, (DEEP ? full_turns++ : (uint32_t)i) & 1, abort_flag);   // cs and cb are there
            if (!ok && !(DEEP && two)) continue;
            tc_fence_after();
            // The next tile's MMAs wait for the accumulators: a warp takes its 128
            // columns of one out at once and frees it before it scales, packs and
            // stores them, and takes the other before it stores the first (freed
            // between blocks of 32 columns, 4096 x 4096 x 11008 took 128 us for 118).
            const int c0 = cg * 128;
            auto release = [&](int h) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(free0 + 8 * h);
            };
            auto scaled = [&](int c, float4 x, float r) {   // columns c .. c + 3
                const float4 s4 = *reinterpret_cast<const float4 *>(cs + c);
                const float4 b4 = *reinterpret_cast<const float4 *>(cb + c);
                return make_float4(__fmaf_rn(__fmul_rn(x.x, r), s4.x, b4.x), __fmaf_rn(__fmul_rn(x.y, r), s4.y, b4.y),
                                   __fmaf_rn(__fmul_rn(x.z, r), s4.z, b4.z), __fmaf_rn(__fmul_rn(x.w, r), s4.w, b4.w));
            };
            auto sums4 = [](const uint32_t *v) {
                if constexpr (DEEP) return make_float4(sum_float(v[0]), sum_float(v[1]), sum_float(v[2]), sum_float(v[3]));
                return make_float4((float)(int)v[0], (float)(int)v[1], (float)(int)v[2], (float)(int)v[3]);
            };
            auto put4 = [](uint32_t *to, float4 v, auto dt) {
                if constexpr (dt == QLORA_DTYPE_FP32) {
                    to[0] = __float_as_uint(v.x), to[1] = __float_as_uint(v.y);
                    to[2] = __float_as_uint(v.z), to[3] = __float_as_uint(v.w);
                } else {
                    to[0] = pack2(v.x, v.y, dt == QLORA_DTYPE_FP16);
                    to[1] = pack2(v.z, v.w, dt == QLORA_DTYPE_FP16);
                }
            };
            if constexpr (DEEP) {
                if (two) {
                    auto pairs16 = [&](int c, float (&v)[16]) {   // 16 columns of the two accumulators, joined
                        uint32_t raw[32];
                        tmem_ld16(tmem + lanes + c, *reinterpret_cast<uint32_t(*)[16]>(raw));
                        tmem_ld16(tmem + lanes + 256 + c, *reinterpret_cast<uint32_t(*)[16]>(raw + 16));
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[j] = join_digits(sum_float(raw[j]), sum_float(raw[16 + j]));
                    };
                    float upper[8][16];
                    if (ok) {
#pragma unroll
                        for (int g = 0; g < 8; ++g) pairs16(c0 + 16 * g, upper[g]);
                        release(0), release(1);
                    }
                    ok = mbar_wait_turn<1, kWEpiThreads>(ok, acc_full, full_turns++ & 1, abort_flag);
                    if (!ok) continue;
                    tc_fence_after();
                    const bool mine = mrow < p.M && __ldcg(p.deep + mrow) != 0;
                    auto finish_two = [&](auto dt) {              // a 16-bit type: 32 columns a block
                        uint32_t out[64];
#pragma unroll
                        for (int g = 0; g < 8; ++g) {
                            float low[16];
                            pairs16(c0 + 16 * g, low);
                            if (g == 7) release(0), release(1);
#pragma unroll
                            for (int j = 0; j < 16; j += 4) {
                                const float *u = upper[g] + j, *l = low + j;
                                const float4 x = mine ? make_float4(join_pairs(u[0], l[0]), join_pairs(u[1], l[1]),
                                                                    join_pairs(u[2], l[2]), join_pairs(u[3], l[3]))
                                                      : make_float4(u[0], u[1], u[2], u[3]);
                                put4(out + 8 * g + j / 2, scaled(c0 + 16 * g + j, x, rs[0]), dt);
                            }
                            const int64_t n = n0 + c0 + 32 * (g / 2);
                            if (p.aligned && g % 2 == 1 && n < p.N && mblk < p.M)
                                store_tile(&tmY, (int)(n * 2), (int)mblk, out + 8 * (g - 1), turn);
                        }
                        if (!p.aligned) store_ragged<false>(p, mblk, n0 + c0, out, turn_words);
                    };
                    if (p.dtype == QLORA_DTYPE_BF16) finish_two(std::integral_constant<int, QLORA_DTYPE_BF16>{});
                    else finish_two(std::integral_constant<int, QLORA_DTYPE_FP16>{});
                    continue;
                }
            }
            auto finish = [&](auto dt) {
                constexpr bool f32 = dt == QLORA_DTYPE_FP32;
                constexpr int per = f32 ? 1 : 2, cols = 16 * per, count = 128 / cols;   // a block's columns
                uint32_t out[64 * 2 / per];                                             // a row block's 128 columns
                auto store = [&](int h, int b) {
                    if (p.aligned) {
                        const int64_t n = n0 + c0 + cols * b;
                        if (n < p.N && mblk + 256 * h < p.M)
                            store_tile(&tmY, (int)(n * (4 / per)), (int)(mblk + 256 * h), out + 16 * b, turn);
                    } else if (b % 4 == 3) {
                        store_ragged<f32>(p, mblk + 256 * h, n0 + c0 + cols * (b - 3), out + 16 * (b - 3), turn_words);
                    }
                };
                if (p.digits) {
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const int c = c0 + 32 * g;
                        uint32_t raw[64];
                        tmem_ld32_issue(tmem + lanes + c, raw);
                        tmem_ld32_issue(tmem + lanes + 256 + c, raw + 32);
                        tmem_wait(raw);
                        if (g == 3) release(0), release(1);
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
                            const float4 u = sums4(raw + j), l = sums4(raw + 32 + j);
                            const float4 x = make_float4(join_digits(u.x, l.x), join_digits(u.y, l.y),
                                                         join_digits(u.z, l.z), join_digits(u.w, l.w));
                            put4(out + (32 * g + j) / per, scaled(c + j, x, rs[0]), dt);
                        }
                    }
#pragma unroll
                    for (int b = 0; b < count; ++b) store(0, b);
                } else {
                    uint32_t raw[128];
                    auto take = [&](int h) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) tmem_ld32_issue(tmem + lanes + 256 * h + c0 + 32 * c, raw + 32 * c);
                        tmem_wait(raw);
                        release(h);
                    };
                    auto convert = [&](int h, int b) {
#pragma unroll
                        for (int j = 0; j < cols; j += 4)
                            put4(out + 16 * b + j / per, scaled(c0 + cols * b + j, sums4(raw + cols * b + j), rs[h]), dt);
                    };
                    take(0);
                    if constexpr (f32) {
#pragma unroll
                        for (int b = 0; b < count; ++b) convert(0, b), store(0, b);
                        take(1);
#pragma unroll
                        for (int b = 0; b < count; ++b) convert(1, b), store(1, b);
                    } else {                         // packed, so that the registers hold both
#pragma unroll
                        for (int b = 0; b < count; ++b) convert(0, b);
                        take(1);
                        if (p.aligned) {
#pragma unroll
                            for (int b = 0; b < count; ++b) store(0, b), convert(1, b);
                        } else {
                            store(0, 3);
#pragma unroll
                            for (int b = 0; b < count; ++b) convert(1, b);
                        }
#pragma unroll
                        for (int b = 0; b < count; ++b) store(1, b);
                    }
                }
            };
            if (p.dtype == QLORA_DTYPE_BF16) finish(std::integral_constant<int, QLORA_DTYPE_BF16>{});
            else if (p.dtype == QLORA_DTYPE_FP16) finish(std::integral_constant<int, QLORA_DTYPE_FP16>{});
            else if (!DEEP) finish(std::integral_constant<int, QLORA_DTYPE_FP32>{});   // gradients are 16-bit
        }
        if (lane == 0) bulk_wait_all();              // no memory of this CTA is read behind its end
        if (!ok) *abort_flag = 1;
    }

    if (!ok && p.status) atomicOr(p.status, QLORA_STATUS_TIMEOUT);
    __syncwarp();   // reconverge single-lane roles before the barriers
    tc_fence_before();
    __syncthreads();
    if (warp == 0 && lane == 0 && *abort_flag && rank == 0) {
        // a wait gave up: time (tens of milliseconds) for both CTAs' copies to land
        for (uint32_t i = 0; i < 20000; ++i) __nanosleep(1000);
    }
    __syncwarp();
    cluster_sync();   // no CTA leaves while its peer may still signal it
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(512u));
    }
}

}  // namespace

// How a product is cut: columns of B a tile, splits of the reduction.  The
// least of a model of the measured times (900 of them: 16 to 4300 tokens on weights
// of 700 to 11008 channels, reductions of 500 to 28638, 16 to 256 columns, 1 to 8
// splits; off by 10%, and the plan it finds takes 0.6% longer than the fastest of
// them): 0.2 us, 4.5 us a wave of CTAs, for each k-tile of a CTA 0.18 us + 0.5 ns a
// column alone on its SM (0.085 us more where the ring has only four stages: 192
// columns beat 256), 2 ns a column where two share it (as N <= 128 lets them), 69 ns
// a column for the results, which the splits divide, 0.7 us + 0.27 us a split for the
// exchange, the k-tiles half as much again for rows off 128-byte borders (their
// pieces straddle two lines).  Clusters past 2 leave places free: a wave of them is
// counted as 0.92 of the SMs' (288 CTAs in clusters of 6 took two waves), and
// clusters of big CTAs past 6 do not all find a place at once (8 splits of N = 176
// took twice the time of 6).
struct TallPlan {
    int nt, splits, per;
    double us;
};
static TallPlan plan_tall(const Int8Product &g, int planes, int64_t Q, int nk) {
    const int sms = device_sms();
    const int cap = 256 / planes / 16 * 16;
    const int64_t pt = (g.P + kTP - 1) / kTP;
    const double lines = g.lda % 128 || g.ldb % 128 ? 1.5 : 1.0;
    TallPlan best{};
    int last = 0;
    for (int at_most = cap; at_most >= 16; at_most -= 16) {
        const int64_t tq = (Q + at_most - 1) / at_most;
        const int nt = (int)(((Q + tq - 1) / tq + 15) / 16 * 16);      // as even as that many tiles can be
        if (nt == last) continue;
        last = nt;
        const int N = nt * planes, most = N <= 64 ? kTMaxSplits : 6;
        const int64_t slots = (N <= kTTwoN ? 2 : 1) * (int64_t)sms, tiles = pt * ((Q + nt - 1) / nt);
        for (int s = 1; s <= most && (s == 1 || 2 * s <= nk); ++s) {
            const int per = (nk + s - 1) / s;
            if ((nk + per - 1) / per != s) continue;
            const int64_t units = tiles * s, places = s > 2 ? slots * 23 / 25 : slots;
            const double waves = (double)((units + places - 1) / places);
            const double column = units > sms && N <= kTTwoN ? 0.002 : 0.0005;
            const double tile = (0.18 + column * N + (N > 224 ? 0.085 : 0.0)) * lines;
            const double us = 0.2 + waves * (4.5 + per * tile + 0.069 * N / s) + (s > 1 ? 0.7 + 0.27 * s : 0.0);
            if (best.nt == 0 || us < best.us) {
                best = TallPlan{nt, s, per, us};
            }
        }
    }
    return best;
}

// only_deep: the launch of its DEEP form, after the product of two planes has run.
static int launch_int8_tall(const Int8Product &g, int planes, const TallPlan &plan, bool only_deep, uint32_t *d_status,
                            cudaStream_t st) {
    if (g.P <= 0 || g.Q <= 0) return QLORA_OK;
    TallParams p{};
    p.P = g.P;
    p.Q = g.Q;
    p.planes = planes;
    p.deep = g.deep;
    p.plane_rows = g.plane_rows;
    p.nk = (int)((g.R + kTK - 1) / kTK);
    p.a_mn = g.a_mn;
    p.nt = plan.nt;
    p.per = plan.per;
    const int N = p.planes * p.nt;
    const int64_t tiles_q = (g.Q + p.nt - 1) / p.nt, splits = plan.splits;
    p.stage_bytes = kTABytes + N * kTK;
    p.tmem_cols = 32;
    while ((int)p.tmem_cols < N) p.tmem_cols *= 2;
    p.stages = (int)((N <= kTTwoN ? kTSmemTwo : kTSmemOne) / p.stage_bytes);
    if (p.stages > kTMaxStages) p.stages = kTMaxStages;
    p.qscale = g.qscale;
    p.pscale = g.pscale;
    p.mul = g.mul;
    p.bias = g.bias;
    p.out = g.out;
    p.ldo = g.ldo;
    p.q_inner = g.q_inner;
    p.pool = g.pool;
    p.dtype = g.dtype;
    const int esize = g.dtype == QLORA_DTYPE_FP32 ? 4 : 2;
    p.vec = g.ldo % 4 == 0 && (reinterpret_cast<uintptr_t>(g.out) & (4 * esize - 1)) == 0;
    p.pdl = g.pdl && !only_deep;
    p.tiles_q = tiles_q;
    p.status = d_status;
    const int64_t brows = g.plane_rows * (planes - 1) + g.Q;
    CUtensorMap tA, tB;
    bool ok = g.a_mn ? make_map(&tA, g.a, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, g.P, g.R, g.lda, 128, kTK,
                                CU_TENSOR_MAP_SWIZZLE_128B)
                     : make_map(&tA, g.a, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, g.R, g.P, g.lda, kTK, kTP,
                                CU_TENSOR_MAP_SWIZZLE_128B);
    ok = ok && make_map(&tB, g.b, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, g.R, brows, g.ldb, kTK, (uint32_t)p.nt,
                        CU_TENSOR_MAP_SWIZZLE_128B);
    if (!ok) return QLORA_EUNSUPPORTED;
    const size_t ring = (size_t)p.stages * p.stage_bytes;
    if (ring < (size_t)N * kTP * 4) return QLORA_EUNSUPPORTED;   // the sums take the ring's place
    const int smem = (int)ring + 1024 + 256 + 1024;
    auto *k = only_deep ? k_int8_tall<true, true> : planes == 4 ? k_int8_tall<true, false> : k_int8_tall<false, false>;
    if (set_max_smem(reinterpret_cast<const void *>(k), smem) != cudaSuccess) return QLORA_ECUDA;
    cudaLaunchConfig_t cfg{};
    const int64_t tiles_p = (g.P + kTP - 1) / kTP;
    int64_t rows_y = tiles_q;
    if (only_deep) {   // about one CTA an SM
        rows_y = device_sms() / (tiles_p * splits);
        rows_y = rows_y < 1 ? 1 : rows_y < tiles_q ? rows_y : tiles_q;
    }
    cfg.gridDim = dim3((unsigned)tiles_p, (unsigned)rows_y, (unsigned)splits);
    cfg.blockDim = dim3(kTThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = (unsigned)splits;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.pdl ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, k, tA, tB, p) != cudaSuccess) return QLORA_ECUDA;
    QLORA_LAUNCH_CHECK();
    return QLORA_OK;
}

static int launch_int8_wide(const Int8Product &g, uint32_t *d_status, cudaStream_t st) {
    WideParams p{};
    p.M = g.Q;
    p.N = g.P;
    p.digits = g.planes == 2;
    p.plane_rows = g.plane_rows;
    p.nk = (int)((g.R + kTK - 1) / kTK);
    const int mrows = p.digits ? 256 : 512;
    p.mt = (int)((p.M + mrows - 1) / mrows);
    p.nt = (int)((p.N + 255) / 256);
    p.b_mn = g.a_mn;
    p.rscale = g.qscale;
    p.cscale = g.pscale;
    p.mul = g.mul;
    p.bias = g.bias;
    p.out = g.out;
    p.ldo = g.ldo;
    p.dtype = g.dtype;
    const uintptr_t at = reinterpret_cast<uintptr_t>(g.out) | (uintptr_t)(g.ldo * (g.dtype == QLORA_DTYPE_FP32 ? 4 : 2));
    p.aligned = at % 16 == 0 && p.N < (1 << 29);          // a TMA coordinate in bytes
    p.pdl = g.pdl;
    p.deep = g.deep;
    p.status = d_status;
    const int64_t xrows = g.plane_rows * (g.deep ? 3 : g.planes - 1) + g.Q;
    CUtensorMap tX, tW;
    bool ok = make_map(&tX, g.b, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, g.R, xrows, g.ldb, kTK, 128,
                       CU_TENSOR_MAP_SWIZZLE_128B);
    ok = ok && (g.a_mn ? make_map(&tW, g.a, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, g.P, g.R, g.lda, 128, kTK,
                                  CU_TENSOR_MAP_SWIZZLE_128B)
                       : make_map(&tW, g.a, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, g.R, g.P, g.lda, kTK, 128,
                                  CU_TENSOR_MAP_SWIZZLE_128B));
    const int size = g.dtype == QLORA_DTYPE_FP32 ? 4 : 2;
    CUtensorMap tY = tX;                                   // unused for rows off 16-byte borders
    if (p.aligned)
        ok = ok && make_map(&tY, g.out, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p.N * size, p.M, g.ldo * size, 64, 32,
                            CU_TENSOR_MAP_SWIZZLE_64B);
    if (!ok) return QLORA_EUNSUPPORTED;
    auto *k = g.deep ? k_int8_wide<true> : k_int8_wide<false>;
    if (set_max_smem(reinterpret_cast<const void *>(k), kWSmemBytes) != cudaSuccess) return QLORA_ECUDA;
    const int64_t tiles = (int64_t)p.mt * p.nt, pairs = device_sms() / 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs)));
    cfg.blockDim = dim3(kWThreads);
    cfg.dynamicSmemBytes = kWSmemBytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = g.pdl ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, k, tX, tW, tY, p) != cudaSuccess) return QLORA_ECUDA;
    QLORA_LAUNCH_CHECK();
    return QLORA_OK;
}

// The wide kernel: 8.5 us of start and end, and for each of a pair's tiles 1 us and
// 0.575 us a k-tile (512 x 256 outputs, or 256 x 256 of two digits), though no less
// than its results take where another tile follows: 3.5 us and as much for full
// rows.  4096 tokens on 1024 x 1024: 14.1 us wide, 16.4 tall; 512 on 11008 x 4096: 29
// and 45; 5 on 131072 x 128: 34 and 18; 384 on 11008 x 8192: 46 and 41; 4096 on 512 x
// 4096: 26 and 17, as the model has them in order.
// With deep tokens (which only the device knows) the wide kernel takes the tiles that hold
// one in two passes; few tokens have four planes for all of them in one launch of the tall one where
// that costs no more than two planes and a second launch, for the deep ones alone (it finds none in 3 us).
int launch_int8_product(const Int8Product &g, uint32_t *d_status, cudaStream_t st) {
    if (g.P <= 0 || g.Q <= 0) return QLORA_OK;
    const int nk = (int)((g.R + kTK - 1) / kTK);
    const TallPlan plan = plan_tall(g, g.planes, g.Q, nk);
    bool wide = false;
    double us = plan.us;
    // a product (not a gradient) of 131072 terms stays with the tall kernel: the wide one converts its
    // sums without sum_float, which costs it registers (7253 x 560 x 12160: 78 us for 77)
    if (!g.q_inner && g.planes <= 2 && (g.R < 131072 || g.deep)) {
        const int64_t mrows = g.planes == 2 ? 256 : 512, pairs = device_sms() / 2;
        const int64_t tiles = ((g.Q + mrows - 1) / mrows) * ((g.P + 255) / 256);
        const int64_t rounds = (tiles + pairs - 1) / pairs;
        const double tile = 1.0 + 0.575 * nk, rows = g.Q < mrows ? (double)g.Q / mrows : 1.0;
        const double results = 3.5 + 3.5 * rows;
        const double wide_us = 8.5 + tile + (double)(rounds - 1) * (tile > results ? tile : results);
        const bool grid = (g.Q + plan.nt - 1) / plan.nt <= 65535;          // the tall kernel's grid
        wide = !grid || wide_us < plan.us;
        if (wide) us = wide_us;
    }
    if (g.deep) {
        const TallPlan all = plan_tall(g, 4, g.Q, nk);
        if (all.us <= us + (wide ? 0.0 : 3.0) && (g.Q + all.nt - 1) / all.nt <= 65535)
            return launch_int8_tall(g, 4, all, false, d_status, st);
    }
    if (wide) return launch_int8_wide(g, d_status, st);
    const int rc = launch_int8_tall(g, g.planes, plan, false, d_status, st);
    if (rc || !g.deep) return rc;
    return launch_int8_tall(g, 4, plan_tall(g, 4, g.Q < 64 ? g.Q : 64, nk), true, d_status, st);
}

}  // namespace qlora
