// bsa_attention_q8.cu -- sparse decode attention over a paged cache held in 8
// bits with a scale per 16-token page and head.
//
// What it computes, for a row (t, h) with G query heads and its first ctx
// table tokens (codes kc, vc, page scales ks, vs):
//   y_j = log2(e) scale ks_j (q . kc_j),
//   out = sum_j 2^(y_j - max y) vs_j vc_j / sum_j 2^(y_j - max y).
//
// Both products run on the tensor core on the cached codes as they are, with
// no widening pass: the tokens (or, for the values, the head's dimensions) are
// the 128 rows of a tcgen05 f8 MMA and the G query heads its few columns.  The
// other operand is made 8-bit too, as a sum of two terms in their own
// columns, x = hi + lo / 16 with hi = e4m3(x), lo = e4m3(16 (x - hi)).
//  - A bf16 query has 8 significant bits; scaled by a power of two so that the
//    head's largest magnitude lies in [128, 256), hi takes 4 of them and the
//    rounded rest of at most 2^-4 fits lo: exact down to 2^-21 of the largest.
//  - A probability keeps a relative error below 2^-8 (bf16's), down to 2^-22
//    of the row's largest p_j vs_j, which is scaled to 256.
// The sums, maxima and accumulators are fp32.
//
// The work: a CTA takes an item (a row, or a share of its 128-token blocks
// when rows are few) and walks it in chunks of as many blocks as their scores
// fit in 256 TMEM columns (16 blocks up to 8 query heads, 8 up to 16).  A
// chunk's scores are complete before its probabilities are formed, so there
// is one maximum per chunk and no correction of accumulators in TMEM.
//  warp 4     copies blocks by TMA into a ring of shared-memory stages: the
//             chunk's key blocks, then its value blocks, a box per page;
//             pages outside the context or the cache are boxes past the end
//             of the tensor, which arrive as zeros,
//  warp 5     issues the MMAs and frees the stages,
//  warps 0-3  thread i is token i of a block (probabilities) and dimension i
//             of the head (output).
// Values behind the context's end in its last page are set to zero in shared
// memory (they may be NaN codes); such keys only reach their own scores.
// The kernel is bound by the copies: 2 D bytes a token.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <mutex>

#include "bsa_internal.h"
#include "bsa_tcgen05.cuh"

namespace bsa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kSoftmaxThreads = 128;
constexpr int kQ8Threads = kSoftmaxThreads + 64;
constexpr int kScoreCols = 256;          // TMEM columns of a chunk's scores
constexpr int kTmemCols = 512;

template <int D, int GP>
struct Q8Cfg {
    static constexpr int N = GP <= 8 ? 16 : 32;       // MMA columns: two terms of each head
    static constexpr int NB = kScoreCols / N;         // blocks per chunk
    static constexpr int PANELS = D == 256 ? 2 : 1;   // 128-byte parts of a head's row
    static constexpr int ROWB = D / PANELS;           // bytes of a row in a panel: 64 or 128
    static constexpr int PANEL_BYTES = 128 * ROWB;
    static constexpr int STAGE = 128 * D;
    static constexpr int RING = 184320 / STAGE;       // 22, 11 or 5 stages of 8, 16 or 32 KB
    static constexpr int P_BYTES = NB * N * 128;      // 32 KB
    static constexpr int Q_PANEL = N * ROWB;
    static constexpr int Q_BYTES = PANELS * Q_PANEL;
    static constexpr int SMEM = RING * STAGE + P_BYTES + Q_BYTES + 1024;
    static constexpr uint32_t SWIZZLE = ROWB == 128 ? 2 : 4;
    static constexpr uint32_t ATOM = 8 * ROWB;        // 8 rows: the swizzle's period
};

struct Q8Params {
    const uint16_t* q;
    const float* ks;
    const float* vs;
    const int32_t* bt;
    const int32_t* ctx;
    uint16_t* out;
    float* part;             // partial results of split rows, or null
    int64_t num_pages;
    int32_t rows, H, G, width;
    int32_t splits;          // items per row
    uint32_t k_idesc, v_idesc;
    float scale_log2e;
    uint32_t* status;
};

// floats of one partial result: G x D outputs, then per head the largest
// score, the largest weighted score and the sum
__host__ __device__ inline int64_t part_floats(int G, int D) { return (int64_t)G * D + 3 * G; }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max_warp(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, o));
    return x;
}
__device__ __forceinline__ float sum_warp(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
    return x;
}
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// two values as e4m3 codes: a in the low byte
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ float2 unpack_e4m3(uint32_t c) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
    float2 f;
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
        : "=f"(f.x), "=f"(f.y)
        : "r"(h));
    return f;
}

// The blocks [b0, b1) of an item.
struct Item {
    int row, split, ctx, b0, b1;
};
__device__ __forceinline__ Item load_item(const Q8Params& A, int i) {
    Item it;
    it.row = i / A.splits;
    it.split = i - it.row * A.splits;
    it.ctx = max(0, min(__ldg(A.ctx + it.row), A.width * kSubPage));
    const int n = (it.ctx + kPageSize - 1) / kPageSize;
    it.b0 = (int)((int64_t)n * it.split / A.splits);
    it.b1 = (int)((int64_t)n * (it.split + 1) / A.splits);
    return it;
}

template <int D, int GP>
__global__ void __launch_bounds__(kQ8Threads, 1)
attention_q8_kernel(const Q8Params A, const __grid_constant__ CUtensorMap kmap,
                    const __grid_constant__ CUtensorMap vmap) {
    using C = Q8Cfg<D, GP>;
    constexpr int N = C::N, NB = C::NB, RING = C::RING;
    extern __shared__ uint8_t raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    uint8_t* psm = ring + RING * C::STAGE;     // [NB][N][128] swizzled, K-major
    uint8_t* qsm = psm + C::P_BYTES;           // [PANELS][N][ROWB] swizzled, K-major
    __shared__ uint64_t full[RING], empty[RING], s_full[NB], p_full[NB], q_full, o_full, drained;
    __shared__ uint32_t tmem_base;
    __shared__ int gave_up;
    __shared__ float2 page_scale[NB * kPagesPerBlock];   // ks * scale * log2 e, log2 vs (-inf: no page)
    __shared__ float qinv[GP];
    __shared__ float red[4][2 * GP];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (warp == 5) tmem_alloc(&tmem_base, kTmemCols);
    if (tid == 0) {
        for (int i = 0; i < RING; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < NB; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], kSoftmaxThreads);
        }
        mbar_init(&q_full, kSoftmaxThreads);
        mbar_init(&o_full, 1);
        mbar_init(&drained, 1);
        gave_up = 0;
        mbar_fence_init();
    }
    // columns of heads past G stay zero
    for (int i = tid; i < (C::P_BYTES + C::Q_BYTES) / 16; i += kQ8Threads)
        reinterpret_cast<uint4*>(psm)[i] = make_uint4(0, 0, 0, 0);
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    const int items = A.rows * A.splits;
    volatile int* quit = &gave_up;

    if (warp == 4) {
        // ------------------------------------------------ copies
        if (lane == 0) {
            tma_prefetch_map(&kmap);
            tma_prefetch_map(&vmap);
        }
        const int outside = (int)max((int64_t)1, A.num_pages) * kSubPage;   // past the tensor's end
        uint32_t n = 0;   // blocks copied so far: stage n % RING
        bool ok = true;
        for (int i = blockIdx.x; ok && i < items; i += gridDim.x) {
            const Item it = load_item(A, i);
            const int h = it.row % A.H;
            const int32_t* bt = A.bt + (int64_t)it.row * A.width;
            const int used = (it.ctx + kSubPage - 1) / kSubPage;      // pages of the context
            for (int c0 = it.b0; ok && c0 < it.b1; c0 += NB) {
                const int nb = min(NB, it.b1 - c0);
                // the chunk's page coordinates, page p of the chunk in lane p % 32
                int z[NB * kPagesPerBlock / 32];
#pragma unroll
                for (int r = 0; r < NB * kPagesPerBlock / 32; ++r) {
                    const int p = c0 * kPagesPerBlock + r * 32 + lane;
                    int pg = -1;
                    if (p < used && r * 32 + lane < nb * kPagesPerBlock) pg = __ldg(bt + p);
                    z[r] = pg >= 0 && pg < A.num_pages ? pg * kSubPage : outside;
                }
                for (int kv = 0; ok && kv < 2; ++kv) {
                    const CUtensorMap* map = kv == 0 ? &kmap : &vmap;
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        // page b * 8 + lane % 8 sits in register b / 4 of lane b % 4 * 8 + lane % 8
                        const int zc = __shfl_sync(kFull, z[b / 4], (b & 3) * 8 + (lane & 7));
                        if (b < nb && ok) {
                            const uint32_t st = n % RING;
                            ok = n < RING || mbar_wait(&empty[st], (n / RING - 1) & 1, quit);
                            ok = __all_sync(kFull, ok);
                            if (ok) {
                                if (lane == 0) mbar_expect(&full[st], C::STAGE);
                                __syncwarp();
                                if (lane < kPagesPerBlock * C::PANELS) {
                                    const int panel = lane / kPagesPerBlock;
                                    tma_load_3d(ring + st * C::STAGE + panel * C::PANEL_BYTES +
                                                    (lane & 7) * kSubPage * C::ROWB,
                                                map, panel * 128, h, zc, &full[st]);
                                }
                                ++n;
                            }
                        }
                    }
                }
            }
        }
        // the copies in flight land before the CTA's memory goes away
        if (!ok) {
            for (uint32_t k = n > RING ? n - RING : 0; k < n; ++k) {
                int none = 0;
                mbar_wait(&full[k % RING], (k / RING) & 1, &none);
            }
        }
    } else if (warp == 5) {
        // ------------------------------------------------ MMAs
        if (lane == 0) {
            constexpr uint32_t kSteps = C::ROWB / 32;
            const uint32_t q0 = smem_addr(qsm), p0 = smem_addr(psm), r0 = smem_addr(ring);
            const uint32_t o_cols = tmem + kScoreCols;
            uint32_t n = 0, items_done = 0, p_phase = 0;
            bool ok = true;
            for (int i = blockIdx.x; ok && i < items; i += gridDim.x) {
                const Item it = load_item(A, i);
                if (it.b0 == it.b1) continue;
                ok = mbar_wait(&q_full, items_done & 1, quit);
                ++items_done;
                for (int c0 = it.b0; ok && c0 < it.b1; c0 += NB) {
                    const int nb = min(NB, it.b1 - c0);
                    for (int b = 0; ok && b < nb; ++b, ++n) {
                        const uint32_t st = n % RING;
                        ok = mbar_wait(&full[st], (n / RING) & 1, quit);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int panel = 0; panel < C::PANELS; ++panel)
#pragma unroll
                            for (uint32_t k = 0; k < kSteps; ++k)
                                mma_f8(tmem + b * N,
                                       smem_desc(r0 + st * C::STAGE + panel * C::PANEL_BYTES + k * 32, 0, C::ATOM, C::SWIZZLE),
                                       smem_desc(q0 + panel * C::Q_PANEL + k * 32, 0, C::ATOM, C::SWIZZLE), A.k_idesc,
                                       panel + k > 0);
                        tc_commit(&empty[st]);
                        tc_commit(&s_full[b]);
                    }
                    for (int b = 0; ok && b < nb; ++b, ++n) {
                        const uint32_t st = n % RING;
                        ok = mbar_wait(&p_full[b], (p_phase >> b) & 1, quit) &&
                             mbar_wait(&full[st], (n / RING) & 1, quit);
                        if (!ok) break;
                        p_phase ^= 1u << b;
                        tc_fence_after();
                        // values: 32 tokens a step; the head's dimensions run along
                        // the rows.  A 64-byte row fills 64 of the 128 MMA rows;
                        // the leading offset 0 reads it again for the others.
#pragma unroll
                        for (int panel = 0; panel < C::PANELS; ++panel)
#pragma unroll
                            for (uint32_t k = 0; k < 4; ++k)
                                mma_f8(o_cols + panel * N,
                                       smem_desc(r0 + st * C::STAGE + panel * C::PANEL_BYTES + k * 32 * C::ROWB, 0,
                                                 C::ATOM, C::SWIZZLE),
                                       smem_desc(p0 + b * N * 128 + k * 32, 0, 1024, 2), A.v_idesc, b > 0 || k > 0);
                        tc_commit(&empty[st]);
                    }
                    if (ok) tc_commit(&o_full);
                }
            }
            // no MMA runs on into the release of its memory
            if (!ok) {
                int none = 0;
                tc_commit(&drained);
                mbar_wait(&drained, 0, &none);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------ softmax and output
        const uint32_t lanes = tmem + ((uint32_t)warp << 21);    // this warp's 32 TMEM lanes
        const int chunk16 = tid >> 4;                              // byte tid's 16-byte part of a P row
        uint32_t n = 0, s_phase = 0, chunks = 0;
        // These warps meet in barriers, so none leaves early: after a wait
        // that ran out they go through their loops on what there is, and
        // write NaN.
        for (int i = blockIdx.x; i < items; i += gridDim.x) {
            const Item it = load_item(A, i);
            const int h = it.row % A.H;
            const int32_t* bt = A.bt + (int64_t)it.row * A.width;
            if (tid == 0 && it.split == 0)
                report_status(A.status, __ldg(A.ctx + it.row) != it.ctx, BSA_STATUS_BAD_CONTEXT);
            float acc[C::PANELS][GP], my[GP], mt[GP], l[GP];
#pragma unroll
            for (int g = 0; g < GP; ++g) {
#pragma unroll
                for (int p = 0; p < C::PANELS; ++p) acc[p][g] = 0.f;
                my[g] = mt[g] = -INFINITY;
                l[g] = 0.f;
            }
            if (it.b0 < it.b1) {
                // the queries as two e4m3 terms
                for (int g = warp; g < A.G; g += 4) {
                    const uint16_t* q = A.q + ((int64_t)it.row * A.G + g) * D;
                    constexpr int QL = D / 32;         // values per lane, contiguous
                    float x[QL], m = 0.f;
#pragma unroll
                    for (int k = 0; k < QL; ++k) {
                        x[k] = __uint_as_float((uint32_t)__ldg(q + lane * QL + k) << 16);
                        m = fmaxf(m, fabsf(x[k]));
                    }
                    m = max_warp(m);
                    // scale by a power of two: the largest magnitude to [128, 256)
                    const int e = min(max((int)(__float_as_uint(m) >> 23) - 127, -100), 127);
                    const float up = __uint_as_float((uint32_t)(127 + 7 - e) << 23);
#pragma unroll
                    for (int k = 0; k < QL; k += 2) {
                        // an infinite query has no finite result: NaN
                        const float a = (x[k] - x[k] == 0.f) ? x[k] * up : NAN;
                        const float b = (x[k + 1] - x[k + 1] == 0.f) ? x[k + 1] * up : NAN;
                        const uint32_t hi = pack_e4m3(a, b);
                        const float2 f = unpack_e4m3(hi);
                        const uint32_t lo = pack_e4m3((a - f.x) * 16.f, (b - f.y) * 16.f);
                        const int d = lane * QL + k, panel = d / C::ROWB, dc = d % C::ROWB;
#pragma unroll
                        for (int term = 0; term < 2; ++term) {
                            const int row = term * GP + g;
                            const int sw = C::ROWB == 128 ? (row & 7) : ((row >> 1) & 3);
                            uint8_t* dst = qsm + panel * C::Q_PANEL + row * C::ROWB + (((dc >> 4) ^ sw) << 4) + (dc & 15);
                            *reinterpret_cast<uint16_t*>(dst) = (uint16_t)(term ? lo : hi);
                        }
                    }
                    if (lane == 0) qinv[g] = __uint_as_float((uint32_t)(127 - 7 + e) << 23);
                }
                for (int g = tid; g < GP; g += kSoftmaxThreads)
                    if (g >= A.G) qinv[g] = 0.f;
                fence_async_smem();
                mbar_arrive(&q_full);
            }
            for (int c0 = it.b0; c0 < it.b1; c0 += NB) {
                const int nb = min(NB, it.b1 - c0);
                softmax_sync();                  // the last chunk's page_scale and red have been read
                if (tid < nb * kPagesPerBlock) {
                    const int p = c0 * kPagesPerBlock + tid;
                    float2 sc = make_float2(0.f, -INFINITY);
                    if (p * kSubPage < it.ctx) {
                        const int32_t pg = __ldg(bt + p);
                        const bool good = pg >= 0 && pg < A.num_pages;
                        report_status(A.status, !good, BSA_STATUS_BAD_PAGE);
                        if (good) {
                            sc.x = __ldg(A.ks + (int64_t)pg * A.H + h) * A.scale_log2e;
                            sc.y = log2f(fmaxf(__ldg(A.vs + (int64_t)pg * A.H + h), 0x1p-126f));
                        }
                    }
                    page_scale[tid] = sc;
                }
                softmax_sync();
                float qi[GP];
#pragma unroll
                for (int g = 0; g < GP; ++g) qi[g] = qinv[g];
                // ---- the chunk's maxima, block by block as scores complete ----
                float cy[GP], ct[GP];
#pragma unroll
                for (int g = 0; g < GP; ++g) cy[g] = ct[g] = -INFINITY;
                for (int b = 0; b < nb; ++b) {
                    mbar_wait(&s_full[b], (s_phase >> b) & 1, quit);
                    __syncwarp();
                    tc_fence_after();
                    float s[2 * GP];
                    if constexpr (GP == 4) tmem_ld8(lanes + b * N, s);
                    else if constexpr (GP == 8) tmem_ld16(lanes + b * N, s);
                    else {
                        tmem_ld16(lanes + b * N, *reinterpret_cast<float(*)[16]>(s));
                        tmem_ld16(lanes + b * N + 16, *reinterpret_cast<float(*)[16]>(s + 16));
                    }
                    const float2 sc = page_scale[b * kPagesPerBlock + (tid >> 4)];
                    const bool live = (c0 + b) * kPageSize + tid < it.ctx && sc.y != -INFINITY;
                    if (live) {
#pragma unroll
                        for (int g = 0; g < GP; ++g) {
                            const float y = fmaf(s[GP + g], 0.0625f, s[g]) * (qi[g] * sc.x);
                            cy[g] = fmaxf(cy[g], y);
                            ct[g] = fmaxf(ct[g], y + sc.y);
                        }
                    }
                }
#pragma unroll
                for (int g = 0; g < GP; ++g) {
                    const float a = max_warp(cy[g]), t = max_warp(ct[g]);
                    if (lane == 0) {
                        red[warp][2 * g] = a;
                        red[warp][2 * g + 1] = t;
                    }
                }
                softmax_sync();
#pragma unroll
                for (int g = 0; g < GP; ++g) {
                    const float a = fmaxf(fmaxf(red[0][2 * g], red[1][2 * g]), fmaxf(red[2][2 * g], red[3][2 * g]));
                    ct[g] = fmaxf(fmaxf(red[0][2 * g + 1], red[1][2 * g + 1]),
                                  fmaxf(red[2][2 * g + 1], red[3][2 * g + 1]));
                    const float top = fmaxf(my[g], a);
                    l[g] *= top == -INFINITY ? 1.f : ex2(my[g] - top);
                    my[g] = top;
                }
                // ---- the probabilities ----
                for (int b = 0; b < nb; ++b) {
                    float s[2 * GP];
                    if constexpr (GP == 4) tmem_ld8(lanes + b * N, s);
                    else if constexpr (GP == 8) tmem_ld16(lanes + b * N, s);
                    else {
                        tmem_ld16(lanes + b * N, *reinterpret_cast<float(*)[16]>(s));
                        tmem_ld16(lanes + b * N + 16, *reinterpret_cast<float(*)[16]>(s + 16));
                    }
                    const float2 sc = page_scale[b * kPagesPerBlock + (tid >> 4)];
                    const int left = it.ctx - (c0 + b) * kPageSize;       // context tokens from this block on
                    const bool live = tid < left && sc.y != -INFINITY;
                    float w[GP];
#pragma unroll
                    for (int g = 0; g < GP; ++g) {
                        const float y = fmaf(s[GP + g], 0.0625f, s[g]) * (qi[g] * sc.x);
                        l[g] += live ? ex2(y - my[g]) : 0.f;
                        w[g] = live ? ex2(y + sc.y - ct[g] + 8.f) : 0.f;
                    }
                    uint8_t* pb = psm + b * N * 128 + (tid & 15);
#pragma unroll
                    for (int g = 0; g < GP; g += 2) {
                        const uint32_t hi = pack_e4m3(w[g], w[g + 1]);
                        const float2 f = unpack_e4m3(hi);
                        const uint32_t lo = pack_e4m3((w[g] - f.x) * 16.f, (w[g + 1] - f.y) * 16.f);
                        const int r0 = g, r1 = g + 1, r2 = GP + g, r3 = GP + g + 1;
                        pb[r0 * 128 + ((chunk16 ^ (r0 & 7)) << 4)] = (uint8_t)hi;
                        pb[r1 * 128 + ((chunk16 ^ (r1 & 7)) << 4)] = (uint8_t)(hi >> 8);
                        pb[r2 * 128 + ((chunk16 ^ (r2 & 7)) << 4)] = (uint8_t)lo;
                        pb[r3 * 128 + ((chunk16 ^ (r3 & 7)) << 4)] = (uint8_t)(lo >> 8);
                    }
                    if (left < kPageSize) {
                        // the last block: no value behind the context's end
                        const uint32_t k = n + nb + b, st = k % RING;
                        mbar_wait(&full[st], (k / RING) & 1, quit);
                        if (tid >= left) {
#pragma unroll
                            for (int x = 0; x < D / 16; ++x)
                                *reinterpret_cast<uint4*>(ring + st * C::STAGE + (x * 16 / C::ROWB) * C::PANEL_BYTES +
                                                          tid * C::ROWB + (x * 16 % C::ROWB)) = make_uint4(0, 0, 0, 0);
                        }
                        __syncwarp();
                    }
                    fence_async_smem();
                    tc_fence_before();
                    mbar_arrive(&p_full[b]);
                }
                s_phase ^= (1u << nb) - 1;
                n += 2 * nb;
                // ---- the chunk's outputs join the item's ----
                mbar_wait(&o_full, chunks & 1, quit);
                __syncwarp();
                ++chunks;
                tc_fence_after();
                float keep[GP], add[GP];
#pragma unroll
                for (int g = 0; g < GP; ++g) {
                    const float top = fmaxf(mt[g], ct[g]);
                    keep[g] = top == -INFINITY ? 1.f : ex2(mt[g] - top);
                    add[g] = top == -INFINITY ? 0.f : ex2(ct[g] - top);
                    mt[g] = top;
                }
#pragma unroll
                for (int p = 0; p < C::PANELS; ++p) {
                    float s[2 * GP];
                    const uint32_t at = lanes + kScoreCols + p * N;
                    if constexpr (GP == 4) tmem_ld8(at, s);
                    else if constexpr (GP == 8) tmem_ld16(at, s);
                    else {
                        tmem_ld16(at, *reinterpret_cast<float(*)[16]>(s));
                        tmem_ld16(at + 16, *reinterpret_cast<float(*)[16]>(s + 16));
                    }
#pragma unroll
                    for (int g = 0; g < GP; ++g)
                        acc[p][g] = acc[p][g] * keep[g] + fmaf(s[GP + g], 0.0625f, s[g]) * add[g];
                }
                tc_fence_before();
            }
            // ---- the item's result: the sums over the four warps' tokens ----
            softmax_sync();
#pragma unroll
            for (int g = 0; g < GP; ++g) {
                const float a = sum_warp(l[g]);
                if (lane == 0) red[warp][g] = a;
            }
            softmax_sync();
            if (A.part == nullptr) {
                uint16_t* o = A.out + (int64_t)it.row * A.G * D;
#pragma unroll
                for (int g = 0; g < GP; ++g) {
                    if (g >= A.G) break;
                    float sum = red[0][g] + red[1][g] + red[2][g] + red[3][g];
                    if (*quit) sum = NAN;
                    const float f = sum == 0.f ? 0.f : ex2(mt[g] - my[g] - 8.f) / sum;
#pragma unroll
                    for (int p = 0; p < C::PANELS; ++p)
                        if (tid < C::ROWB)
                            o[g * D + p * 128 + tid] =
                                __bfloat16_as_ushort(__float2bfloat16_rn(sum == 0.f ? 0.f : acc[p][g] * f));
                }
            } else {
                float* o = A.part + (int64_t)i * part_floats(A.G, D);
#pragma unroll
                for (int g = 0; g < GP; ++g) {
                    if (g >= A.G) break;
#pragma unroll
                    for (int p = 0; p < C::PANELS; ++p)
                        if (tid < C::ROWB) o[g * D + p * 128 + tid] = acc[p][g];
                    if (tid == 0) {
                        o[A.G * D + g] = my[g];
                        o[A.G * D + A.G + g] = mt[g];
                        o[A.G * D + 2 * A.G + g] =
                            *quit ? NAN : red[0][g] + red[1][g] + red[2][g] + red[3][g];
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0) report_status(A.status, gave_up != 0, BSA_STATUS_TIMEOUT);
    if (warp == 5) tmem_free(tmem, kTmemCols);
}

// Joins the partial results of a split row: one CTA per row.
__global__ void __launch_bounds__(256)
attention_q8_join_kernel(const float* part, uint16_t* out, int splits, int G, int D) {
    const int64_t row = blockIdx.x;
    const int64_t len = part_floats(G, D);
    const float* base = part + row * splits * len;
    for (int i = threadIdx.x; i < G * D; i += 256) {
        const int g = i / D;
        float my = -INFINITY, mt = -INFINITY;
        for (int s = 0; s < splits; ++s) {
            my = fmaxf(my, base[s * len + G * D + g]);
            mt = fmaxf(mt, base[s * len + G * D + G + g]);
        }
        float sum = 0.f, o = 0.f;
        for (int s = 0; s < splits; ++s) {
            const float l = base[s * len + G * D + 2 * G + g];
            if (l == 0.f) continue;
            sum += l * ex2(base[s * len + G * D + g] - my);
            o += base[s * len + i] * ex2(base[s * len + G * D + G + g] - mt);
        }
        out[row * G * D + i] =
            __bfloat16_as_ushort(__float2bfloat16_rn(sum == 0.f ? 0.f : o * (ex2(mt - my - 8.f) / sum)));
    }
}

// ---- host ------------------------------------------------------------------

using EncodeFn = decltype(&cuTensorMapEncodeTiled);

EncodeFn encode_fn() {
    static EncodeFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) == cudaSuccess &&
            r == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeFn>(p);
    });
    return fn;
}

// The cache as a tensor of (dimension, head, token) bytes, read in boxes of
// one page of one head (128 bytes of it at most).
bool encode_cache(CUtensorMap* map, const void* base, int64_t tokens, int64_t H, int64_t D) {
    const EncodeFn fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)D, (cuuint64_t)(H * D)};
    const cuuint32_t box[3] = {(cuuint32_t)(D < 128 ? D : 128), 1, (cuuint32_t)kSubPage};
    const cuuint32_t unit[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, unit,
              CU_TENSOR_MAP_INTERLEAVE_NONE, D < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int GP>
cudaError_t launch_q8(Q8Params& A, const CUtensorMap& km, const CUtensorMap& vm, bool e4m3, int sms, cudaStream_t st) {
    using C = Q8Cfg<D, GP>;
    const uint32_t fmt = e4m3 ? 0 : 1;
    A.k_idesc = f8_idesc(fmt, 0, false, 128, C::N);
    A.v_idesc = f8_idesc(fmt, 0, true, 128, C::N);
    auto kern = attention_q8_kernel<D, GP>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    const int64_t items = (int64_t)A.rows * A.splits;
    kern<<<(unsigned)(items < sms ? items : sms), kQ8Threads, C::SMEM, st>>>(A, km, vm);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_q8_g(Q8Params& A, const CUtensorMap& km, const CUtensorMap& vm, bool e4m3, int sms, cudaStream_t st) {
    if (A.G <= 4) return launch_q8<D, 4>(A, km, vm, e4m3, sms, st);
    if (A.G <= 8) return launch_q8<D, 8>(A, km, vm, e4m3, sms, st);
    return launch_q8<D, 16>(A, km, vm, e4m3, sms, st);
}

bool sizes_ok(int64_t T, int64_t H, int64_t G, int64_t D) {
    return T >= 0 && T <= INT32_MAX && H >= 1 && H <= 65536 && T * H <= (1 << 24) && G >= 1 &&
           G <= BSA_MAX_ATTN_Q8_GROUP && (D == 64 || D == 128 || D == 256);
}

// Items per row: the count with the least work on the longest CTA, a
// block's copy against an item's fixed cost and the joining launch.
int pick_splits(int64_t rows, int64_t D, int32_t K, int sms) {
    int best = 1;
    double least = 0;
    for (int s = 1; s <= K; ++s) {
        const int64_t waves = (rows * s + sms - 1) / sms;
        const double us = waves * ((K + s - 1) / s * (D / 128.0) * 0.75 + 1.5) + (s > 1 ? 3.0 + 0.02 * s : 0.0);
        if (s == 1 || us < least) {
            best = s;
            least = us;
        }
        if (waves > 8) break;      // enough items to even out
    }
    return best;
}

size_t workspace_need(int64_t rows, int64_t G, int64_t D, int splits) {
    return splits > 1 ? (size_t)(rows * splits * part_floats((int)G, (int)D)) * sizeof(float) : 0;
}

}  // namespace
}  // namespace bsa

using namespace bsa;

extern "C" size_t bsa_attention_q8_workspace_bytes(int64_t T, int64_t H, int64_t G, int64_t D, int32_t K) {
    if (!sizes_ok(T, H, G, D) || T == 0 || K < 1 || K > BSA_MAX_TOPK) return 0;
    return workspace_need(T * H, G, D, pick_splits(T * H, D, K, device_sm_count()));
}

extern "C" int bsa_sparse_decode_attention_q8(const void* q, const void* k_cache, const void* v_cache,
                                              int32_t cache_dtype, const float* k_scale,
                                              const float* v_scale, int64_t num_pages,
                                              const int32_t* sparse_bt, const int32_t* sparse_ctx,
                                              int64_t T, int64_t H, int64_t G, int64_t D, int32_t K,
                                              float scale, void* out, void* workspace,
                                              size_t workspace_bytes, void* stream) {
    if (cache_dtype != BSA_DTYPE_E4M3 && cache_dtype != BSA_DTYPE_E5M2) return BSA_ERR_DTYPE;
    if (!sizes_ok(T, H, G, D) || num_pages < 0 || num_pages >= (1ll << 27)) return BSA_ERR_SHAPE;
    if (K < 1 || K > BSA_MAX_TOPK) return BSA_ERR_TOPK;
    if (T == 0) return BSA_OK;
    if (q == nullptr || sparse_bt == nullptr || sparse_ctx == nullptr || out == nullptr ||
        (num_pages > 0 && (k_cache == nullptr || v_cache == nullptr || k_scale == nullptr || v_scale == nullptr)))
        return BSA_ERR_NULL;
    const void* wide[4] = {q, k_cache, v_cache, out};
    for (const void* p : wide)
        if ((reinterpret_cast<uintptr_t>(p) & 15) != 0) return BSA_ERR_ALIGN;
    const int sms = device_sm_count();
    Q8Params A{};
    A.q = static_cast<const uint16_t*>(q);
    A.ks = k_scale;
    A.vs = v_scale;
    A.bt = sparse_bt;
    A.ctx = sparse_ctx;
    A.out = static_cast<uint16_t*>(out);
    A.num_pages = num_pages;
    A.rows = (int32_t)(T * H);
    A.H = (int32_t)H;
    A.G = (int32_t)G;
    A.width = K * kPagesPerBlock;
    A.splits = pick_splits(T * H, D, K, sms);
    A.scale_log2e = scale * 1.44269504f;
    A.status = current_status_word();
    if (A.splits > 1) {
        if (workspace == nullptr || workspace_bytes < workspace_need(A.rows, G, D, A.splits) ||
            (reinterpret_cast<uintptr_t>(workspace) & 255) != 0)
            return BSA_ERR_WORKSPACE;
        A.part = static_cast<float*>(workspace);
    }
    // an empty cache: no box lies inside, any address serves
    CUtensorMap km, vm;
    const int64_t tokens = (num_pages > 0 ? num_pages : 1) * kSubPage;
    if (!encode_cache(&km, num_pages > 0 ? k_cache : q, tokens, H, D) ||
        !encode_cache(&vm, num_pages > 0 ? v_cache : q, tokens, H, D))
        return (int)cudaErrorInvalidValue;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool e4m3 = cache_dtype == BSA_DTYPE_E4M3;
    cudaError_t e;
    if (D == 64) e = launch_q8_g<64>(A, km, vm, e4m3, sms, st);
    else if (D == 128) e = launch_q8_g<128>(A, km, vm, e4m3, sms, st);
    else e = launch_q8_g<256>(A, km, vm, e4m3, sms, st);
    if (e == cudaSuccess && A.splits > 1) {
        attention_q8_join_kernel<<<(unsigned)A.rows, 256, 0, st>>>(A.part, A.out, A.splits, A.G, (int)D);
        e = cudaGetLastError();
    }
    return e == cudaSuccess ? BSA_OK : (int)e;
}
