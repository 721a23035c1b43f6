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
// The work: a CTA takes items (a row, or a share of its 128-token blocks when
// rows are few) and walks each in chunks of as many blocks as their scores
// fit in 192 TMEM columns (12 blocks up to 8 query heads, 6 up to 16).  A
// chunk's scores are complete before its probabilities are formed, so there
// is one maximum per chunk and no correction of accumulators in TMEM.
//  warps 0-3  thread i is token i of a block (probabilities) and dimension i
//             of the head (output),
//  warp 4     copies blocks by TMA into a ring of shared-memory stages: the
//             chunk's key blocks, then its value blocks, a box per page;
//             pages outside the context or the cache are boxes past the end
//             of the tensor, which arrive as zeros,
//  warp 5     issues the MMAs and frees the stages,
//  warp 6     reads the next chunk's page scales and the next item's queries.
// Two CTAs share an SM, so that one's copies and MMAs run through the other's
// softmax.  Values behind the context's end in its last page are set to zero
// in shared memory (they may be NaN codes); such keys only reach their own
// scores.  The kernel is bound by the copies: 2 D bytes a token.
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
constexpr int kQ8Threads = kSoftmaxThreads + 96;
constexpr int kQ8Ctas = 2;               // per SM
constexpr int kScoreCols = 192;          // TMEM columns of a chunk's scores
constexpr int kTmemCols = 256;
constexpr int kQ8Smem = 115712;          // half an SM's shared memory, less 1 KB a CTA

template <int D, int GP>
struct Q8Cfg {
    static constexpr int N = GP <= 8 ? 16 : 32;       // MMA columns: two terms of each head
    static constexpr int NB = kScoreCols / N;         // blocks per chunk
    static constexpr int PANELS = D == 256 ? 2 : 1;   // 128-byte parts of a head's row
    static constexpr int ROWB = D / PANELS;           // bytes of a row in a panel: 64 or 128
    static constexpr int STAGE = 128 * ROWB;          // a panel of a block: 8 or 16 KB
    static constexpr int P_BYTES = NB * N * 128;      // 24 KB
    static constexpr int Q_PANEL = N * ROWB;
    static constexpr int Q_BYTES = PANELS * Q_PANEL;
    static constexpr int PAGES = NB * kPagesPerBlock;
    static constexpr int STATIC = 2 * PAGES * 16 + 1280;   // scales, barriers and the rest
    static constexpr int RING = (kQ8Smem - STATIC - 1024 - P_BYTES - 2 * Q_BYTES) / STAGE;
    static constexpr int SMEM = RING * STAGE + P_BYTES + 2 * Q_BYTES + 1024;
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
// weighted score and the sum
__host__ __device__ inline int64_t part_floats(int G, int D) { return (int64_t)G * D + 2 * G; }

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

// The blocks [b0, b1) of an item, and how it is cut into chunks of at most NB
// blocks of even size.
struct Item {
    int row, split, ctx, b0, b1, step;
};
template <int NB>
__device__ __forceinline__ Item load_item(const Q8Params& A, int i) {
    Item it;
    it.row = i / A.splits;
    it.split = i - it.row * A.splits;
    it.ctx = max(0, min(__ldg(A.ctx + it.row), A.width * kSubPage));
    const int n = (it.ctx + kPageSize - 1) / kPageSize;
    it.b0 = (int)((int64_t)n * it.split / A.splits);
    it.b1 = (int)((int64_t)n * (it.split + 1) / A.splits);
    const int len = it.b1 - it.b0;
    const int chunks = (len + NB - 1) / NB;
    it.step = chunks > 0 ? (len + chunks - 1) / chunks : 1;
    return it;
}

// A chunk as warp 6 hands it on.
struct Chunk {
    int row, ctx, c0, nb;    // nb < 0: no more
    int item, qbuf, first, last;
};

template <int GP>
__device__ __forceinline__ void load_cols(uint32_t addr, float (&s)[2 * GP]) {
    if constexpr (GP == 4) tmem_ld8(addr, s);
    else if constexpr (GP == 8) tmem_ld16(addr, s);
    else {
        tmem_ld16(addr, *reinterpret_cast<float(*)[16]>(s));
        tmem_ld16(addr + 16, *reinterpret_cast<float(*)[16]>(s + 16));
    }
}

template <int D, int GP>
__global__ void __launch_bounds__(kQ8Threads, kQ8Ctas)
attention_q8_kernel(const Q8Params A, const __grid_constant__ CUtensorMap kmap,
                    const __grid_constant__ CUtensorMap vmap) {
    using C = Q8Cfg<D, GP>;
    constexpr int N = C::N, NB = C::NB, RING = C::RING, PANELS = C::PANELS;
    extern __shared__ uint8_t raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    uint8_t* psm = ring + RING * C::STAGE;     // [NB][N][128] swizzled, K-major
    uint8_t* qsm = psm + C::P_BYTES;           // [2][PANELS][N][ROWB] swizzled, K-major
    // ks * scale * log2 e, log2 vs (-inf: no page), 1 / vs of the pages of two chunks
    __shared__ float4 page_scale[2][C::PAGES];
    __shared__ uint64_t full[RING], empty[RING], s_full[NB], p_full[NB], c_full[2], c_empty[2], o_full, drained;
    __shared__ Chunk chunk[2];
    __shared__ float qinv[2][GP];
    __shared__ float red[4][GP];
    __shared__ uint32_t tmem_base;
    __shared__ int gave_up;
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
        for (int i = 0; i < 2; ++i) {
            mbar_init(&c_full[i], 32);
            mbar_init(&c_empty[i], kSoftmaxThreads);
        }
        mbar_init(&o_full, 1);
        mbar_init(&drained, 1);
        gave_up = 0;
        mbar_fence_init();
    }
    // columns of heads past G stay zero
    for (int i = tid; i < (C::P_BYTES + 2 * C::Q_BYTES) / 16; i += kQ8Threads)
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
        uint32_t n = 0;   // panels copied so far: stage n % RING
        bool ok = true;
        for (int i = blockIdx.x; ok && i < items; i += gridDim.x) {
            const Item it = load_item<NB>(A, i);
            const int h = it.row % A.H;
            const int32_t* bt = A.bt + (int64_t)it.row * A.width;
            const int used = (it.ctx + kSubPage - 1) / kSubPage;      // pages of the context
            for (int c0 = it.b0; ok && c0 < it.b1; c0 += it.step) {
                const int nb = min(it.step, it.b1 - c0);
                // the chunk's page coordinates, page p of the chunk in lane p % 32
                int z[(C::PAGES + 31) / 32];
#pragma unroll
                for (int r = 0; r < (C::PAGES + 31) / 32; ++r) {
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
                        if (b < nb) {
#pragma unroll
                            for (int panel = 0; panel < PANELS; ++panel) {
                                if (!ok) break;
                                const uint32_t st = n % RING;
                                ok = n < RING || mbar_wait(&empty[st], (n / RING - 1) & 1, quit);
                                ok = __all_sync(kFull, ok);
                                if (!ok) break;
                                if (lane == 0) mbar_expect(&full[st], C::STAGE);
                                __syncwarp();
                                if (lane < kPagesPerBlock)
                                    tma_load_3d(ring + st * C::STAGE + lane * kSubPage * C::ROWB, map, panel * 128, h,
                                                zc, &full[st]);
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
            uint32_t n = 0, p_phase = 0;
            bool ok = true;
            for (uint32_t c = 0; ok; ++c) {
                ok = mbar_wait(&c_full[c & 1], (c >> 1) & 1, quit);
                if (!ok) break;
                const int nb = chunk[c & 1].nb;
                if (nb < 0) break;
                const uint32_t qb = q0 + chunk[c & 1].qbuf * C::Q_BYTES;
                for (int b = 0; ok && b < nb; ++b) {
#pragma unroll
                    for (int panel = 0; panel < PANELS; ++panel, ++n) {
                        const uint32_t st = n % RING;
                        ok = ok && mbar_wait(&full[st], (n / RING) & 1, quit);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (uint32_t k = 0; k < kSteps; ++k)
                            mma_f8(tmem + b * N, smem_desc(r0 + st * C::STAGE + k * 32, 0, C::ATOM, C::SWIZZLE),
                                   smem_desc(qb + panel * C::Q_PANEL + k * 32, 0, C::ATOM, C::SWIZZLE), A.k_idesc,
                                   panel + k > 0);
                        tc_commit(&empty[st]);
                    }
                    if (ok) tc_commit(&s_full[b]);
                }
                for (int b = 0; ok && b < nb; ++b) {
                    ok = mbar_wait(&p_full[b], (p_phase >> b) & 1, quit);
                    p_phase ^= 1u << b;
#pragma unroll
                    for (int panel = 0; panel < PANELS; ++panel, ++n) {
                        const uint32_t st = n % RING;
                        ok = ok && mbar_wait(&full[st], (n / RING) & 1, quit);
                        if (!ok) break;
                        tc_fence_after();
                        // values: 32 tokens a step; the head's dimensions run along
                        // the rows.  A 64-byte row fills 64 of the 128 MMA rows;
                        // the leading offset 0 reads it again for the others.
#pragma unroll
                        for (uint32_t k = 0; k < 4; ++k)
                            mma_f8(o_cols + panel * N,
                                   smem_desc(r0 + st * C::STAGE + k * 32 * C::ROWB, 0, C::ATOM, C::SWIZZLE),
                                   smem_desc(p0 + b * N * 128 + k * 32, 0, 1024, 2), A.v_idesc, b > 0 || k > 0);
                        tc_commit(&empty[st]);
                    }
                }
                if (ok && nb > 0) tc_commit(&o_full);
            }
            // no MMA runs on into the release of its memory
            if (!ok) {
                int none = 0;
                tc_commit(&drained);
                mbar_wait(&drained, 0, &none);
            }
        }
        __syncwarp();
    } else if (warp == 6) {
        // ------------------------------------------------ scales and queries
        uint32_t c = 0;
        int qbuf = 0;
        bool ok = true;
        for (int i = blockIdx.x; ok && i < items; i += gridDim.x) {
            const Item it = load_item<NB>(A, i);
            const int h = it.row % A.H;
            const int32_t* bt = A.bt + (int64_t)it.row * A.width;
            if (lane == 0 && it.split == 0)
                report_status(A.status, __ldg(A.ctx + it.row) != it.ctx, BSA_STATUS_BAD_CONTEXT);
            int c0 = it.b0;
            do {
                const int nb = min(it.step, it.b1 - c0);
                const int buf = c & 1;
                ok = c < 2 || mbar_wait(&c_empty[buf], ((c >> 1) - 1) & 1, quit);
                ok = __all_sync(kFull, ok);
                if (!ok) break;
#pragma unroll
                for (int r = 0; r < (C::PAGES + 31) / 32; ++r) {
                    const int p = r * 32 + lane;
                    if (p >= nb * kPagesPerBlock) continue;
                    float4 sc = make_float4(0.f, -INFINITY, 0.f, 0.f);
                    if ((c0 * kPagesPerBlock + p) * kSubPage < it.ctx) {
                        const int32_t pg = __ldg(bt + c0 * kPagesPerBlock + p);
                        const bool good = pg >= 0 && pg < A.num_pages;
                        report_status(A.status, !good, BSA_STATUS_BAD_PAGE);
                        if (good) {
                            const float vs = fmaxf(__ldg(A.vs + (int64_t)pg * A.H + h), 0x1p-100f);
                            sc = make_float4(__ldg(A.ks + (int64_t)pg * A.H + h) * A.scale_log2e, log2f(vs),
                                             __frcp_rn(vs), 0.f);
                        }
                    }
                    page_scale[buf][p] = sc;
                }
                if (c0 == it.b0 && nb > 0) {
                    // the queries as two e4m3 terms
                    qbuf ^= 1;
                    uint8_t* qd = qsm + qbuf * C::Q_BYTES;
                    constexpr int QL = D / 32;         // values per lane, contiguous
                    const int d = lane * QL, panel = d / C::ROWB, dc = d % C::ROWB;
#pragma unroll 4
                    for (int g = 0; g < A.G; ++g) {
                        const uint16_t* q = A.q + ((int64_t)it.row * A.G + g) * D + d;
                        uint32_t w[QL / 2];
                        if constexpr (QL == 2) w[0] = __ldg(reinterpret_cast<const unsigned*>(q));
                        else if constexpr (QL == 4) {
                            const uint2 v = __ldg(reinterpret_cast<const uint2*>(q));
                            w[0] = v.x, w[1] = v.y;
                        } else {
                            const uint4 v = __ldg(reinterpret_cast<const uint4*>(q));
                            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
                        }
                        float x[QL], m = 0.f;
#pragma unroll
                        for (int k = 0; k < QL; ++k) {
                            x[k] = __uint_as_float(k & 1 ? w[k / 2] & 0xFFFF0000u : w[k / 2] << 16);
                            m = fmaxf(m, fabsf(x[k]));
                        }
                        m = max_warp(m);
                        // scale by a power of two: the largest magnitude to [128, 256)
                        const int e = min(max((int)(__float_as_uint(m) >> 23) - 127, -100), 127);
                        const float up = __uint_as_float((uint32_t)(127 + 7 - e) << 23);
                        uint32_t hi[QL / 2], lo[QL / 2];
#pragma unroll
                        for (int k = 0; k < QL; k += 2) {
                            // an infinite query has no finite result: NaN
                            const float a = (x[k] - x[k] == 0.f) ? x[k] * up : NAN;
                            const float b = (x[k + 1] - x[k + 1] == 0.f) ? x[k + 1] * up : NAN;
                            hi[k / 2] = pack_e4m3(a, b);
                            const float2 f = unpack_e4m3(hi[k / 2]);
                            lo[k / 2] = pack_e4m3((a - f.x) * 16.f, (b - f.y) * 16.f);
                        }
#pragma unroll
                        for (int term = 0; term < 2; ++term) {
                            const uint32_t* v = term ? lo : hi;
                            const int row = term * GP + g;
                            const int sw = C::ROWB == 128 ? (row & 7) : ((row >> 1) & 3);
                            uint8_t* dst = qd + panel * C::Q_PANEL + row * C::ROWB + (((dc >> 4) ^ sw) << 4) + (dc & 15);
                            if constexpr (QL == 2) *reinterpret_cast<uint16_t*>(dst) = (uint16_t)v[0];
                            else if constexpr (QL == 4) *reinterpret_cast<uint32_t*>(dst) = v[0] | v[1] << 16;
                            else *reinterpret_cast<uint2*>(dst) = make_uint2(v[0] | v[1] << 16, v[2] | v[3] << 16);
                        }
                        if (lane == 0) qinv[qbuf][g] = __uint_as_float((uint32_t)(127 - 7 + e) << 23);
                    }
                    if (lane >= A.G && lane < GP) qinv[qbuf][lane] = 0.f;
                }
                if (lane == 0)
                    chunk[buf] = Chunk{it.row, it.ctx, c0, nb, i, qbuf, c0 == it.b0, c0 + nb == it.b1};
                fence_async_smem();
                mbar_arrive(&c_full[buf]);
                ++c;
                c0 += it.step;
            } while (c0 < it.b1);
        }
        if (ok) ok = c < 2 || mbar_wait(&c_empty[c & 1], ((c >> 1) - 1) & 1, quit);
        __syncwarp();
        if (lane == 0) chunk[c & 1].nb = -1;
        __syncwarp();
        mbar_arrive(&c_full[c & 1]);
    } else {
        // ------------------------------------------------ softmax and output
        const uint32_t lanes = tmem + ((uint32_t)warp << 21);    // this warp's 32 TMEM lanes
        const int part16 = tid >> 4;                               // byte tid's 16-byte part of a P row
        uint32_t n = 0, s_phase = 0, o_phase = 0;
        float acc[PANELS][GP], mt[GP], l[GP];
        // These warps meet in barriers, so none leaves alone: a wait that ran
        // out anywhere ends at the next chunk for all, or lets the loops go on
        // with what there is; outputs are NaN then.
        for (uint32_t c = 0;; ++c) {
            mbar_wait(&c_full[c & 1], (c >> 1) & 1, quit);
            softmax_sync();                  // also: red has been read
            const bool gone = *quit;
            const Chunk ch = chunk[c & 1];
            int stop = gone || ch.nb < 0;
            // one answer for the four warps
            asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %0, 0;\n\tbar.red.or.pred q, 1, 128, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
                         : "+r"(stop)::"memory");
            if (stop) break;
            const float4* scales = page_scale[c & 1];
            const int nb = ch.nb;
            if (ch.first) {
#pragma unroll
                for (int g = 0; g < GP; ++g) {
#pragma unroll
                    for (int p = 0; p < PANELS; ++p) acc[p][g] = 0.f;
                    mt[g] = -INFINITY;
                    l[g] = 0.f;
                }
            }
            if (nb > 0) {
                float qi[GP], ct[GP];
#pragma unroll
                for (int g = 0; g < GP; ++g) {
                    qi[g] = qinv[ch.qbuf][g];
                    ct[g] = -INFINITY;
                }
                // ---- the chunk's maxima, block by block as scores complete ----
                for (int b = 0; b < nb; ++b) {
                    mbar_wait(&s_full[b], (s_phase >> b) & 1, quit);
                    __syncwarp();
                    tc_fence_after();
                    float s[2 * GP];
                    load_cols<GP>(lanes + b * N, s);
                    const float4 sc = scales[b * kPagesPerBlock + part16];
                    const bool live = (ch.c0 + b) * kPageSize + tid < ch.ctx && sc.y != -INFINITY;
                    if (live) {
#pragma unroll
                        for (int g = 0; g < GP; ++g)
                            ct[g] = fmaxf(ct[g], fmaf(fmaf(s[GP + g], 0.0625f, s[g]), qi[g] * sc.x, sc.y));
                    }
                }
#pragma unroll
                for (int g = 0; g < GP; ++g) {
                    const float t = max_warp(ct[g]);
                    if (lane == 0) red[warp][g] = t;
                }
                softmax_sync();
                float keep[GP], add[GP];
#pragma unroll
                for (int g = 0; g < GP; ++g) {
                    ct[g] = fmaxf(fmaxf(red[0][g], red[1][g]), fmaxf(red[2][g], red[3][g]));
                    const float top = fmaxf(mt[g], ct[g]);
                    keep[g] = top == -INFINITY ? 1.f : ex2(mt[g] - top);
                    add[g] = top == -INFINITY ? 0.f : ex2(ct[g] - top);
                    mt[g] = top;
                    l[g] *= keep[g];
                    ct[g] = 8.f - ct[g];         // probabilities in units of 2^-8 of the largest
                }
                // ---- the probabilities ----
                for (int b = 0; b < nb; ++b) {
                    float s[2 * GP];
                    load_cols<GP>(lanes + b * N, s);
                    const float4 sc = scales[b * kPagesPerBlock + part16];
                    const int left = ch.ctx - (ch.c0 + b) * kPageSize;       // context tokens from this block on
                    const bool live = tid < left && sc.y != -INFINITY;
                    float w[GP];
#pragma unroll
                    for (int g = 0; g < GP; ++g) {
                        const float t = fmaf(fmaf(s[GP + g], 0.0625f, s[g]), qi[g] * sc.x, sc.y + ct[g]);
                        w[g] = live ? ex2(t) : 0.f;
                        l[g] = fmaf(w[g] * sc.z, add[g], l[g]);
                    }
                    uint8_t* pb = psm + b * N * 128 + (tid & 15);
#pragma unroll
                    for (int g = 0; g < GP; g += 2) {
                        const uint32_t hi = pack_e4m3(w[g], w[g + 1]);
                        const float2 f = unpack_e4m3(hi);
                        const uint32_t lo = pack_e4m3((w[g] - f.x) * 16.f, (w[g + 1] - f.y) * 16.f);
                        const int r0 = g, r1 = g + 1, r2 = GP + g, r3 = GP + g + 1;
                        pb[r0 * 128 + ((part16 ^ (r0 & 7)) << 4)] = (uint8_t)hi;
                        pb[r1 * 128 + ((part16 ^ (r1 & 7)) << 4)] = (uint8_t)(hi >> 8);
                        pb[r2 * 128 + ((part16 ^ (r2 & 7)) << 4)] = (uint8_t)lo;
                        pb[r3 * 128 + ((part16 ^ (r3 & 7)) << 4)] = (uint8_t)(lo >> 8);
                    }
                    if (left < kPageSize) {
                        // the last block: no value behind the context's end
#pragma unroll
                        for (int panel = 0; panel < PANELS; ++panel) {
                            const uint32_t k = n + (nb + b) * PANELS + panel, st = k % RING;
                            mbar_wait(&full[st], (k / RING) & 1, quit);
                            if (tid >= left) {
#pragma unroll
                                for (int x = 0; x < C::ROWB / 16; ++x)
                                    *reinterpret_cast<uint4*>(ring + st * C::STAGE + tid * C::ROWB + x * 16) =
                                        make_uint4(0, 0, 0, 0);
                            }
                        }
                        __syncwarp();
                    }
                    fence_async_smem();
                    tc_fence_before();
                    mbar_arrive(&p_full[b]);
                }
                s_phase ^= (1u << nb) - 1;
                n += 2 * nb * PANELS;
                // ---- the chunk's outputs join the item's ----
                mbar_wait(&o_full, o_phase, quit);
                __syncwarp();
                o_phase ^= 1;
                tc_fence_after();
#pragma unroll
                for (int p = 0; p < PANELS; ++p) {
                    float s[2 * GP];
                    load_cols<GP>(lanes + kScoreCols + p * N, s);
#pragma unroll
                    for (int g = 0; g < GP; ++g)
                        acc[p][g] = acc[p][g] * keep[g] + fmaf(s[GP + g], 0.0625f, s[g]) * add[g];
                }
                tc_fence_before();
            }
            if (ch.last) {
                // ---- the item's result: the sums over the four warps' tokens ----
                softmax_sync();
#pragma unroll
                for (int g = 0; g < GP; ++g) {
                    const float a = sum_warp(l[g]);
                    if (lane == 0) red[warp][g] = a;
                }
                softmax_sync();
                const bool bad = *quit;
                uint16_t* o16 = A.out + (int64_t)ch.row * A.G * D;
                float* o32 = A.part + (int64_t)ch.item * part_floats(A.G, D);
#pragma unroll
                for (int g = 0; g < GP; ++g) {
                    if (g >= A.G) break;
                    const float sum = bad ? NAN : red[0][g] + red[1][g] + red[2][g] + red[3][g];
                    if (A.part == nullptr) {
                        const float f = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
                        for (int p = 0; p < PANELS; ++p)
                            if (tid < C::ROWB)
                                o16[g * D + p * 128 + tid] =
                                    __bfloat16_as_ushort(__float2bfloat16_rn(sum == 0.f ? 0.f : acc[p][g] * f));
                    } else {
#pragma unroll
                        for (int p = 0; p < PANELS; ++p)
                            if (tid < C::ROWB) o32[g * D + p * 128 + tid] = acc[p][g];
                        if (tid == 0) {
                            o32[A.G * D + g] = mt[g];
                            o32[A.G * D + A.G + g] = sum;
                        }
                    }
                }
            }
            mbar_arrive(&c_empty[c & 1]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0) report_status(A.status, gave_up != 0, BSA_STATUS_TIMEOUT);
    if (warp == 5) tmem_free(tmem, kTmemCols);
}

// Joins the partial results of a split row, head by head: a thread per
// dimension.
__global__ void __launch_bounds__(256)
attention_q8_join_kernel(const float* __restrict__ part, uint16_t* __restrict__ out, int splits, int G, int D) {
    extern __shared__ float weight[];          // [splits]
    __shared__ float total[2];
    const int64_t row = blockIdx.x;
    const int g = blockIdx.y, tid = threadIdx.x;
    const int64_t len = part_floats(G, D);
    const float* base = part + row * splits * len;
    if (tid < 32) {
        float m = -INFINITY, sum = 0.f;
        for (int s = tid; s < splits; s += 32) m = fmaxf(m, base[s * len + G * D + g]);
        m = max_warp(m);
        for (int s = tid; s < splits; s += 32) {
            const float l = base[s * len + G * D + G + g];
            const float w = l == 0.f ? 0.f : ex2(base[s * len + G * D + g] - m);
            weight[s] = w;
            sum += l * w;
        }
        sum = sum_warp(sum);
        if (tid == 0) total[0] = sum;
    }
    __syncthreads();
    const float sum = total[0];
    float o = 0.f;
    const float* src = base + g * D + tid;
#pragma unroll 8
    for (int s = 0; s < splits; ++s) {
        const float w = weight[s];
        o = fmaf(w == 0.f ? 0.f : src[s * len], w, o);
    }
    out[(row * G + g) * D + tid] = __bfloat16_as_ushort(__float2bfloat16_rn(sum == 0.f ? 0.f : o / sum));
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
    const int64_t slots = (int64_t)sms * kQ8Ctas;
    static_assert(C::RING >= 4 && C::SMEM + C::STATIC <= kQ8Smem, "the ring fits beside another CTA");
    kern<<<(unsigned)(items < slots ? items : slots), kQ8Threads, C::SMEM, st>>>(A, km, vm);
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
    const int64_t slots = (int64_t)sms * kQ8Ctas;
    for (int s = 1; s <= K; ++s) {
        const int64_t waves = (rows * s + slots - 1) / slots;
        const double us = waves * ((K + s - 1) / s * (D / 128.0) * 1.5 + 1.5) + (s > 1 ? 3.0 + 0.02 * s : 0.0);
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
        attention_q8_join_kernel<<<dim3((unsigned)A.rows, (unsigned)A.G), (unsigned)D, A.splits * sizeof(float), st>>>(
            A.part, A.out, A.splits, A.G, (int)D);
        e = cudaGetLastError();
    }
    return e == cudaSuccess ? BSA_OK : (int)e;
}
