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
// other operand is made 8-bit too, as a sum of terms in their own columns.
//  - A query is two e4m3 terms, x = hi + lo / 16 with hi = e4m3(x), lo =
//    e4m3(16 (x - hi)).  A bf16 query has 8 significant bits; scaled by a power of
//    two so that the head's largest magnitude lies in [128, 256), hi takes 4 of
//    them and the rounded rest of at most 2^-4 fits lo: exact down to 2^-21 of the
//    largest.
//  - A weight w_j = p_j vs_j, scaled so that the chunk's largest is 2^15, is
//    rounded to fp16 and cut into four e5m2 terms of three bits each, the last two
//    64-fold: they hold the fp16 value exactly down to 2^-27 of the chunk's
//    largest (so w_j within 2^-12 of itself), and within 2^-37 of that below.
//    e5m2 has that range, e4m3 would end at 2^-22: a token that takes the probability
//    and has no value, or a page with a larger scale than others, leaves the others'
//    weights their bits.  Pages of zeros (the append gives them the scale 1) whose
//    scale is the chunk's largest, and far above its least, take the least instead, as
//    their codes are zero under any scale.
// Probabilities are summed in fp32 before their rounding, chunks are joined in
// fp32, and maxima and accumulators are fp32.
//
// The work: a CTA takes items (a row, or a share of its 128-token blocks when
// rows are few; a cluster of CTAs or a second launch joins the shares) and walks
// each in chunks of up to 6 blocks.  A chunk's scores are complete in TMEM before
// its probabilities are formed, so there is one maximum per chunk and the
// accumulators in TMEM start anew with each chunk.
//  softmax    thread i of a group of four warps is token i of a block
//             (probabilities) and dimension i of the head (output); a second
//             group takes query heads 8 to 15,
//  copies     one warp copies blocks by TMA into a ring of shared-memory stages:
//             the next chunk's key blocks, then this chunk's value blocks.  A
//             block whose eight pages follow one another in the cache, as the
//             selector's table has them, is one box; other blocks, and the
//             context's last, are a box per page (issuing eight boxes a block
//             throughout took longer than their bytes), with pages outside the
//             context or the cache as boxes past the end of the tensor, which
//             arrive as zeros,
//  MMAs       one warp issues the next chunk's scores, then this chunk's
//             output, and frees the stages: the scores of one chunk are formed
//             under the softmax of the one before (two score buffers),
//  ahead      one warp reads later chunks' page scales and later items' queries.
// Up to 8 query heads two CTAs share an SM.  Values behind the context's end in
// its last page are set to zero in shared memory (they may be NaN codes); such
// keys only reach their own scores.
//
// Bound by the copies, 2 D bytes a token: 256 rows of 8192 tokens (8 query heads,
// D 128) take 86 to 88 us, 6.2 TB/s, with DRAM reads of just those bytes; rows whose
// blocks lie in L2 reach 10 TB/s.  64-wide heads are bound by the copies' rows, of
// 64 bytes each, at about 3.4 cycles a row and SM (1024 rows of up to 2048
// tokens 47 us); 9 to 16 query heads by the softmax of the SM's one CTA.  With 8
// heads of 128 a CTA has a ring of five blocks beside its weights and three chunks
// announced ahead (with two, 2000 rows of one prompt take 107 us instead of 97).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>
#include <mutex>

#include "bsa_internal.h"
#include "bsa_overlap.h"
#include "bsa_tcgen05.cuh"

namespace bsa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kDepth = 3;                // chunks announced ahead
constexpr int kMaxRing = 12;             // stages of 16 KB
constexpr int kMaxCluster = 8;           // items per row that a cluster joins
constexpr int kSmSmem = 233472;          // an SM's shared memory; 1 KB of it goes to each CTA
constexpr int kTerms = 4;                // terms of a weight
constexpr float kTop = 15.f;             // log2 of a chunk's largest weight as it is rounded
constexpr float kSpread = 65536.f;       // a largest scale this much above the chunk's least may be that of zeros

// A chunk as it is announced to the other warps.
struct Chunk {
    int row, ctx, c0, nb;    // nb < 0: no more
    int qbuf, last;
};

template <int PAGES, int GP, int NU, int GROUPS, int HG>
struct Q8Shared {
    float2 page_scale[kDepth][PAGES];       // ks * scale * log2 e, log2 vs (-inf: no page) of the announced chunks
    // c_full: a chunk's queries are there, x_full: its scales too
    uint64_t full[kMaxRing], empty[kMaxRing], s_full[2][NU], p_full[NU], c_full[kDepth], x_full[kDepth], c_empty[kDepth];
    uint64_t o_full, drained;
    Chunk chunk[kDepth];
    float mid[kDepth];                      // log2 of the middle of a chunk's value scales
    float qinv[kDepth][GP];
    float red[GROUPS][4][HG];
    int box_z[2][PAGES];                    // page coordinates of the copied chunks
    uint32_t tmem_base;
    int gave_up;
};

template <int D, int GP>
struct Q8Cfg {
    static constexpr int HG = GP < 8 ? GP : 8;        // heads a softmax group takes
    static constexpr int GROUPS = GP / HG;
    static constexpr int CTAS = GROUPS == 1 ? 2 : 1;  // per SM
    static constexpr int SOFTMAX = 128 * GROUPS;
    static constexpr int THREADS = SOFTMAX + 96;
    static constexpr int N = GP <= 8 ? 16 : 32;       // MMA columns of the scores: two terms of each head
    static constexpr int NP = kTerms * GP;            // of the outputs: four terms
    static constexpr int NB = 6;                      // blocks per chunk
    static constexpr int S_COLS = NB * N;             // TMEM columns of a chunk's scores
    static constexpr int TMEM = 512 / CTAS;
    static constexpr int PANELS = D == 256 ? 2 : 1;   // 128-byte parts of a head's row
    static constexpr int ROWB = D / PANELS;           // bytes of a row in a panel: 64 or 128
    static constexpr int PANEL = 128 * ROWB;          // a panel of a block: 8 or 16 KB
    static constexpr int BPS = ROWB == 64 ? 2 : 1;    // blocks per ring stage
    static constexpr int STAGE = BPS * PANEL;         // 16 KB
    static constexpr int NU = NB / 2;                 // pairs of blocks: the warps' handshakes are a pair's
    static constexpr int P_BYTES = NB * NP * 128;
    static constexpr int Q_PANEL = N * ROWB;
    static constexpr int Q_BYTES = PANELS * Q_PANEL;
    static constexpr int PAGES = NB * kPagesPerBlock;
    using Shared = Q8Shared<PAGES, GP, NU, GROUPS, HG>;
    static constexpr int FIXED = P_BYTES + kDepth * Q_BYTES + (int)sizeof(Shared);
    static constexpr int RING = (kSmSmem / CTAS - 1024 - FIXED) / STAGE;
    static constexpr int SMEM = RING * STAGE + FIXED;
    static constexpr uint32_t SWIZZLE = ROWB == 128 ? 2 : 4;
    static constexpr uint32_t ATOM = 8 * ROWB;        // 8 rows: the swizzle's period
    __host__ __device__ static constexpr int stages(int nb) { return (nb * PANELS + BPS - 1) / BPS; }
    static_assert(2 * S_COLS + PANELS * NP <= TMEM, "two score buffers and the outputs fit");
    static_assert(RING >= 4 && RING <= kMaxRing, "the ring holds two blocks of the widest heads");
};

struct Q8Params {
    const uint16_t* q;
    const float* ks;
    const float* vs;
    const uint8_t* v;
    const int32_t* bt;
    const int32_t* ctx;
    uint16_t* out;
    float* part;             // partial results of split rows joined by a launch of their own, or null
    int64_t num_pages;
    int32_t rows, H, G, width;
    int32_t splits;          // items per row
    int32_t cluster;         // 1: a row's items are one cluster's CTAs, which join them
    uint32_t k_idesc, v_idesc;
    float scale_log2e;
    uint32_t* status;
    unsigned long long wait_ns;     // a wait's limit
    uint32_t stall;                 // stages after which a CTA's copies stop, for tests
};

// The caches as tensors read in boxes of one page and of one block of a head.
struct Q8Maps {
    CUtensorMap k_page, v_page, k_block, v_block;
};

// floats of one partial result: G x D outputs, then per head the reference m
// and the sum of 2^(y - m)
__host__ __device__ inline int64_t part_floats(int G, int D) { return (int64_t)G * D + 2 * G; }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max_warp(float x) {
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float sum_warp(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
    return x;
}
// barrier 1 + group of a softmax group's 128 threads
__device__ __forceinline__ void group_sync(int group) {
    asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory");
}
__device__ __forceinline__ bool group_any(int group, bool x) {
    int r = x;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %0, 0;\n\tbar.red.popc.u32 %0, %1, 128, p;\n\t}"
        : "+r"(r)
        : "r"(1 + group)
        : "memory");
    return r != 0;
}

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
__device__ __forceinline__ Item make_item(const Q8Params& A, int i, int ctx) {
    Item it;
    it.row = i / A.splits;
    it.split = i - it.row * A.splits;
    it.ctx = max(0, min(ctx, A.width * kSubPage));
    const int n = (it.ctx + kPageSize - 1) / kPageSize;
    it.b0 = (int)((int64_t)n * it.split / A.splits);
    it.b1 = (int)((int64_t)n * (it.split + 1) / A.splits);
    const int len = it.b1 - it.b0;
    const int chunks = (len + NB - 1) / NB;
    it.step = chunks > 0 ? (len + chunks - 1) / chunks : 1;
    return it;
}

// The chunks of a CTA's items in order, each item's context length read one
// item ahead and each chunk's page ids one chunk ahead (page p of the chunk in
// register p / 32 of lane p % 32; INT32_MIN outside the context).
template <int NB>
struct Walk {
    static constexpr int R = (NB * kPagesPerBlock + 31) / 32;
    int i, items, c0, ctx_next, ctx_raw;
    Item it;
    int32_t page[R];

    __device__ __forceinline__ bool done() const { return i >= items; }
    __device__ __forceinline__ int blocks() const { return min(it.step, it.b1 - c0); }
    __device__ __forceinline__ void enter(const Q8Params& A) {
        ctx_raw = ctx_next;
        it = make_item<NB>(A, i, ctx_raw);
        c0 = it.b0;
        const int next = i + (int)gridDim.x;
        if (next < items) ctx_next = __ldg(A.ctx + next / A.splits);
    }
    __device__ __forceinline__ void read(const Q8Params& A) {
        const int lane = threadIdx.x & 31;
        const int32_t* bt = A.bt + (int64_t)it.row * A.width + c0 * kPagesPerBlock;
        const int n = min(blocks() * kPagesPerBlock, (it.ctx + kSubPage - 1) / kSubPage - c0 * kPagesPerBlock);
#pragma unroll
        for (int r = 0; r < R; ++r) page[r] = r * 32 + lane < n ? max(__ldg(bt + r * 32 + lane), -1) : INT32_MIN;
    }
    __device__ __forceinline__ void begin(const Q8Params& A) {
        items = A.rows * A.splits;
        i = blockIdx.x;
        if (done()) return;
        ctx_next = __ldg(A.ctx + i / A.splits);
        enter(A);
        read(A);
    }
    __device__ __forceinline__ void advance(const Q8Params& A) {
        c0 += it.step;
        if (c0 >= it.b1) {
            i += gridDim.x;
            if (done()) return;
            enter(A);
        }
        read(A);
    }
};

// two terms of HG heads: columns [0, HG) and [GP, GP + HG) at addr
template <int HG, int GP>
__device__ __forceinline__ void load_terms(uint32_t addr, float (&s)[2 * HG]) {
    if constexpr (HG == GP && GP == 4) tmem_ld8(addr, s);
    else if constexpr (HG == GP) tmem_ld16(addr, s);
    else tmem_ld8x2(addr, addr + GP, s);
}

__device__ __forceinline__ uint32_t bits_of(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }

// The four lanes of a quad exchange their words' bytes: lane i gets byte i of each.
__device__ __forceinline__ void turn_bytes(uint32_t& a, uint32_t& b, const uint32_t (&s)[6]) {
#pragma unroll
    for (int step = 0; step < 2; ++step) {
        const uint32_t x = __shfl_xor_sync(kFull, __byte_perm(a, b, s[3 * step]), 1 + step);
        a = __byte_perm(a, x, s[3 * step + 1]);
        b = __byte_perm(b, x, s[3 * step + 2]);
    }
}

// the four terms of HG heads' outputs, joined
template <int HG, int GP>
__device__ __forceinline__ void load_output(uint32_t addr, float (&o)[HG]) {
    if constexpr (HG == 4) {
        float x[16];
        tmem_ld16(addr, x);
#pragma unroll
        for (int g = 0; g < 4; ++g) o[g] = fmaf(x[8 + g] + x[12 + g], 0x1p-6f, x[g] + x[4 + g]);
    } else {
        float x[16], y[16];
        tmem_ld8x2(addr + 2 * GP, addr + 3 * GP, y);
        tmem_ld8x2(addr, addr + GP, x);
#pragma unroll
        for (int g = 0; g < 8; ++g) o[g] = fmaf(y[g] + y[8 + g], 0x1p-6f, x[g] + x[8 + g]);
    }
}

template <int D, int GP>
__global__ void __launch_bounds__(Q8Cfg<D, GP>::THREADS, Q8Cfg<D, GP>::CTAS)
attention_q8_kernel(const Q8Params A, const __grid_constant__ Q8Maps M) {
    using C = Q8Cfg<D, GP>;
    constexpr int N = C::N, NP = C::NP, NB = C::NB, RING = C::RING, PANELS = C::PANELS, HG = C::HG;
    constexpr int kCopyWarp = C::SOFTMAX / 32, kMmaWarp = kCopyWarp + 1, kAheadWarp = kCopyWarp + 2;
    extern __shared__ __align__(1024) uint8_t ring[];
    uint8_t* psm = ring + RING * C::STAGE;     // [NB][NP][128] swizzled, K-major
    uint8_t* qsm = psm + C::P_BYTES;           // [kDepth][PANELS][N][ROWB] swizzled, K-major
    typename C::Shared& S = *reinterpret_cast<typename C::Shared*>(qsm + kDepth * C::Q_BYTES);
    auto& page_scale = S.page_scale;
    auto &full = S.full, &empty = S.empty;
    auto& s_full = S.s_full;
    auto& p_full = S.p_full;
    auto &c_full = S.c_full, &x_full = S.x_full, &c_empty = S.c_empty;
    auto &o_full = S.o_full, &drained = S.drained;
    auto& chunk = S.chunk;
    auto& qinv = S.qinv;
    auto& red = S.red;
    auto& box_z = S.box_z;
    int& gave_up = S.gave_up;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int group = C::GROUPS == 1 ? 0 : warp >> 2;      // of a softmax warp
    int item = blockIdx.x;                                 // the first that it has not written

    // the first chunk's pages are on their way while the CTA sets itself up
    Walk<NB> walk;
    if (warp == kCopyWarp || warp == kAheadWarp) walk.begin(A);
    if (warp == kMmaWarp) tmem_alloc(&S.tmem_base, C::TMEM);
    if (tid == 0) {
        for (int i = 0; i < RING; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < C::NU; ++i) {
            mbar_init(&s_full[0][i], 1);
            mbar_init(&s_full[1][i], 1);
            mbar_init(&p_full[i], C::SOFTMAX);
        }
        for (int i = 0; i < kDepth; ++i) {
            mbar_init(&c_full[i], 32);
            mbar_init(&x_full[i], 32);
            mbar_init(&c_empty[i], C::SOFTMAX + 1);      // and the MMA warp
        }
        mbar_init(&o_full, 1);
        mbar_init(&drained, 1);
        gave_up = 0;
        mbar_fence_init();
    }
    // query columns past G stay zero
    for (int i = tid; i < kDepth * C::Q_BYTES / 16; i += C::THREADS)
        reinterpret_cast<uint4*>(qsm)[i] = make_uint4(0, 0, 0, 0);
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    asm volatile("griddepcontrol.launch_dependents;");
    const uint32_t tmem = S.tmem_base;
    volatile int* quit = &gave_up;

    if (warp == kCopyWarp) {
        // ------------------------------------------------ copies
        if (elect_one()) {
            tma_prefetch_map(&M.k_block);
            tma_prefetch_map(&M.v_block);
            tma_prefetch_map(&M.k_page);
            tma_prefetch_map(&M.v_page);
        }
        __syncwarp();
        const int outside = (int)max((int64_t)1, A.num_pages) * kSubPage;   // past the tensor's end
        uint32_t n = 0;   // stages filled so far: stage n % RING
        uint32_t issued = 0;      // the same as the elected thread counts them
        // One thread: nb blocks with page coordinates z; bit b of `runs`: block
        // b's pages follow one another.  Stages from number n on.  False when a wait
        // ran out; nothing is copied after that, as the stages' uses would no longer be
        // in order.
        auto copy = [&](const CUtensorMap* page_map, const CUtensorMap* block_map, const int* z, uint32_t runs, int h,
                        int nb, uint32_t n) -> bool {
            uint32_t st = n % RING, use = n / RING;
            for (int b = 0; b < nb; ++b) {
#pragma unroll
                for (int panel = 0; panel < PANELS; ++panel) {
                    const int sub = C::BPS == 1 ? 0 : b & 1;          // the block's place in its stage
                    if (sub == 0) {
                        if (issued == A.stall) return false;
                        if (use > 0 && !mbar_wait(&empty[st], (use - 1) & 1, quit, A.wait_ns)) return false;
                        mbar_expect(&full[st], C::PANEL * (C::BPS == 2 && b + 1 < nb ? 2 : 1));
                    }
                    uint8_t* dst = ring + st * C::STAGE + sub * C::PANEL;
                    if (runs >> b & 1) {
                        tma_load_3d(dst, block_map, panel * 128, h, z[b * kPagesPerBlock], &full[st]);
                    } else {
#pragma unroll
                        for (int p = 0; p < kPagesPerBlock; ++p)
                            tma_load_3d(dst + p * kSubPage * C::ROWB, page_map, panel * 128, h,
                                        z[b * kPagesPerBlock + p], &full[st]);
                    }
                    if (sub == C::BPS - 1 || b + 1 == nb) {
                        ++issued;
                        if (++st == RING) {
                            st = 0;
                            ++use;
                        }
                    }
                }
            }
            return true;
        };
        bool ok = true;
        int hv = 0, nbv = 0;      // the chunk whose values are still to come
        uint32_t runsv = 0, buf = 0;
        for (; !walk.done() && !__any_sync(kFull, *quit); buf ^= 1) {
            const int h = walk.it.row % A.H, nb = walk.blocks();
            // the chunk's coordinates, and which blocks are runs
            uint32_t runs = 0;
#pragma unroll
            for (int r = 0; r < Walk<NB>::R; ++r) {
                const int pg = walk.page[r];
                const int z = pg >= 0 && pg < A.num_pages ? pg * kSubPage : outside;
                if (r * 32 + lane < C::PAGES) box_z[buf][r * 32 + lane] = z;
                const int first = __shfl_sync(kFull, z, lane & 24);
                const uint32_t follow = __ballot_sync(kFull, z < outside && z == first + (lane & 7) * kSubPage);
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    if ((follow >> (8 * b) & 255u) == 255u) runs |= 1u << (4 * r + b);
            }
            __syncwarp();
            walk.advance(A);
            if (elect_one()) {
                ok = ok && copy(&M.k_page, &M.k_block, box_z[buf], runs, h, nb, n);
                ok = ok && copy(&M.v_page, &M.v_block, box_z[buf ^ 1], runsv, hv, nbv, n + C::stages(nb));
            }
            __syncwarp();
            n += C::stages(nb) + C::stages(nbv);
            runsv = runs;
            hv = h;
            nbv = nb;
        }
        // the copies in flight land before the CTA's memory goes away, also when
        // nobody waits for them any more
        if (elect_one()) {
            if (ok) copy(&M.v_page, &M.v_block, box_z[buf ^ 1], runsv, hv, nbv, n);
            int none = 0;
            for (uint32_t k = issued > RING ? issued - RING : 0; k < issued; ++k)
                mbar_wait(&full[k % RING], (k / RING) & 1, &none);
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------ MMAs
        if (elect_one()) {
            constexpr uint32_t kSteps = C::ROWB / 32;
            // operand descriptors; a byte offset adds offset / 16
            const uint64_t k_desc = smem_desc(smem_addr(ring), 0, C::ATOM, C::SWIZZLE);
            const uint64_t q_desc = smem_desc(smem_addr(qsm), 0, C::ATOM, C::SWIZZLE);
            const uint64_t p_desc = smem_desc(smem_addr(psm), 0, 1024, 2);
            const uint32_t o_cols = tmem + 2 * C::S_COLS;
            uint32_t st = 0, use = 0, p_phase = 0, c = 0, s = 0;      // s: chunks with blocks so far
            int nbv = 0, leftv = 0;              // the chunk whose output is to come: blocks, context tokens
            bool ok = true, more = true;
            while (ok && more) {
                ok = mbar_wait(&c_full[c % kDepth], (c / kDepth) & 1, quit, A.wait_ns);
                if (!ok) break;
                const Chunk ch = chunk[c % kDepth];
                const int nb = ch.nb;
                more = nb >= 0;
                const uint64_t qb = q_desc + ch.qbuf * (C::Q_BYTES / 16);
                mbar_arrive(&c_empty[c % kDepth]);
                ++c;
                // ---- the new chunk's scores ----
                for (int b = 0; ok && b < nb; ++b) {
                    const int sub = C::BPS == 1 ? 0 : b & 1;
                    const bool ends = (b & 1) == 1 || b + 1 == nb;        // of a pair
#pragma unroll
                    for (int panel = 0; panel < PANELS; ++panel) {
                        if (sub == 0) {
                            ok = ok && mbar_wait(&full[st], use & 1, quit, A.wait_ns);
                            if (!ok) break;
                            tc_fence_after();
                        }
                        const uint64_t kd = k_desc + (st * C::STAGE + sub * C::PANEL) / 16;
#pragma unroll
                        for (uint32_t k = 0; k < kSteps; ++k)
                            mma_f8(tmem + (s & 1) * C::S_COLS + b * N, kd + k * 2, qb + panel * (C::Q_PANEL / 16) + k * 2,
                                   A.k_idesc, panel + k > 0);
                        if (C::BPS == 1 || ends) {
                            tc_commit(&empty[st]);
                            if (++st == RING) {
                                st = 0;
                                ++use;
                            }
                        }
                    }
                    if (ok && ends) tc_commit(&s_full[s & 1][b >> 1]);
                }
                // ---- the last chunk's output ----
                for (int b = 0; ok && b < nbv; ++b) {
                    const int sub = C::BPS == 1 ? 0 : b & 1;
                    if ((b & 1) == 0) {
                        ok = mbar_wait(&p_full[b >> 1], (p_phase >> (b >> 1)) & 1, quit, A.wait_ns);
                        p_phase ^= 1u << (b >> 1);
                    }
                    const int left = leftv - b * kPageSize;
#pragma unroll
                    for (int panel = 0; panel < PANELS; ++panel) {
                        if (sub == 0) ok = ok && mbar_wait(&full[st], use & 1, quit, A.wait_ns);
                        if (!ok) break;
                        if (left < kPageSize && left % kSubPage != 0) {
                            // the context ends in a page: the page's other values are not the row's
                            uint4* v = reinterpret_cast<uint4*>(ring + st * C::STAGE + sub * C::PANEL + left * C::ROWB);
                            const int n = (kSubPage - left % kSubPage) * (C::ROWB / 16);
                            for (int i = 0; i < n; ++i) v[i] = make_uint4(0, 0, 0, 0);
                            fence_async_smem();
                        }
                        tc_fence_after();
                        // values: 32 tokens a step; the head's dimensions run along
                        // the rows.  A 64-byte row fills 64 of the 128 MMA rows;
                        // the leading offset 0 reads it again for the others.
                        const uint64_t vd = k_desc + (st * C::STAGE + sub * C::PANEL) / 16;
                        const uint64_t pd = p_desc + b * (NP * 128 / 16);
#pragma unroll
                        for (uint32_t k = 0; k < 4; ++k)
                            mma_f8(o_cols + panel * NP, vd + k * (32 * C::ROWB / 16), pd + k * 2, A.v_idesc, b > 0 || k > 0);
                        if (C::BPS == 1 || sub == 1 || b + 1 == nbv) {
                            tc_commit(&empty[st]);
                            if (++st == RING) {
                                st = 0;
                                ++use;
                            }
                        }
                    }
                }
                if (ok && nbv > 0) tc_commit(&o_full);
                if (nb > 0) ++s;
                nbv = nb;
                leftv = ch.ctx - ch.c0 * kPageSize;
            }
            // no MMA runs on into the release of its memory, also when nobody waits
            // for it any more
            int none = 0;
            tc_commit(&drained);
            mbar_wait(&drained, 0, &none);
        }
        __syncwarp();
    } else if (warp == kAheadWarp) {
        // ------------------------------------------------ scales and queries
        constexpr int LPH = D / 8;         // lanes per query head, 8 values each
        constexpr int HPP = 32 / LPH;      // heads a pass
        const int d = lane % LPH * 8, panel = d / C::ROWB, dc = d % C::ROWB;
        uint32_t c = 0, queries = 0;
        int qbuf = 0;
        bool ok = true;
        for (; !walk.done(); ++c) {
            const Item it = walk.it;
            const int c0 = walk.c0, nb = walk.blocks(), h = it.row % A.H, buf = c % kDepth;
            int32_t pg[Walk<NB>::R];
#pragma unroll
            for (int r = 0; r < Walk<NB>::R; ++r) pg[r] = walk.page[r];
            if (lane == 0 && it.split == 0 && c0 == it.b0)
                report_status(A.status, walk.ctx_raw != it.ctx, BSA_STATUS_BAD_CONTEXT);
            walk.advance(A);
            ok = c < kDepth || mbar_wait(&c_empty[buf], (c / kDepth - 1) & 1, quit, A.wait_ns);
            ok = __all_sync(kFull, ok);
            if (!ok) break;
            {
                // the pages' scales
                float ks[Walk<NB>::R], vs[Walk<NB>::R];
#pragma unroll
                for (int r = 0; r < Walk<NB>::R; ++r) {
                    const bool good = pg[r] >= 0 && pg[r] < A.num_pages;
                    report_status(A.status, !good && pg[r] != INT32_MIN, BSA_STATUS_BAD_PAGE);
                    ks[r] = vs[r] = 0.f;
                    if (good) {
                        const int64_t at = (int64_t)pg[r] * A.H + h;
                        ks[r] = __ldg(A.ks + at);
                        vs[r] = __ldg(A.vs + at);
                    } else {
                        pg[r] = -1;
                    }
                }
                if (c0 == it.b0 && nb > 0) {
                    // the queries as two e4m3 terms
                    qbuf = queries++ % kDepth;
                    uint8_t* qd = qsm + qbuf * C::Q_BYTES;
                    constexpr int PASSES = (GP + HPP - 1) / HPP;
                    uint4 w[PASSES];
#pragma unroll
                    for (int r = 0; r < PASSES; ++r) {
                        const int g = r * HPP + lane / LPH;
                        w[r] = make_uint4(0, 0, 0, 0);
                        if (g < A.G)
                            w[r] = __ldg(reinterpret_cast<const uint4*>(A.q + ((int64_t)it.row * A.G + g) * D + d));
                    }
#pragma unroll
                    for (int r = 0; r < PASSES; ++r) {
                        const int g = r * HPP + lane / LPH;
                        if (r * HPP >= A.G) break;
                        const uint32_t v[4] = {w[r].x, w[r].y, w[r].z, w[r].w};
                        float x[8], m = 0.f;
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            x[k] = __uint_as_float(k & 1 ? v[k / 2] & 0xFFFF0000u : v[k / 2] << 16);
                            m = fmaxf(m, fabsf(x[k]));
                        }
#pragma unroll
                        for (int o = LPH / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
                        // scale by a power of two: the largest magnitude to [128, 256)
                        const int e = min(max((int)(__float_as_uint(m) >> 23) - 127, -100), 127);
                        const float up = __uint_as_float((uint32_t)(127 + 7 - e) << 23);
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            // an infinite query has no finite result: NaN
                            const float a = (x[2 * k] - x[2 * k] == 0.f) ? x[2 * k] * up : NAN;
                            const float b = (x[2 * k + 1] - x[2 * k + 1] == 0.f) ? x[2 * k + 1] * up : NAN;
                            hi[k] = pack_e4m3(a, b);
                            const float2 f = unpack_e4m3(hi[k]);
                            lo[k] = pack_e4m3((a - f.x) * 16.f, (b - f.y) * 16.f);
                        }
                        if (g < A.G) {
#pragma unroll
                            for (int term = 0; term < 2; ++term) {
                                const uint32_t* t = term ? lo : hi;
                                const int row = term * GP + g;
                                const int sw = C::ROWB == 128 ? (row & 7) : ((row >> 1) & 3);
                                uint8_t* dst = qd + panel * C::Q_PANEL + row * C::ROWB + (((dc >> 4) ^ sw) << 4) + (dc & 15);
                                *reinterpret_cast<uint2*>(dst) = make_uint2(t[0] | t[1] << 16, t[2] | t[3] << 16);
                            }
                            if (lane % LPH == 0) qinv[qbuf][g] = __uint_as_float((uint32_t)(127 - 7 + e) << 23);
                        }
                    }
                    if (lane >= A.G && lane < GP) qinv[qbuf][lane] = 0.f;
                }
                // the scores may start; their scales follow
                if (lane == 0) chunk[buf] = Chunk{it.row, it.ctx, c0, nb, qbuf, c0 + nb == it.b1};
                fence_async_smem();
                mbar_arrive(&c_full[buf]);
                // the least and the largest of the values' scales
                uint32_t least = 0x7F800000u, most = 0;
#pragma unroll
                for (int r = 0; r < Walk<NB>::R; ++r) {
                    if (pg[r] < 0) continue;
                    vs[r] = fmaxf(vs[r], 0x1p-149f);         // a scale of 0 has a logarithm too
                    least = min(least, __float_as_uint(vs[r]));
                    most = max(most, __float_as_uint(vs[r]));
                }
                least = __reduce_min_sync(kFull, least);
                most = __reduce_max_sync(kFull, most);
                const float low = __uint_as_float(least);
                // the pages of the largest scale, and while they are all zeros of the next
                while (__uint_as_float(most) > low * kSpread) {
                    bool zeros = true;
#pragma unroll
                    for (int r = 0; r < Walk<NB>::R; ++r) {
                        uint32_t top = __ballot_sync(kFull, pg[r] >= 0 && __float_as_uint(vs[r]) == most);
                        for (; zeros && top != 0; top &= top - 1) {
                            const int l = __ffs(top) - 1, tokens = it.ctx - (c0 * kPagesPerBlock + r * 32 + l) * kSubPage;
                            const uint8_t* v = A.v + ((int64_t)__shfl_sync(kFull, pg[r], l) * kSubPage * A.H + h) * D;
                            uint32_t any = 0;
#pragma unroll
                            for (int k = 0; k < D / 32; ++k) {
                                const int u = lane + 32 * k, slot = u / (D / 16);
                                if (slot < tokens) {
                                    const uint4 x = __ldg(reinterpret_cast<const uint4*>(v + (int64_t)slot * A.H * D) + u % (D / 16));
                                    any |= x.x | x.y | x.z | x.w;
                                }
                            }
                            zeros = !__any_sync(kFull, (any & 0x7F7F7F7Fu) != 0);
                            if (zeros && lane == l) vs[r] = low;
                        }
                    }
                    if (!zeros) break;
                    most = least;
#pragma unroll
                    for (int r = 0; r < Walk<NB>::R; ++r)
                        if (pg[r] >= 0) most = max(most, __float_as_uint(vs[r]));
                    most = __reduce_max_sync(kFull, most);
                }
                // a weight 2^-100 of the largest possible one counts for its probability alone
                const float floor_vs = fmaxf(low, __uint_as_float(most) * 0x1p-100f);
#pragma unroll
                for (int r = 0; r < Walk<NB>::R; ++r) {
                    const int p = r * 32 + lane;
                    if (p >= nb * kPagesPerBlock) continue;
                    page_scale[buf][p] = pg[r] < 0 ? make_float2(0.f, -INFINITY)
                                                   : make_float2(ks[r] * A.scale_log2e, log2f(fmaxf(vs[r], floor_vs)));
                }
                if (lane == 0) S.mid[buf] = most == 0 ? 0.f : 0.5f * (log2f(floor_vs) + log2f(__uint_as_float(most)));
                mbar_arrive(&x_full[buf]);
            }
        }
        if (ok) ok = c < kDepth || mbar_wait(&c_empty[c % kDepth], (c / kDepth - 1) & 1, quit, A.wait_ns);
        __syncwarp();
        if (lane == 0) chunk[c % kDepth].nb = -1;
        __syncwarp();
        mbar_arrive(&c_full[c % kDepth]);
        mbar_arrive(&x_full[c % kDepth]);
    } else {
        // ------------------------------------------------ softmax and output
        const int tok = tid & 127, quad = warp & 3;
        const int g0 = group * HG;                                 // this group's first head
        const uint32_t lanes = tmem + ((uint32_t)quad << 21) + g0;   // the warp's 32 TMEM lanes
        const int part16 = tok >> 4;                               // byte tok's 16-byte part of a P row
        // the place of this lane's four tokens in row g0 + lane % 4 of a block's weights, and
        // in the row four further
        const uint32_t row0 = (uint32_t)(g0 + (lane & 3)) * 128 + (tok & 12);
        const uint32_t place[2] = {row0 + ((part16 ^ (lane & 3)) << 4), row0 + 512 + ((part16 ^ (4 + (lane & 3))) << 4)};
        // bytes that go to a neighbouring lane, and that stay with those that come (turn_bytes)
        const uint32_t turn[6] = {lane & 1 ? 0x6420u : 0x7531u, lane & 1 ? 0x3514u : 0x5240u, lane & 1 ? 0x3716u : 0x7260u,
                                  lane & 2 ? 0x5410u : 0x7632u, lane & 2 ? 0x3254u : 0x5410u, lane & 2 ? 0x3276u : 0x7610u};
        uint32_t s_phase = 0, o_phase = 0, s = 0;      // s: chunks with blocks so far
        // sums in units of 2^ml, outputs in units of 2^(mt - kTop), the open chunk's in
        // units of take^2 of those.  Chunks of zeros among tiny values lie further apart than
        // fp32's powers of two, their products with outputs do not: hence in two factors.
        float acc[PANELS][HG], mt[HG], ml[HG], l[HG], take[HG];
#pragma unroll
        for (int g = 0; g < HG; ++g) {
#pragma unroll
            for (int p = 0; p < PANELS; ++p) acc[p][g] = 0.f;
            mt[g] = ml[g] = -INFINITY;
            l[g] = take[g] = 0.f;
        }
        int row = 0;
        bool open = false, last = false;      // a chunk whose output is to come, and whether it ends its item

        // Adds the open chunk's output, and writes the item's result at its end.
        auto close_chunk = [&]() {
            if (open) {
                mbar_wait(&o_full, o_phase, quit, A.wait_ns);
                __syncwarp();
                o_phase ^= 1;
                tc_fence_after();
#pragma unroll
                for (int p = 0; p < PANELS; ++p) {
                    float o[HG];
                    load_output<HG, GP>(lanes + 2 * C::S_COLS + p * NP, o);
#pragma unroll
                    for (int g = 0; g < HG; ++g) acc[p][g] = fmaf(o[g] * take[g], take[g], acc[p][g]);
                }
                tc_fence_before();
            }
            if (last) {
                // the sums over the group's tokens
                group_sync(group);
#pragma unroll
                for (int g = 0; g < HG; ++g) {
                    const float a = sum_warp(l[g]);
                    if (lane == 0) red[group][quad][g] = a;
                }
                group_sync(group);
                const bool bad = *quit;             // what was not waited for is not a result
                uint16_t* o16 = A.out + (int64_t)row * A.G * D;
                // a split row's part: to the workspace, or to this CTA's own
                // memory, where its probabilities are no longer needed
                float* o32 = A.cluster ? reinterpret_cast<float*>(psm) : A.part + (int64_t)item * part_floats(A.G, D);
#pragma unroll
                for (int g = 0; g < HG; ++g) {
                    if (g0 + g < A.G && !bad) {
                        const float sum = red[group][0][g] + red[group][1][g] + red[group][2][g] + red[group][3][g];
                        const float f = sum == 0.f ? 0.f : 1.f / sum, e = sum == 0.f ? 0.f : ex2(0.5f * (mt[g] - ml[g] - kTop));
#pragma unroll
                        for (int p = 0; p < PANELS; ++p) {
                            const float o = acc[p][g] * e * f * e;
                            const int at = (g0 + g) * D + p * 128 + tok;
                            if (tok < C::ROWB) {
                                if (A.splits == 1) o16[at] = __bfloat16_as_ushort(__float2bfloat16_rn(o));
                                else o32[at] = o;
                            }
                        }
                        if (A.splits > 1 && tok == 0) {
                            o32[A.G * D + g0 + g] = ml[g];
                            o32[A.G * D + A.G + g0 + g] = sum;
                        }
                    }
#pragma unroll
                    for (int p = 0; p < PANELS; ++p) acc[p][g] = 0.f;
                    mt[g] = ml[g] = -INFINITY;
                    l[g] = 0.f;
                }
                if (!bad) item += gridDim.x;
            }
            open = last = false;
        };

        // These warps meet in barriers, so none leaves alone: a wait that ran
        // out anywhere ends at the next chunk for the whole group, or lets the
        // loops go on with what there is; the items from that on are not written here.
        for (uint32_t c = 0;; ++c) {
            const int buf = c % kDepth;
            mbar_wait(&x_full[buf], (c / kDepth) & 1, quit, A.wait_ns);
            const bool gone = *quit;
            const Chunk ch = chunk[buf];
            const int nb = ch.nb;
            if (group_any(group, gone || nb < 0)) break;
            const float2* scales = page_scale[buf];
            const float mid = S.mid[buf];
            float qi[HG], ct[HG];
#pragma unroll
            for (int g = 0; g < HG; ++g) {
                qi[g] = qinv[ch.qbuf][g0 + g];
                ct[g] = -INFINITY;
            }
            // ---- the chunk's maxima, block by block as scores complete ----
            const uint32_t sbuf = s & 1;
            const uint32_t s_cols = lanes + sbuf * C::S_COLS;
            for (int b = 0; b < nb; b += 2) {
                mbar_wait(&s_full[sbuf][b >> 1], (s_phase >> (sbuf * 8 + (b >> 1))) & 1, quit, A.wait_ns);
                __syncwarp();
                tc_fence_after();
                // both blocks of the pair; one that is not there has no live token
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float x[2 * HG];
                    load_terms<HG, GP>(s_cols + (b + j) * N, x);
                    const float2 sc = scales[(b + j) * kPagesPerBlock + part16];
                    const bool live = b + j < nb && (ch.c0 + b + j) * kPageSize + tok < ch.ctx && sc.y != -INFINITY;
#pragma unroll
                    for (int g = 0; g < HG; ++g) {
                        const float t = fmaf(fmaf(x[HG + g], 0.0625f, x[g]), qi[g] * sc.x, sc.y);
                        if (live) ct[g] = fmaxf(ct[g], t);
                    }
                }
            }
            close_chunk();
            row = ch.row;
            last = ch.last;
            if (nb > 0) {
                open = true;
                group_sync(group);                       // red has been read
#pragma unroll
                for (int g = 0; g < HG; ++g) {
                    const float t = max_warp(ct[g]);
                    if (lane == 0) red[group][quad][g] = t;
                }
                group_sync(group);
#pragma unroll
                for (int g = 0; g < HG; ++g) {
                    const float t = fmaxf(fmaxf(red[group][0][g], red[group][1][g]), fmaxf(red[group][2][g], red[group][3][g]));
                    const float top = fmaxf(mt[g], t), m = fmaxf(ml[g], t - mid);
                    if (t > -INFINITY) {
                        const float keep = ex2(0.5f * (mt[g] - top));
#pragma unroll
                        for (int p = 0; p < PANELS; ++p) acc[p][g] = acc[p][g] * keep * keep;
                        l[g] *= ex2(ml[g] - m);
                    }
                    take[g] = t > -INFINITY ? ex2(0.5f * (t - top)) : 0.f;
                    mt[g] = top;
                    ml[g] = m;
                    ct[g] = kTop - t;
                }
                // ---- the weights, and the probabilities' sums in units of 2^(t - mid) ----
                float lc[HG];
#pragma unroll
                for (int g = 0; g < HG; ++g) lc[g] = 0.f;
                for (int b = 0; b < nb; b += 2) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float x[2 * HG];
                        load_terms<HG, GP>(s_cols + (b + j) * N, x);
                        const float2 sc = scales[(b + j) * kPagesPerBlock + part16];
                        const bool live = b + j < nb && (ch.c0 + b + j) * kPageSize + tok < ch.ctx && sc.y != -INFINITY;
                        const float per_w = live ? ex2(mid - sc.y - kTop) : 0.f;     // p_j / w_j
                        float w[HG];
#pragma unroll
                        for (int g = 0; g < HG; ++g) {
                            const float t = fmaf(fmaf(x[HG + g], 0.0625f, x[g]), qi[g] * sc.x, sc.y + ct[g]);
                            w[g] = live ? ex2(t) : 0.f;
                            lc[g] = fmaf(w[g], per_w, lc[g]);
                        }
                        uint8_t* pb = psm + (b + j) * NP * 128;
                        __half2 rest[HG / 2];
#pragma unroll
                        for (int g = 0; g < HG / 2; ++g) rest[g] = __floats2half2_rn(w[2 * g], w[2 * g + 1]);
                        uint32_t word[HG / 4 * kTerms];
#pragma unroll
                        for (int term = 0; term < kTerms; ++term) {
                            // a term is the upper byte of the fp16 values
#pragma unroll
                            for (int g = 0; g < HG / 4; ++g)
                                word[term * (HG / 4) + g] = __byte_perm(bits_of(rest[2 * g]), bits_of(rest[2 * g + 1]), 0x7531);
#pragma unroll
                            for (int g = 0; g < HG / 2; ++g) {
                                const uint32_t top = bits_of(rest[g]) & 0xFF00FF00u;
                                rest[g] = __hsub2_rn(rest[g], *reinterpret_cast<const __half2*>(&top));
                                if (term == 1) rest[g] = __hmul2_rn(rest[g], __float2half2_rn(64.f));
                            }
                        }
                        // word i has one token's terms of rows R(i), R(i) + 1, ..; turned, row
                        // R(i) + lane % 4's of four tokens
#pragma unroll
                        for (int i = 0; i < HG / 4 * kTerms; i += 2) {
                            turn_bytes(word[i], word[i + 1], turn);
                            const int r0 = HG == 4 ? 4 * i : (i / 2) * GP;
                            *reinterpret_cast<uint32_t*>(pb + place[0] + r0 * 128) = word[i];
                            *reinterpret_cast<uint32_t*>(pb + place[1] + r0 * 128) = word[i + 1];
                        }
                    }
                    fence_async_smem();
                    tc_fence_before();
                    mbar_arrive(&p_full[b >> 1]);
                }
#pragma unroll
                for (int g = 0; g < HG; ++g) l[g] = fmaf(lc[g], ct[g] < INFINITY ? ex2(kTop - ct[g] - mid - ml[g]) : 1.f, l[g]);
                s_phase ^= ((1u << ((nb + 1) >> 1)) - 1) << (sbuf * 8);
                ++s;
            }
            mbar_arrive(&c_empty[buf]);
        }
        close_chunk();
    }
    tc_fence_before();
    __syncthreads();
    if (warp < kCopyWarp) {
        // after a wait that ran out: NaN for the items not written (every thread has its
        // own count; without such a wait none is left)
        for (; item < A.rows * A.splits; item += gridDim.x) {
            const int h0 = group * HG, h1 = min(A.G, h0 + HG), t = tid & 127;
            float* o32 = A.cluster ? reinterpret_cast<float*>(psm) : A.part + (int64_t)item * part_floats(A.G, D);
            for (int g = h0; g < h1; ++g) {
                for (int d = t; d < D; d += 128) {
                    const int at = g * D + d;
                    if (A.splits == 1) A.out[(int64_t)item * A.G * D + at] = 0x7FFF;
                    else o32[at] = NAN;
                }
                if (A.splits > 1 && t == 0) {
                    o32[A.G * D + g] = -INFINITY;
                    o32[A.G * D + A.G + g] = NAN;
                }
            }
        }
    }
    if (tid == 0) report_status(A.status, gave_up != 0, BSA_STATUS_TIMEOUT);
    if (warp == kMmaWarp) tmem_free(tmem, C::TMEM);
    if (A.cluster) {
        // the row's parts lie in the cluster's CTAs: each joins every so many-th head
        cluster_sync();
        const uint32_t rank = cluster_rank(), base = smem_addr(psm);
        const int heads = (int)rank < A.G ? (A.G - (int)rank + A.splits - 1) / A.splits : 0;
        const int64_t row = blockIdx.x / A.splits;
        for (int i = tid; i < heads * D; i += C::THREADS) {
            const int g = (int)rank + i / D * A.splits, d = i % D;
            float mt[kMaxCluster], l[kMaxCluster], o[kMaxCluster], top = -INFINITY;
#pragma unroll
            for (int s = 0; s < kMaxCluster; ++s) {
                mt[s] = -INFINITY;
                l[s] = o[s] = 0.f;
                if (s < A.splits) {
                    mt[s] = cluster_read(base + 4 * (A.G * D + g), s);
                    l[s] = cluster_read(base + 4 * (A.G * D + A.G + g), s);
                    o[s] = cluster_read(base + 4 * (g * D + d), s);
                }
                top = fmaxf(top, mt[s]);
            }
            float sum = 0.f, acc = 0.f;
#pragma unroll
            for (int s = 0; s < kMaxCluster; ++s) {
                const float w = l[s] == 0.f ? 0.f : l[s] * ex2(mt[s] - top);
                sum += w;
                if (w != 0.f) acc = fmaf(o[s], w, acc);
            }
            A.out[(row * A.G + g) * D + d] = __bfloat16_as_ushort(__float2bfloat16_rn(sum == 0.f ? 0.f : acc / sum));
        }
        cluster_sync();          // no CTA leaves while another reads its memory
    }
}

// Joins the partial results of a split row, head by head: D threads wide, and
// several such slices that take every so many-th part, the first kJoinAhead of
// each read before the parts' weights are known.  Launched to start beside the
// last items (programmatic dependent launch), it waits for their end here.
constexpr int kJoinThreads = 512;
constexpr int kJoinAhead = 4;
__global__ void __launch_bounds__(kJoinThreads)
attention_q8_join_kernel(const float* part, uint16_t* out, int splits, int G, int D) {
    extern __shared__ float weight[];          // [splits], then a sum per thread
    __shared__ float total;
    const int64_t row = blockIdx.x;
    const int g = blockIdx.y, tid = threadIdx.x, d = tid % D, slice = tid / D, slices = blockDim.x / D;
    asm volatile("griddepcontrol.wait;" ::: "memory");     // the parts are written
    const int64_t len = part_floats(G, D);
    const float* base = part + row * splits * len;
    const float* src = base + g * D + d;
    float ahead[kJoinAhead];
#pragma unroll
    for (int j = 0; j < kJoinAhead; ++j) {
        const int s = slice + j * slices;
        ahead[j] = s < splits ? src[s * len] : 0.f;
    }
    if (tid < 32) {
        float m = -INFINITY, sum = 0.f;
        for (int s = tid; s < splits; s += 32) m = fmaxf(m, base[s * len + G * D + g]);
        m = max_warp(m);
        for (int s = tid; s < splits; s += 32) {
            const float l = base[s * len + G * D + G + g];
            const float w = l == 0.f ? 0.f : l * ex2(base[s * len + G * D + g] - m);
            weight[s] = w;
            sum += w;
        }
        sum = sum_warp(sum);
        if (tid == 0) total = sum;
    }
    __syncthreads();
    // a part without tokens has weight 0
    float o = 0.f;
#pragma unroll
    for (int j = 0; j < kJoinAhead; ++j) {
        const int s = slice + j * slices;
        const float w = s < splits ? weight[s] : 0.f;
        if (w != 0.f) o = fmaf(ahead[j], w, o);
    }
#pragma unroll 4
    for (int s = slice + kJoinAhead * slices; s < splits; s += slices) {
        const float w = weight[s];
        if (w != 0.f) o = fmaf(src[s * len], w, o);
    }
    float* sums = weight + splits;
    sums[tid] = o;
    __syncthreads();
    if (slice > 0) return;
    for (int i = 1; i < slices; ++i) o += sums[i * D + d];
    out[(row * G + g) * D + d] = __bfloat16_as_ushort(__float2bfloat16_rn(total == 0.f ? 0.f : o / total));
}

// ---- host ------------------------------------------------------------------

std::atomic<unsigned long long> g_wait_ns{kWaitNs};
std::atomic<uint32_t> g_stall{UINT32_MAX};

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
// `box_tokens` tokens of one head (128 bytes of it at most).
bool encode_cache(CUtensorMap* map, const void* base, int64_t tokens, int64_t H, int64_t D, int box_tokens) {
    const EncodeFn fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)D, (cuuint64_t)(H * D)};
    const cuuint32_t box[3] = {(cuuint32_t)(D < 128 ? D : 128), 1, (cuuint32_t)box_tokens};
    const cuuint32_t unit[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, unit,
              CU_TENSOR_MAP_INTERLEAVE_NONE, D < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int GP>
cudaError_t launch_q8(Q8Params& A, const Q8Maps& M, bool e4m3, int sms, cudaStream_t st) {
    using C = Q8Cfg<D, GP>;
    const uint32_t fmt = e4m3 ? 0 : 1;
    A.k_idesc = f8_idesc(fmt, 0, false, 128, C::N);
    A.v_idesc = f8_idesc(fmt, 1, true, 128, C::NP);
    auto kern = attention_q8_kernel<D, GP>;
    static FuncOnce once;
    const cudaError_t e = once.smem(reinterpret_cast<const void*>(kern), C::SMEM);
    if (e != cudaSuccess) return e;
    const int64_t items = (int64_t)A.rows * A.splits;
    const int64_t slots = (int64_t)sms * C::CTAS;
    static_assert((GP * D + 2 * GP) * (int)sizeof(float) <= C::P_BYTES, "a part fits where the probabilities were");
    if (!A.cluster) {
        kern<<<(unsigned)(items < slots ? items : slots), C::THREADS, C::SMEM, st>>>(A, M);
        return cudaGetLastError();
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)items);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)A.splits;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, (const Q8Params)A, M);
}

template <int D>
cudaError_t launch_q8_g(Q8Params& A, const Q8Maps& M, bool e4m3, int sms, cudaStream_t st) {
    if (A.G <= 4) return launch_q8<D, 4>(A, M, e4m3, sms, st);
    if (A.G <= 8) return launch_q8<D, 8>(A, M, e4m3, sms, st);
    return launch_q8<D, 16>(A, M, e4m3, sms, st);
}

bool sizes_ok(int64_t T, int64_t H, int64_t G, int64_t D) {
    return T >= 0 && T <= INT32_MAX && H >= 1 && H <= 65536 && T * H <= (1 << 24) && G >= 1 &&
           G <= BSA_MAX_ATTN_Q8_GROUP && (D == 64 || D == 128 || D == 256);
}

// Items per row.  For each number of rounds over the resident CTAs the largest
// split that keeps to it, the fewest items of that block count, is weighed: the
// longest CTA's blocks and items, not less than the copies of all blocks over
// all SMs, and the join.  The constants are in us, fitted to sweeps of 1 to 50
// items per row over 14 shapes: e.g. one row of 16 blocks takes 16.3 unsplit,
// 10.0 in 8; 160 rows of 16 blocks 32 unsplit, 33 in 3; 111 rows of 17
// blocks 256 wide 28 unsplit, 25 in 2; six rows of 1024 blocks 675
// unsplit, 44 in 25, 57 in 32.  2, 4 or 8 items of a row, all resident at once, are
// the CTAs of a cluster, which join them through its shared memory (no second
// launch, no workspace): one row of 16 blocks 9.1 us, joined by a launch 10.0; 32 such
// rows 11.0 and 13.1.
struct Split {
    int items;         // per row
    bool cluster;      // joined by their cluster
};
Split pick_splits(int64_t rows, int64_t G, int64_t D, int32_t K, int sms) {
    const int64_t slots = (int64_t)sms * (G <= 8 ? 2 : 1);
    const double copy_us = (double)rows * K * D * 256 / 6.0e6;     // 6 TB/s
    const double block_us = D == 256 ? 1.4 : 0.7, item_us = 4.0, join_us = 2.5, cluster_us = 1.0;
    auto cost = [&](int64_t s, double joined) {
        const int64_t blocks = (K + s - 1) / s;
        const double cta_us = (double)((rows * s + slots - 1) / slots) * (blocks * block_us + item_us);
        return (cta_us > copy_us ? cta_us : copy_us) + joined;
    };
    Split best{1, false};
    double least = cost(1, 0.0);
    auto weigh = [&](int64_t s, bool cluster) {
        const double us = cost(s, cluster ? cluster_us : join_us + 0.1 * s + 0.004 * rows * s);
        if (us < least) {
            best = Split{(int)s, cluster};
            least = us;
        }
    };
    for (int64_t rounds = 1; rounds <= 8; ++rounds) {
        int64_t s = rounds * slots / rows;
        if (s > K) s = K;
        // the halves too: fewer items may cost less to join than their blocks save
        for (; s >= 2; s /= 2) weigh((K + (K + s - 1) / s - 1) / ((K + s - 1) / s), false);   // the fewest of that block count
    }
    for (int s = 2; s <= kMaxCluster && s <= K && rows * s <= slots; s *= 2) weigh(s, true);
    return best;
}

size_t workspace_need(int64_t rows, int64_t G, int64_t D, Split s) {
    return s.items > 1 && !s.cluster ? (size_t)(rows * s.items * part_floats((int)G, (int)D)) * sizeof(float) : 0;
}

}  // namespace
}  // namespace bsa

using namespace bsa;

extern "C" void bsa_attention_q8_stall(uint32_t stages, uint64_t wait_ns) {
    g_stall.store(stages, std::memory_order_relaxed);
    g_wait_ns.store(wait_ns == 0 ? kWaitNs : wait_ns, std::memory_order_relaxed);
}

extern "C" size_t bsa_attention_q8_workspace_bytes(int64_t T, int64_t H, int64_t G, int64_t D, int32_t K) {
    if (!sizes_ok(T, H, G, D) || T == 0 || K < 1 || K > BSA_MAX_TOPK) return 0;
    return workspace_need(T * H, G, D, pick_splits(T * H, G, D, K, device_sm_count()));
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
    // out may be q itself: a row is written when its queries have been read
    const int64_t row_bytes = T * H * G * D * 2, cache_bytes = num_pages * kSubPage * H * D, scale_bytes = num_pages * H * 4;
    const Rows o = whole_rows(out, row_bytes);
    if ((q != out && rows_overlap(o, whole_rows(q, row_bytes))) || rows_overlap(o, whole_rows(k_cache, cache_bytes)) ||
        rows_overlap(o, whole_rows(v_cache, cache_bytes)) || rows_overlap(o, whole_rows(k_scale, scale_bytes)) ||
        rows_overlap(o, whole_rows(v_scale, scale_bytes)))
        return BSA_ERR_SHAPE;
    const int sms = device_sm_count();
    Q8Params A{};
    A.q = static_cast<const uint16_t*>(q);
    A.ks = k_scale;
    A.vs = v_scale;
    A.v = static_cast<const uint8_t*>(v_cache);
    A.bt = sparse_bt;
    A.ctx = sparse_ctx;
    A.out = static_cast<uint16_t*>(out);
    A.num_pages = num_pages;
    A.rows = (int32_t)(T * H);
    A.H = (int32_t)H;
    A.G = (int32_t)G;
    A.width = K * kPagesPerBlock;
    const Split split = pick_splits(T * H, G, D, K, sms);
    A.splits = split.items;
    A.cluster = split.cluster;
    A.scale_log2e = scale * 1.44269504f;
    A.status = current_status_word();
    A.wait_ns = g_wait_ns.load(std::memory_order_relaxed);
    A.stall = g_stall.load(std::memory_order_relaxed);
    const size_t need = workspace_need(A.rows, G, D, split);
    if (need > 0) {
        if (workspace == nullptr || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255) != 0)
            return BSA_ERR_WORKSPACE;
        A.part = static_cast<float*>(workspace);
    }
    // an empty cache: no box lies inside, any address serves
    Q8Maps M;
    const int64_t tokens = (num_pages > 0 ? num_pages : 1) * kSubPage;
    const void* kb = num_pages > 0 ? k_cache : q;
    const void* vb = num_pages > 0 ? v_cache : q;
    if (!encode_cache(&M.k_page, kb, tokens, H, D, kSubPage) || !encode_cache(&M.v_page, vb, tokens, H, D, kSubPage) ||
        !encode_cache(&M.k_block, kb, tokens, H, D, kPageSize) || !encode_cache(&M.v_block, vb, tokens, H, D, kPageSize))
        return (int)cudaErrorInvalidValue;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool e4m3 = cache_dtype == BSA_DTYPE_E4M3;
    cudaError_t e;
    if (D == 64) e = launch_q8_g<64>(A, M, e4m3, sms, st);
    else if (D == 128) e = launch_q8_g<128>(A, M, e4m3, sms, st);
    else e = launch_q8_g<256>(A, M, e4m3, sms, st);
    if (e == cudaSuccess && A.part != nullptr) {
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)A.rows, (unsigned)A.G);
        // slices: four parts each at least
        int slices = (A.splits + kJoinAhead - 1) / kJoinAhead;
        if (slices > kJoinThreads / (int)D) slices = kJoinThreads / (int)D;
        cfg.blockDim = dim3((unsigned)(slices * D));
        cfg.dynamicSmemBytes = (A.splits + kJoinThreads) * sizeof(float);
        cfg.stream = st;
        cudaLaunchAttribute attr{};
        attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr.val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, attention_q8_join_kernel, (const float*)A.part, A.out, A.splits, A.G, (int)D);
    }
    return e == cudaSuccess ? BSA_OK : (int)e;
}
