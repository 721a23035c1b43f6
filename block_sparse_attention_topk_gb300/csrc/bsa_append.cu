// bsa_append.cu -- a step's keys (rotated) and values into the paged cache, in
// bf16 or in 8 bits with a scale per page and head; the step's queries are
// rotated in the same launch.
//
// One CTA takes a tile of token rows: it forms the rows' cosines and sines once
// in shared memory, rotates the rows' query heads slot by slot (bsa_rope.cuh),
// and appends page by page: the row that is the call's first in its page (its
// leader) stands for all of the call's tokens in that page, at most 16, which
// follow it, possibly into the next tile.  A warp takes such a page's keys or
// values of one head: it takes the maximum of the rotated values, then rotates
// again to round them with the page's scale (rotating twice costs two products
// per value; holding fp32 values would take 64 registers a lane and more).  So a
// page has one writer, and the result does not depend on how the work is spread.
// Bound by memory in long calls, where the queries' read and write are the most
// of it (two 8192-token prompts, 32 query and 4 KV heads of 128, e4m3: 60 us, 5.3
// TB/s), and by its chain of dependent loads (length, table entry, scale) in single
// steps (4 us a token).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "bsa_internal.h"
#include "bsa_overlap.h"
#include "bsa_rope.cuh"

namespace bsa {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kAppendCtas = 4;          // per SM
constexpr int kAppendTile = 16;         // rows per CTA at most
constexpr int kPageRows = BSA_SUB_PAGE_SIZE;
constexpr int kPageBatch = 2;           // slots of a page in flight per lane
constexpr int kQueryBatch = 2;          // slots of the queries in flight per thread

struct AppendParams {
    bsa_append_args_t a;
    RopeParams r;
    const int32_t* seq_lens;   // decode form, else null
    int32_t dql;
    const int32_t* cu;         // varlen form
    const int32_t* prefix;
    uint32_t* status;
    int32_t tile;
};

// The 8-bit types.  The power-of-two scale of a maximum m = f * 2^e, f in
// [1, 2), is 2^(e - 8) or 2^(e - 15), one more when f > 1.75 (both types end
// at 1.75 * 2^k).
template <int FMT>
struct Code {
    static constexpr int kTop = FMT == BSA_DTYPE_E4M3 ? 8 : 15;
    static constexpr __nv_fp8_interpretation_t kKind = FMT == BSA_DTYPE_E4M3 ? __NV_E4M3 : __NV_E5M2;
    // four codes, the first in the low byte
    __device__ static uint32_t pack(float a, float b, float c, float d) {
        return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, kKind) |
               (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, kKind) << 16;
    }
    __device__ static uint32_t scaled(uint32_t c, float f) {
        const __half2 lo = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c & 0xFFFF), kKind));
        const __half2 hi = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c >> 16), kKind));
        const float2 x = __half22float2(lo), y = __half22float2(hi);
        return pack(x.x * f, x.y * f, y.x * f, y.y * f);
    }
    __device__ __forceinline__ static void store(uint8_t* d, const float (&f)[8], float inv) {
        *reinterpret_cast<uint2*>(d) = make_uint2(pack(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                                                  pack(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
    }
    __device__ __forceinline__ static void store(uint8_t* d, const float (&f)[4], float inv) {
        *reinterpret_cast<uint32_t*>(d) = pack(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
    }
    // scale of the largest magnitude (0: none)
    __device__ static float scale(float amax) {
        if (!(amax > 0.f)) return 0.f;
        const uint32_t b = __float_as_uint(amax);
        int e = (int)(b >> 23) - 127 - kTop + ((b & 0x7FFFFFu) > 0x600000u);
        e = max(e, -126);
        return __uint_as_float((uint32_t)(e + 127) << 23);
    }
};

struct Row {
    int32_t req, pos;   // pos < 0: no token
    int32_t left;       // rows of the sequence from this one on
    int32_t index;      // rows of the sequence before this one in the call
};

__device__ Row find_row(const AppendParams& P, int64_t t) {
    Row r{0, -1, 0, 0};
    int64_t pos, left;
    if (P.seq_lens != nullptr) {
        r.req = (int32_t)(t / P.dql);
        r.index = (int32_t)(t - (int64_t)r.req * P.dql);
        left = P.dql - r.index;
        pos = (int64_t)__ldg(P.seq_lens + r.req) - left;
    } else {
        // the sequence with cu[lo] <= t < cu[hi]
        int64_t lo = 0, hi = P.a.num_reqs;
        if (hi == 0 || t < __ldg(P.cu) || t >= __ldg(P.cu + hi)) return r;
        while (hi - lo > 1) {
            const int64_t mid = (lo + hi) >> 1;
            if (__ldg(P.cu + mid) <= t) lo = mid;
            else hi = mid;
        }
        r.req = (int32_t)lo;
        r.index = (int32_t)(t - __ldg(P.cu + lo));
        left = __ldg(P.cu + hi) - t;
        pos = (int64_t)__ldg(P.prefix + lo) + r.index;
    }
    r.pos = (int32_t)(pos < 0 ? -1 : (pos > INT32_MAX ? INT32_MAX : pos));
    r.left = (int32_t)min(left, P.a.T - t);
    return r;
}

// The call's tokens of one page.
struct Segment {
    int64_t page;
    int32_t row;      // the leader, counted from the tile's first row
    int32_t n, off;   // tokens, first slot
};

// One page's n tokens of one head, rows x + t * ts, into slots [off, off + n),
// by groups of GE elements.
template <int FMT, RopeMode MODE, int GE, bool KEEP>
__device__ __forceinline__ void store_page(const AppendParams& P, const uint16_t* __restrict__ x, int64_t ts,
                                           const Segment& S, int h, const float* cs, bool rotate, void* cache,
                                           float* scales) {
    using G = Group<uint16_t, GE>;
    using V = typename G::V;
    const int lane = threadIdx.x & 31;
    const int D = (int)P.a.D, ks = D / (2 * GE), half = rotate ? P.r.half : 0;
    const int64_t row = P.a.H * D;
    const int64_t base = S.page * kPageRows * row + (int64_t)h * D + S.off * row;
    float* sp = FMT == BSA_DTYPE_BF16 ? nullptr : scales + S.page * P.a.H + h;
    float old = 0.f;
    if (FMT != BSA_DTYPE_BF16 && S.off > 0) old = *sp;
    const int total = S.n * ks;     // slots of the page's tokens
    struct Batch {
        V a[kPageBatch], b[kPageBatch];
        int at[kPageBatch];         // token << 8 | slot
    };
    auto load = [&](int i, Batch& B) {
#pragma unroll
        for (int j = 0; j < kPageBatch; ++j) {
            const int u = min(i + 32 * j, total - 1);
            const int t = u / ks, k = u - t * ks;
            int o0, o1;
            slot_groups<MODE, GE>(k, half, o0, o1);
            B.a[j] = __ldg(reinterpret_cast<const V*>(x + t * ts + o0));
            B.b[j] = __ldg(reinterpret_cast<const V*>(x + t * ts + o1));
            B.at[j] = t << 8 | k;
        }
    };
    // Visits this lane's slots, a batch in flight: f(token, first and second
    // group's offset, their rotated values).  KEEP: the first batch, all there
    // is in a decode step, stays in registers for every visit.
    Batch first;
    if constexpr (KEEP) load(lane, first);
    auto visit = [&](auto&& f) {
        Batch B;
        if constexpr (KEEP) B = first;
        for (int i = lane; i < total; i += 32 * kPageBatch) {
            if (!KEEP || i != lane) load(i, B);
#pragma unroll
            for (int j = 0; j < kPageBatch; ++j) {
                if (i + 32 * j >= total) break;
                const int t = B.at[j] >> 8, k = B.at[j] & 255;
                float fa[GE], fb[GE];
                G::widen(B.a[j], fa);
                G::widen(B.b[j], fb);
                slot_rotate<MODE>(x + t * ts, k, cs + t * 2 * rope_pad(P.r.half), half, fa, fb);
                int o0, o1;
                slot_groups<MODE, GE>(k, half, o0, o1);
                f(t, o0, o1, fa, fb);
            }
        }
    };
    if constexpr (FMT == BSA_DTYPE_BF16) {
        uint16_t* c = static_cast<uint16_t*>(cache) + base;
        visit([&](int t, int o0, int o1, const float(&fa)[GE], const float(&fb)[GE]) {
            uint16_t* d = c + t * row;
            *reinterpret_cast<V*>(d + o0) = G::narrow(fa);
            *reinterpret_cast<V*>(d + o1) = G::narrow(fb);
        });
    } else {
        using F = Code<FMT>;
        uint8_t* c = static_cast<uint8_t*>(cache) + base;
        float m = 0.f;
        visit([&](int, int, int, const float(&fa)[GE], const float(&fb)[GE]) {
#pragma unroll
            for (int e = 0; e < GE; ++e) {
                const float u = fabsf(fa[e]), v = fabsf(fb[e]);
                if (u <= 3.402823466e38f) m = fmaxf(m, u);      // finite values only
                if (v <= 3.402823466e38f) m = fmaxf(m, v);
            }
        });
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        float s = fmaxf(old, F::scale(m));
        if (!(s > 0.f)) s = 1.f;
        if (s != old && S.off > 0) {
            // the kept codes follow the page's new scale
            const float ratio = old / s;
            const int parts = D / 16;
            for (int i = lane; i < S.off * parts; i += 32) {
                const int t = i / parts;
                uint4* p = reinterpret_cast<uint4*>(c + (int64_t)(t - S.off) * row) + (i - t * parts);
                uint4 v = *p;
                v.x = F::scaled(v.x, ratio);
                v.y = F::scaled(v.y, ratio);
                v.z = F::scaled(v.z, ratio);
                v.w = F::scaled(v.w, ratio);
                *p = v;
            }
        }
        const float inv = 1.f / s;      // exact: s is a power of two
        visit([&](int t, int o0, int o1, const float(&fa)[GE], const float(&fb)[GE]) {
            uint8_t* d = c + t * row;
            F::store(d + o0, fa, inv);
            F::store(d + o1, fb, inv);
        });
        __syncwarp();                    // every lane has read the old scale
        if (lane == 0) *sp = s;
    }
}

template <int FMT, RopeMode MODE, int GE, bool KEEP>
__global__ void __launch_bounds__(kAppendThreads, KEEP ? kAppendCtas / 2 : kAppendCtas) append_kernel(const AppendParams P) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ Row rows[kAppendTile];
    __shared__ Segment segs[kAppendTile];
    __shared__ int nseg, more;
    const int half = P.r.half, D = (int)P.a.D, tid = threadIdx.x;
    float* cs = reinterpret_cast<float*>(smem);      // [tile + 15][2 rope_pad(half)]
    unsigned long long* steps = reinterpret_cast<unsigned long long*>(cs + (P.tile + kPageRows - 1) * 2 * rope_pad(half));
    const int64_t t0 = (int64_t)blockIdx.x * P.tile;
    const int nt = (int)min((int64_t)P.tile, P.a.T - t0);
    if (tid == 0) nseg = more = 0;
    __syncthreads();
    // warp 0: the rows' places; the others: the frequencies' steps
    Segment seg{-1, 0, 0, 0};
    int64_t entry = -1;                              // the leader's block-table entry
    if (tid < nt) {
        const Row r = find_row(P, t0 + tid);
        rows[tid] = r;
        const int off = r.pos & (kPageRows - 1);
        if (r.pos >= 0 && (r.index == 0 || off == 0)) {
            seg.row = tid;
            seg.off = off;
            seg.n = min(kPageRows - off, r.left);
            const int64_t b = r.pos >> kLogPageSize;
            report_status(P.status, b >= P.a.max_blocks, BSA_STATUS_BAD_CONTEXT);
            if (b < P.a.max_blocks) entry = r.req * P.a.max_blocks + b;
            if (tid + seg.n > nt) more = tid + seg.n - nt;       // the tile's last segment alone
        }
    } else if (tid >= 32) {
        for (int i = tid - 32; i < half; i += kAppendThreads - 32) steps[i] = rope_step(__ldg(P.r.inv_freq + i));
    }
    const int32_t phys = entry >= 0 ? __ldg(P.a.block_table + entry) : -1;
    __syncthreads();
    if (entry >= 0) {
        seg.page = (int64_t)phys * kPagesPerBlock + ((rows[tid].pos & (kPageSize - 1)) >> 4);
        const bool good = phys >= 0 && seg.page < P.a.num_pages;
        report_status(P.status, !good, BSA_STATUS_BAD_BLOCK_ID);
        if (good) segs[atomicAdd(&nseg, 1)] = seg;
    }
    const int filled = nt + more;                    // table rows: the tile's and the last segment's
    for (int i = tid; i < filled * half; i += kAppendThreads) {
        const int t = i / half, f = i - t * half;
        int32_t p;
        if (P.r.positions != nullptr) {
            p = __ldg(P.r.positions + rope_axis(P.r, f) * P.a.T + t0 + t);
        } else {
            p = t < nt ? rows[t].pos : rows[nt - 1].pos + (t - nt + 1);
        }
        const float2 c = rope_turn(p, steps[f]);
        cs[t * 2 * rope_pad(half) + f] = c.x;
        cs[(t * 2 + 1) * rope_pad(half) + f] = P.r.inverse ? -c.y : c.y;
    }
    __syncthreads();
    // ---- pages: a warp per page, head and side ----
    const int warp = tid >> 5;
    for (int u = warp; u < nseg * 2 * P.a.H; u += kAppendThreads / 32) {
        const int side = u & 1, sh = u >> 1;
        const int i = sh / (int)P.a.H, h = sh - i * (int)P.a.H;
        const Segment S = segs[i];
        const int64_t t = t0 + S.row;
        const float* c = cs + S.row * 2 * rope_pad(half);
        if (side == 0)
            store_page<FMT, MODE, GE, KEEP>(P, static_cast<const uint16_t*>(P.a.k) + t * P.a.k_token_stride + h * P.a.k_head_stride,
                                       P.a.k_token_stride, S, h, c, true, P.a.k_cache, P.a.k_scale);
        else
            store_page<FMT, kSplit, 8, KEEP>(P, static_cast<const uint16_t*>(P.a.v) + t * P.a.v_token_stride + h * P.a.v_head_stride,
                                      P.a.v_token_stride, S, h, c, false, P.a.v_cache, P.a.v_scale);
    }
    // ---- queries: slots of two groups ----
    if (P.a.q == nullptr) return;
    using G = Group<uint16_t, GE>;
    using V = typename G::V;
    constexpr int B = kQueryBatch;
    const int ks = D / (2 * GE), Hq = (int)P.a.Hq, total = nt * Hq * ks;
    const uint16_t* __restrict__ q = static_cast<const uint16_t*>(P.a.q) + t0 * P.a.q_token_stride;
    uint16_t* __restrict__ o = static_cast<uint16_t*>(P.a.q_out) + t0 * Hq * D;
    // (row, head, slot) of this thread, advanced by the CTA's width; the
    // pages took the first warps' time, so the count starts at the last thread
    const int first = kAppendThreads - 1 - tid;
    int k = first % ks, th = first / ks;
    int h = Hq > 0 ? th % Hq : 0, t = Hq > 0 ? th / Hq : 0;
    const int dk = kAppendThreads % ks, dth = kAppendThreads / ks;
    const int dh = Hq > 0 ? dth % Hq : 0, dt = Hq > 0 ? dth / Hq : 0;
    for (int i = first; i < total; i += B * kAppendThreads) {
        V a[B], b[B];
        int kk[B], tt[B], hh[B];
#pragma unroll
        for (int j = 0; j < B; ++j) {
            kk[j] = k;
            tt[j] = t;
            hh[j] = h;
            if (i + j * kAppendThreads < total) {
                const uint16_t* xr = q + t * P.a.q_token_stride + h * P.a.q_head_stride;
                int o0, o1;
                slot_groups<MODE, GE>(k, half, o0, o1);
                a[j] = __ldg(reinterpret_cast<const V*>(xr + o0));
                b[j] = __ldg(reinterpret_cast<const V*>(xr + o1));
            }
            k += dk;
            h += dh;
            t += dt;
            if (k >= ks) {
                k -= ks;
                ++h;
            }
            if (h >= Hq) {
                h -= Hq;
                ++t;
            }
        }
#pragma unroll
        for (int j = 0; j < B; ++j) {
            if (i + j * kAppendThreads >= total) break;
            const uint16_t* xr = q + tt[j] * P.a.q_token_stride + hh[j] * P.a.q_head_stride;
            uint16_t* orow = o + ((int64_t)tt[j] * Hq + hh[j]) * D;
            int o0, o1;
            slot_groups<MODE, GE>(kk[j], half, o0, o1);
            if (rows[tt[j]].pos < 0) {
                // padding: zeros, whatever the query holds
                *reinterpret_cast<V*>(orow + o0) = V{};
                *reinterpret_cast<V*>(orow + o1) = V{};
                continue;
            }
            float fa[GE], fb[GE];
            G::widen(a[j], fa);
            G::widen(b[j], fb);
            slot_rotate<MODE>(xr, kk[j], cs + tt[j] * 2 * rope_pad(half), half, fa, fb);
            *reinterpret_cast<V*>(orow + o0) = G::narrow(fa);
            *reinterpret_cast<V*>(orow + o1) = G::narrow(fb);
        }
    }
}

// Half-split pairs whose distance is a multiple of 4 go by groups of 4 (two
// 8192-token prompts with 104 of 128 rotated 72 us, by single partners 128; 1452
// decode rows with 40 of 64 rotated 8.0 and 19.1).
template <int FMT, bool KEEP>
cudaError_t launch_mode(const AppendParams& P, unsigned grid, size_t smem, cudaStream_t st) {
    const RopeMode mode = rope_mode(P.r, 8);
    if (mode == kSplit) append_kernel<FMT, kSplit, 8, KEEP><<<grid, kAppendThreads, smem, st>>>(P);
    else if (mode == kInterleaved) append_kernel<FMT, kInterleaved, 8, KEEP><<<grid, kAppendThreads, smem, st>>>(P);
    else if (rope_mode(P.r, 4) == kSplit) append_kernel<FMT, kSplit, 4, KEEP><<<grid, kAppendThreads, smem, st>>>(P);
    else append_kernel<FMT, kSplitAny, 8, KEEP><<<grid, kAppendThreads, smem, st>>>(P);
    return cudaGetLastError();
}

template <int FMT>
cudaError_t launch_format(const AppendParams& P, bool keep, unsigned grid, size_t smem, cudaStream_t st) {
    return keep ? launch_mode<FMT, true>(P, grid, smem, st) : launch_mode<FMT, false>(P, grid, smem, st);
}

// Rows per CTA, and whether its lanes keep what they read of the tokens or read
// it twice, the second time from L1.  Keeping takes registers for two CTAs per SM,
// reading twice leaves four.  So calls whose CTAs of up to 8 rows fit at two
// per SM keep, in CTAs of as few rows as fit; longer ones do not, in CTAs of 8
// rows while those fit at four per SM, then of 16, a page's.  A sixteenth more than fits
// still counts as fitting: the CTAs left over are few and start early.
// (4 KV x 8 query heads of 128, e4m3, us, kept / not: 256 production rows 4.9 / 5.4;
// 2500 rows, 8 per CTA, 16.6 / 19.0; 3360 rows, 8 per CTA, 22.4 / 19.9; two 8192-token
// prompts 63 / 60.  750 rows kept, 2 and 4 per CTA, 10.9 and 9.2; 4758 rows not
// kept, 8 and 16 per CTA, 23.8 and 28.3; 8547 rows 38.8 and 37.1.)
struct Tiling {
    int rows;
    bool keep;
};
Tiling pick_tiling(int64_t T, int64_t sms) {
    auto fits = [&](int rows, int64_t ctas) { return (T + rows - 1) / rows <= sms * ctas * 17 / 16; };
    for (int rows = 1; rows < kAppendTile; rows *= 2)
        if (fits(rows, kAppendCtas / 2)) return {rows, true};
    return {fits(kAppendTile / 2, kAppendCtas) ? kAppendTile / 2 : kAppendTile, false};
}

int check_append(const bsa_append_args_t* a) {
    if (a->cache_dtype != BSA_DTYPE_BF16 && a->cache_dtype != BSA_DTYPE_E4M3 && a->cache_dtype != BSA_DTYPE_E5M2)
        return BSA_ERR_DTYPE;
    if (a->T < 0 || a->T > INT32_MAX || a->H < 1 || a->H > 65536 || a->Hq < 0 || a->Hq > 65536 ||
        a->D < 16 || a->D > BSA_MAX_CACHE_DIM || a->D % 16 != 0 || a->num_pages < 0 ||
        a->num_reqs < 0 || a->num_reqs > INT32_MAX || a->max_blocks < 0 || a->max_blocks > (INT32_MAX >> kLogPageSize))
        return BSA_ERR_SHAPE;
    const int64_t strides[6] = {a->k_token_stride, a->k_head_stride, a->v_token_stride,
                                a->v_head_stride, a->q_token_stride, a->q_head_stride};
    for (int i = 0; i < (a->q != nullptr ? 6 : 4); ++i) {
        if (strides[i] < 0) return BSA_ERR_SHAPE;
        if (strides[i] % 8 != 0) return BSA_ERR_ALIGN;
    }
    if ((a->q == nullptr) != (a->q_out == nullptr)) return BSA_ERR_NULL;
    const int rc = check_rope(a->D, a->positions, a->axes, a->inv_freq, a->freq_axis, a->rot_dim, a->flags, false);
    if (rc != BSA_OK) return rc;
    if (a->T == 0) return BSA_OK;
    if (a->k == nullptr || a->v == nullptr || (a->num_pages > 0 && (a->k_cache == nullptr || a->v_cache == nullptr)) ||
        (a->num_reqs * a->max_blocks > 0 && a->block_table == nullptr))
        return BSA_ERR_NULL;
    if (a->cache_dtype != BSA_DTYPE_BF16 && a->num_pages > 0 && (a->k_scale == nullptr || a->v_scale == nullptr))
        return BSA_ERR_NULL;
    const void* wide[6] = {a->k, a->v, a->q, a->q_out, a->k_cache, a->v_cache};
    for (const void* p : wide)
        if ((reinterpret_cast<uintptr_t>(p) & 15) != 0) return BSA_ERR_ALIGN;
    if (((reinterpret_cast<uintptr_t>(a->k_scale) | reinterpret_cast<uintptr_t>(a->v_scale)) & 3) != 0)
        return BSA_ERR_ALIGN;
    return BSA_OK;
}

// The arguments with the strides along dimensions of one entry set to 0: they
// may be anything.
bsa_append_args_t plain_strides(bsa_append_args_t a) {
    if (a.T == 1) a.k_token_stride = a.v_token_stride = a.q_token_stride = 0;
    if (a.H == 1) a.k_head_stride = a.v_head_stride = 0;
    if (a.Hq == 1) a.q_head_stride = 0;
    return a;
}

// Nothing that the call writes shares memory with anything else of it.
bool outputs_apart(const bsa_append_args_t& a) {
    auto heads = [&](const void* p, int64_t H, int64_t ts, int64_t hs) { return Rows{p, p != nullptr ? a.T : 0, H, a.D * 2, ts * 2, hs * 2}; };
    const int64_t cache = a.num_pages * kPageRows * a.H * a.D * (a.cache_dtype == BSA_DTYPE_BF16 ? 2 : 1);
    const int64_t scales = a.cache_dtype == BSA_DTYPE_BF16 ? 0 : a.num_pages * a.H * 4;
    const Rows r[8] = {whole_rows(a.q_out, a.q_out != nullptr ? a.T * a.Hq * a.D * 2 : 0),
                       whole_rows(a.k_cache, cache), whole_rows(a.v_cache, cache),
                       whole_rows(a.k_scale, scales), whole_rows(a.v_scale, scales),
                       heads(a.q, a.Hq, a.q_token_stride, a.q_head_stride),
                       heads(a.k, a.H, a.k_token_stride, a.k_head_stride), heads(a.v, a.H, a.v_token_stride, a.v_head_stride)};
    for (int i = 0; i < 5; ++i)
        for (int j = i + 1; j < 8; ++j)
            if (rows_overlap(r[i], r[j])) return false;
    return true;
}

int launch_append(AppendParams& P, cudaStream_t st) {
    if (!outputs_apart(P.a)) return BSA_ERR_SHAPE;
    P.r = RopeParams{P.a.positions, P.a.T, P.a.inv_freq, P.a.freq_axis, P.a.axes, P.a.rot_dim / 2,
                     (P.a.flags & BSA_ROPE_INTERLEAVED) != 0, (P.a.flags & BSA_ROPE_INVERSE) != 0};
    P.status = current_status_word();
    if (P.a.q == nullptr) P.a.Hq = 0;
    const Tiling tiling = pick_tiling(P.a.T, device_sm_count());
    const int tile = tiling.rows;
    P.tile = tile;
    const size_t smem = (size_t)(tile + kPageRows - 1) * 2 * rope_pad(P.r.half) * sizeof(float) + P.r.half * sizeof(unsigned long long);
    const unsigned grid = (unsigned)((P.a.T + tile - 1) / tile);
    cudaError_t e;
    if (P.a.cache_dtype == BSA_DTYPE_BF16) e = launch_format<BSA_DTYPE_BF16>(P, tiling.keep, grid, smem, st);
    else if (P.a.cache_dtype == BSA_DTYPE_E4M3) e = launch_format<BSA_DTYPE_E4M3>(P, tiling.keep, grid, smem, st);
    else e = launch_format<BSA_DTYPE_E5M2>(P, tiling.keep, grid, smem, st);
    return e == cudaSuccess ? BSA_OK : (int)e;
}

}  // namespace
}  // namespace bsa

using namespace bsa;

extern "C" int bsa_append_kv_decode(const bsa_append_args_t* args, const int32_t* seq_lens,
                                    int32_t decode_query_len, void* stream) {
    if (args == nullptr) return BSA_ERR_NULL;
    AppendParams P{};
    P.a = plain_strides(*args);
    const int rc = check_append(&P.a);
    if (rc != BSA_OK) return rc;
    if (decode_query_len < 1) return BSA_ERR_SHAPE;
    if (P.a.T != P.a.num_reqs * decode_query_len) return BSA_ERR_ROWS;
    if (P.a.T == 0) return BSA_OK;
    if (seq_lens == nullptr) return BSA_ERR_NULL;
    P.seq_lens = seq_lens;
    P.dql = decode_query_len;
    return launch_append(P, static_cast<cudaStream_t>(stream));
}

extern "C" int bsa_append_kv_varlen(const bsa_append_args_t* args, const int32_t* cu_seqlens_q,
                                    const int32_t* prefix_lens, void* stream) {
    if (args == nullptr) return BSA_ERR_NULL;
    AppendParams P{};
    P.a = plain_strides(*args);
    const int rc = check_append(&P.a);
    if (rc != BSA_OK) return rc;
    if (P.a.T == 0) return BSA_OK;
    if (cu_seqlens_q == nullptr || (P.a.num_reqs > 0 && prefix_lens == nullptr)) return BSA_ERR_NULL;
    P.cu = cu_seqlens_q;
    P.prefix = prefix_lens;
    return launch_append(P, static_cast<cudaStream_t>(stream));
}
