// bsa_append.cu -- a step's keys (rotated) and values into the paged cache, in
// bf16 or in 8 bits with a scale per page and head; the step's queries are
// rotated in the same launch.
//
// One CTA per token row.  The row that is the call's first in its page (its
// leader) takes all of the call's tokens in that page: at most 16, which
// follow it.  So a page has one writer and its scale is one maximum.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "bsa_internal.h"
#include "bsa_rope.cuh"

namespace bsa {
namespace {

constexpr int kAppendThreads = 128;

struct AppendParams {
    bsa_append_args_t a;
    RopeParams r;
    const int32_t* seq_lens;   // decode form, else null
    int32_t dql;
    const int32_t* cu;         // varlen form
    const int32_t* prefix;
    uint32_t* status;
};

__device__ __forceinline__ float bf(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ uint16_t to_bf(float f) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(f));
}

// The 8-bit types.  The power-of-two scale of a maximum m = f * 2^e, f in
// [1, 2), is 2^(e - 8) or 2^(e - 15), one more when f > 1.75 (both types end
// at 1.75 * 2^k).
template <int FMT>
struct Code {
    static constexpr int kTop = FMT == BSA_DTYPE_E4M3 ? 8 : 15;
    static constexpr __nv_fp8_interpretation_t kKind = FMT == BSA_DTYPE_E4M3 ? __NV_E4M3 : __NV_E5M2;
    __device__ static uint8_t pack(float x) { return __nv_cvt_float_to_fp8(x, __NV_SATFINITE, kKind); }
    __device__ static float unpack(uint8_t c) {
        return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, kKind)));
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

// value d of a head's row, rotated by the row's (cos, sin) table
__device__ __forceinline__ float turned(const uint16_t* x, int d, const float2* cs,
                                        const RopeParams& R) {
    const int half = R.half;
    if (d >= 2 * half) return bf(x[d]);
    const int i = R.interleaved ? d >> 1 : (d < half ? d : d - half);
    const int ia = R.interleaved ? 2 * i : i;
    const int ib = R.interleaved ? 2 * i + 1 : i + half;
    const float a = bf(x[ia]), b = bf(x[ib]);
    const float2 c = cs[i];
    return d == ia ? a * c.x - b * c.y : b * c.x + a * c.y;
}

__device__ float block_max(float m, float* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
    m = red[0];
#pragma unroll
    for (int w = 1; w < kAppendThreads / 32; ++w) m = fmaxf(m, red[w]);
    return m;
}

// n tokens of one head into page slots [off, off + n); cs null: not rotated
template <int FMT>
__device__ void store_page(const AppendParams& P, const uint16_t* x, int64_t ts, int n, int off,
                           int64_t page, int h, const float2* cs, void* cache, float* scales, float* red) {
    const int D = (int)P.a.D;
    const int64_t row = P.a.H * D;
    const int64_t base = page * BSA_SUB_PAGE_SIZE * row + (int64_t)h * D;
    auto value = [&](int i) {
        const int t = i / D, d = i - t * D;
        const uint16_t* xr = x + t * ts;
        return cs != nullptr ? turned(xr, d, cs + t * P.r.half, P.r) : bf(xr[d]);
    };
    if constexpr (FMT == BSA_DTYPE_BF16) {
        uint16_t* c = static_cast<uint16_t*>(cache) + base;
        for (int i = threadIdx.x; i < n * D; i += kAppendThreads)
            c[(off + i / D) * row + i % D] = to_bf(value(i));
    } else {
        using F = Code<FMT>;
        uint8_t* c = static_cast<uint8_t*>(cache) + base;
        float m = 0.f;
        for (int i = threadIdx.x; i < n * D; i += kAppendThreads) {
            const float a = fabsf(value(i));
            if (a <= 3.402823466e38f) m = fmaxf(m, a);
        }
        m = block_max(m, red);
        float* sp = scales + page * P.a.H + h;
        const float old = off > 0 ? *sp : 0.f;
        float s = fmaxf(old, F::scale(m));
        if (!(s > 0.f)) s = 1.f;
        if (s != old && off > 0) {
            const float ratio = old / s;
            for (int i = threadIdx.x; i < off * D; i += kAppendThreads) {
                uint8_t* p = c + (i / D) * row + i % D;
                *p = F::pack(F::unpack(*p) * ratio);
            }
        }
        for (int i = threadIdx.x; i < n * D; i += kAppendThreads)
            c[(off + i / D) * row + i % D] = F::pack(value(i) / s);
        __syncthreads();                 // every thread has read the old scale
        if (threadIdx.x == 0) *sp = s;
    }
}

template <int FMT>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendParams P) {
    extern __shared__ __align__(16) float2 cs[];      // [16][half]
    __shared__ float red[kAppendThreads / 32];
    __shared__ Row sh;
    const int64_t t = blockIdx.x;
    if (threadIdx.x == 0) sh = find_row(P, t);
    __syncthreads();
    const Row r = sh;
    const int D = (int)P.a.D, half = P.r.half;
    const int off = r.pos & 15;
    const bool leader = r.pos >= 0 && (r.index == 0 || off == 0);
    const int n = leader ? min(16 - off, r.left) : 1;
    if (r.pos >= 0) {
        for (int i = threadIdx.x; i < n * half; i += kAppendThreads) {
            const int j = i / half, f = i - j * half;
            const int32_t p = P.r.positions == nullptr
                                  ? r.pos + j
                                  : __ldg(P.r.positions + rope_axis(P.r, f) * P.a.T + t + j);
            float2 c = rope_turn(p, rope_step(__ldg(P.r.inv_freq + f)));
            if (P.r.inverse) c.y = -c.y;
            cs[i] = c;
        }
    }
    __syncthreads();
    if (P.a.q != nullptr) {
        const uint16_t* q = static_cast<const uint16_t*>(P.a.q) + t * P.a.q_token_stride;
        uint16_t* o = static_cast<uint16_t*>(P.a.q_out) + t * P.a.Hq * D;
        for (int i = threadIdx.x; i < P.a.Hq * D; i += kAppendThreads) {
            const int h = i / D, d = i - h * D;
            o[i] = r.pos >= 0 ? to_bf(turned(q + h * P.a.q_head_stride, d, cs, P.r)) : (uint16_t)0;
        }
    }
    if (!leader) return;
    const int64_t b = r.pos >> kLogPageSize;
    if (b >= P.a.max_blocks) {
        if (threadIdx.x == 0) report_status(P.status, true, BSA_STATUS_BAD_CONTEXT);
        return;
    }
    const int32_t phys = __ldg(P.a.block_table + r.req * P.a.max_blocks + b);
    const int64_t page = (int64_t)phys * kPagesPerBlock + ((r.pos & (kPageSize - 1)) >> 4);
    if (phys < 0 || page >= P.a.num_pages) {
        if (threadIdx.x == 0) report_status(P.status, true, BSA_STATUS_BAD_BLOCK_ID);
        return;
    }
    for (int h = 0; h < P.a.H; ++h) {
        store_page<FMT>(P, static_cast<const uint16_t*>(P.a.k) + t * P.a.k_token_stride + h * P.a.k_head_stride,
                        P.a.k_token_stride, n, off, page, h, half > 0 ? cs : nullptr, P.a.k_cache, P.a.k_scale, red);
        store_page<FMT>(P, static_cast<const uint16_t*>(P.a.v) + t * P.a.v_token_stride + h * P.a.v_head_stride,
                        P.a.v_token_stride, n, off, page, h, nullptr, P.a.v_cache, P.a.v_scale, red);
    }
}

int check_append(const bsa_append_args_t* a) {
    if (a == nullptr) return BSA_ERR_NULL;
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

int launch_append(AppendParams& P, cudaStream_t st) {
    P.r = RopeParams{P.a.positions, P.a.T, P.a.inv_freq, P.a.freq_axis, P.a.axes, P.a.rot_dim / 2,
                     (P.a.flags & BSA_ROPE_INTERLEAVED) != 0, (P.a.flags & BSA_ROPE_INVERSE) != 0};
    P.status = current_status_word();
    const size_t smem = (size_t)16 * P.r.half * sizeof(float2);
    const unsigned grid = (unsigned)P.a.T;
    if (P.a.cache_dtype == BSA_DTYPE_BF16) append_kernel<BSA_DTYPE_BF16><<<grid, kAppendThreads, smem, st>>>(P);
    else if (P.a.cache_dtype == BSA_DTYPE_E4M3) append_kernel<BSA_DTYPE_E4M3><<<grid, kAppendThreads, smem, st>>>(P);
    else append_kernel<BSA_DTYPE_E5M2><<<grid, kAppendThreads, smem, st>>>(P);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? BSA_OK : (int)e;
}

}  // namespace
}  // namespace bsa

using namespace bsa;

extern "C" int bsa_append_kv_decode(const bsa_append_args_t* args, const int32_t* seq_lens,
                                    int32_t decode_query_len, void* stream) {
    const int rc = check_append(args);
    if (rc != BSA_OK) return rc;
    if (decode_query_len < 1) return BSA_ERR_SHAPE;
    if (args->T != args->num_reqs * decode_query_len) return BSA_ERR_ROWS;
    if (args->T == 0) return BSA_OK;
    if (seq_lens == nullptr) return BSA_ERR_NULL;
    AppendParams P{};
    P.a = *args;
    P.seq_lens = seq_lens;
    P.dql = decode_query_len;
    return launch_append(P, static_cast<cudaStream_t>(stream));
}

extern "C" int bsa_append_kv_varlen(const bsa_append_args_t* args, const int32_t* cu_seqlens_q,
                                    const int32_t* prefix_lens, void* stream) {
    const int rc = check_append(args);
    if (rc != BSA_OK) return rc;
    if (args->T == 0) return BSA_OK;
    if (cu_seqlens_q == nullptr || (args->num_reqs > 0 && prefix_lens == nullptr)) return BSA_ERR_NULL;
    AppendParams P{};
    P.a = *args;
    P.cu = cu_seqlens_q;
    P.prefix = prefix_lens;
    return launch_append(P, static_cast<cudaStream_t>(stream));
}
