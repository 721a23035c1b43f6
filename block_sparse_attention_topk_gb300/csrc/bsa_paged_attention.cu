// bsa_paged_attention.cu -- causal attention of new tokens over everything
// their sequences hold in the paged cache, with an optional sliding window and
// sinks, from a bf16 cache or an 8-bit one.
//
// What it computes, for query head g of KV head h in the row at position p:
//   out = sum_j softmax_j(scale q . k_j) v_j
// over the tokens j <= p of the row's sequence, with a window only those with
// j > p - window or j < sinks; in 8 bits k_j and v_j are codes times the scale of
// their page and head.
//
// A warp takes a row's query head and walks its tokens one at a time with a
// running maximum and sum; each lane holds D / 32 of its dimensions.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "bsa_internal.h"
#include "bsa_overlap.h"

namespace bsa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 4;

struct PagedParams {
    bsa_paged_attention_args_t a;
    const int32_t* seq_lens;      // decode form
    int32_t dql;
    const int32_t* cu;            // varlen form
    const int32_t* prefix;
    uint32_t* status;
};

// The sequence and position of row t; false for rows of no sequence.
__device__ __forceinline__ bool place_row(const PagedParams& P, int64_t t, int64_t* req, int64_t* pos) {
    if (P.cu == nullptr) {
        *req = t / P.dql;
        *pos = (int64_t)__ldg(P.seq_lens + *req) - P.dql + t % P.dql;
        return true;
    }
    int64_t lo = 0, hi = P.a.num_reqs;      // the last sequence that starts at or before t
    while (lo < hi) {
        const int64_t mid = (lo + hi) / 2;
        if (__ldg(P.cu + mid + 1) <= t) lo = mid + 1;
        else hi = mid;
    }
    if (lo >= P.a.num_reqs || __ldg(P.cu + lo) > t) return false;
    *req = lo;
    *pos = (int64_t)__ldg(P.prefix + lo) + t - __ldg(P.cu + lo);
    return true;
}

template <int DTYPE>
__device__ __forceinline__ float load_value(const void* p, int64_t i) {
    if constexpr (DTYPE == BSA_DTYPE_BF16) return __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(p) + i) << 16);
    const __nv_fp8_storage_t c = __ldg(static_cast<const uint8_t*>(p) + i);
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, DTYPE == BSA_DTYPE_E4M3 ? __NV_E4M3 : __NV_E5M2)));
}

template <int DTYPE>
__global__ void __launch_bounds__(kWarps * 32) paged_attention_kernel(const PagedParams P) {
    constexpr int R = BSA_MAX_CACHE_DIM / 32;
    const auto& a = P.a;
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (row >= a.T * a.H * a.G) return;
    const int64_t t = row / (a.H * a.G), h = row / a.G % a.H;
    float q[R], o[R], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int d = lane + 32 * r;
        q[r] = d < a.D ? load_value<BSA_DTYPE_BF16>(a.q, row * a.D + d) : 0.f;
        o[r] = 0.f;
    }
    int64_t req, pos;
    if (place_row(P, t, &req, &pos) && pos >= 0) {
        const int64_t top = a.max_blocks * kPageSize;
        report_status(P.status, pos >= top && lane == 0, BSA_STATUS_BAD_CONTEXT);
        const int64_t end = pos < top ? pos + 1 : top;
        int64_t j = 0;
        while (j < end) {
            if (a.window > 0 && j >= a.sinks && j <= pos - a.window) {
                j = pos - a.window + 1;
                continue;
            }
            const int64_t page = (int64_t)__ldg(a.block_table + req * a.max_blocks + j / kPageSize) * kPagesPerBlock + j % kPageSize / kSubPage;
            if (page < 0 || page >= a.num_pages) {
                report_status(P.status, lane == 0, BSA_STATUS_BAD_BLOCK_ID);
                ++j;
                continue;
            }
            const int64_t at = ((page * kSubPage + j % kSubPage) * a.H + h) * a.D;
            float s = 0.f;
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (lane + 32 * r < a.D) s = fmaf(q[r], load_value<DTYPE>(a.k_cache, at + lane + 32 * r), s);
#pragma unroll
            for (int i = 16; i > 0; i >>= 1) s += __shfl_xor_sync(kFull, s, i);
            float ks = 1.f, vs = 1.f;
            if (DTYPE != BSA_DTYPE_BF16) {
                ks = __ldg(a.k_scale + page * a.H + h);
                vs = __ldg(a.v_scale + page * a.H + h);
            }
            s *= ks * a.scale * 1.44269504f;
            const float m_new = fmaxf(m, s), base = m_new == -INFINITY ? 0.f : m_new;
            const float keep = exp2f(m - base), p = exp2f(s - base);
            l = fmaf(l, keep, p);
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (lane + 32 * r < a.D) o[r] = fmaf(o[r], keep, p * vs * load_value<DTYPE>(a.v_cache, at + lane + 32 * r));
            m = m_new;
            ++j;
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (lane + 32 * r < a.D) static_cast<__nv_bfloat16*>(a.out)[row * a.D + lane + 32 * r] = __float2bfloat16_rn(l == 0.f ? 0.f : o[r] * inv);
}

bool paged_sizes_ok(int64_t T, int64_t H, int64_t G, int64_t D) {
    return T >= 0 && T <= INT32_MAX && H >= 1 && H <= 65536 && G >= 1 && G <= BSA_MAX_PAGED_GROUP && T * H * G <= INT32_MAX &&
           D >= 16 && D <= BSA_MAX_CACHE_DIM && D % 16 == 0;
}

// The checks that both forms share; `ints`: the form's own index tensors.
int check_paged(const bsa_paged_attention_args_t& a, const Rows (&ints)[2]) {
    if (a.cache_dtype != BSA_DTYPE_BF16 && a.cache_dtype != BSA_DTYPE_E4M3 && a.cache_dtype != BSA_DTYPE_E5M2) return BSA_ERR_DTYPE;
    if (!paged_sizes_ok(a.T, a.H, a.G, a.D) || a.num_pages < 0 || a.num_pages >= (1ll << 27) || a.num_reqs < 0 ||
        a.num_reqs > (1 << 24) || a.max_blocks < 0 || a.max_blocks >= (1 << 24) || a.window < 0 || a.sinks < 0)
        return BSA_ERR_SHAPE;
    if (a.T == 0) return BSA_OK;
    const bool bits8 = a.cache_dtype != BSA_DTYPE_BF16;
    if (a.q == nullptr || a.out == nullptr || (a.num_reqs > 0 && a.max_blocks > 0 && a.block_table == nullptr)) return BSA_ERR_NULL;
    if (a.num_pages > 0 && (a.k_cache == nullptr || a.v_cache == nullptr || (bits8 && (a.k_scale == nullptr || a.v_scale == nullptr))))
        return BSA_ERR_NULL;
    const void* wide[4] = {a.q, a.out, a.k_cache, a.v_cache};
    for (const void* p : wide)
        if ((reinterpret_cast<uintptr_t>(p) & 15) != 0) return BSA_ERR_ALIGN;
    const int64_t rows = a.T * a.H * a.G * a.D * 2, cache = a.num_pages * kSubPage * a.H * a.D * (bits8 ? 1 : 2);
    const int64_t scales = bits8 ? a.num_pages * a.H * 4 : 0;
    const Rows in[8] = {whole_rows(a.q, rows), whole_rows(a.k_cache, cache), whole_rows(a.v_cache, cache),
                        whole_rows(a.k_scale, scales), whole_rows(a.v_scale, scales),
                        whole_rows(a.block_table, a.num_reqs * a.max_blocks * 4), ints[0], ints[1]};
    for (const Rows& r : in)
        if (rows_overlap(whole_rows(a.out, rows), r)) return BSA_ERR_SHAPE;
    return BSA_OK;
}

int launch_paged(PagedParams& P, cudaStream_t st) {
    P.status = current_status_word();
    const unsigned grid = (unsigned)((P.a.T * P.a.H * P.a.G + kWarps - 1) / kWarps);
    if (P.a.cache_dtype == BSA_DTYPE_BF16) paged_attention_kernel<BSA_DTYPE_BF16><<<grid, kWarps * 32, 0, st>>>(P);
    else if (P.a.cache_dtype == BSA_DTYPE_E4M3) paged_attention_kernel<BSA_DTYPE_E4M3><<<grid, kWarps * 32, 0, st>>>(P);
    else paged_attention_kernel<BSA_DTYPE_E5M2><<<grid, kWarps * 32, 0, st>>>(P);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? BSA_OK : (int)e;
}

}  // namespace
}  // namespace bsa

using namespace bsa;

extern "C" size_t bsa_paged_attention_workspace_bytes(int64_t T, int64_t H, int64_t G, int64_t D) { return 0; }

extern "C" int bsa_paged_attention_decode(const bsa_paged_attention_args_t* args, const int32_t* seq_lens, int32_t decode_query_len,
                                          void* stream) {
    if (args == nullptr) return BSA_ERR_NULL;
    PagedParams P{};
    P.a = *args;
    const Rows ints[2] = {whole_rows(seq_lens, P.a.num_reqs * 4), whole_rows(nullptr, 0)};
    const int rc = check_paged(P.a, ints);
    if (rc != BSA_OK) return rc;
    if (decode_query_len < 1) return BSA_ERR_SHAPE;
    if (P.a.T != P.a.num_reqs * decode_query_len) return BSA_ERR_ROWS;
    if (P.a.T == 0) return BSA_OK;
    if (seq_lens == nullptr) return BSA_ERR_NULL;
    P.seq_lens = seq_lens;
    P.dql = decode_query_len;
    return launch_paged(P, static_cast<cudaStream_t>(stream));
}

extern "C" int bsa_paged_attention_varlen(const bsa_paged_attention_args_t* args, const int32_t* cu_seqlens_q,
                                          const int32_t* prefix_lens, void* stream) {
    if (args == nullptr) return BSA_ERR_NULL;
    PagedParams P{};
    P.a = *args;
    const Rows ints[2] = {whole_rows(cu_seqlens_q, (P.a.num_reqs + 1) * 4), whole_rows(prefix_lens, P.a.num_reqs * 4)};
    const int rc = check_paged(P.a, ints);
    if (rc != BSA_OK) return rc;
    if (P.a.T == 0) return BSA_OK;
    if (cu_seqlens_q == nullptr || (P.a.num_reqs > 0 && prefix_lens == nullptr)) return BSA_ERR_NULL;
    P.cu = cu_seqlens_q;
    P.prefix = prefix_lens;
    return launch_paged(P, static_cast<cudaStream_t>(stream));
}
