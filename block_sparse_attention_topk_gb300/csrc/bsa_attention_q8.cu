// bsa_attention_q8.cu -- sparse decode attention over a paged cache held in 8
// bits with a scale per 16-token page and head.
//
// out = softmax(scale * q . (kc * ks)) (vc * vs) over the row's first ctx
// table tokens.  One CTA of 4 warps per row and query head; each warp walks
// 32 tokens at a time with a running maximum and sum, and the warps' partial
// results join in shared memory.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "bsa_internal.h"

namespace bsa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kQ8Warps = 4;

struct Q8Params {
    const uint16_t* q;
    const uint8_t* k;
    const uint8_t* v;
    const float* ks;
    const float* vs;
    const int32_t* bt;
    const int32_t* ctx;
    uint16_t* out;
    int64_t num_pages;
    int32_t H, G, width;
    float scale;
    uint32_t* status;
};

template <__nv_fp8_interpretation_t KIND>
__device__ __forceinline__ float unpack8(uint8_t c) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, KIND)));
}

template <int D, __nv_fp8_interpretation_t KIND>
__global__ void __launch_bounds__(kQ8Warps * 32) attention_q8_kernel(const Q8Params A) {
    constexpr int DL = D / 32;
    __shared__ float qs[D];
    __shared__ float pm[kQ8Warps], pl[kQ8Warps], pacc[kQ8Warps][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = blockIdx.x;
    const int g = blockIdx.y, h = (int)(row % A.H);
    const int32_t* bt = A.bt + row * A.width;
    const int ctx_in = __ldg(A.ctx + row);
    const int ctx = max(0, min(ctx_in, A.width * kSubPage));
    if (threadIdx.x == 0) report_status(A.status, ctx != ctx_in, BSA_STATUS_BAD_CONTEXT);
    for (int i = threadIdx.x; i < D; i += kQ8Warps * 32)
        qs[i] = __uint_as_float((uint32_t)A.q[(row * A.G + g) * D + i] << 16);
    __syncthreads();
    const int64_t slot = (int64_t)A.H * D;
    float m = -INFINITY, l = 0.f, acc[DL];
#pragma unroll
    for (int d = 0; d < DL; ++d) acc[d] = 0.f;
    for (int tile = 32 * warp; tile < ctx; tile += 32 * kQ8Warps) {
        const int j = tile + lane;
        const int32_t page = j < ctx ? __ldg(bt + (j >> 4)) : -1;
        const bool ok = page >= 0 && page < A.num_pages;
        report_status(A.status, j < ctx && !ok, BSA_STATUS_BAD_PAGE);
        float s = -INFINITY, vs = 0.f;
        if (ok) {
            const uint8_t* kr = A.k + ((int64_t)page * kSubPage + (j & 15)) * slot + h * D;
            float a = 0.f;
            for (int d = 0; d < D; ++d) a = fmaf(qs[d], unpack8<KIND>(kr[d]), a);
            s = a * A.ks[(int64_t)page * A.H + h] * A.scale;
            vs = A.vs[(int64_t)page * A.H + h];
        }
        float mn = s;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(kFull, mn, o));
        mn = fmaxf(mn, m);
        const float corr = mn == -INFINITY ? 1.f : expf(m - mn);
        float p = ok ? expf(s - mn) : 0.f;
        float sum = p;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
        l = l * corr + sum;
#pragma unroll
        for (int d = 0; d < DL; ++d) acc[d] *= corr;
        m = mn;
        p *= vs;
        for (int u = 0; u < 32; ++u) {
            const int32_t pu = __shfl_sync(kFull, ok ? page : -1, u);
            const float w = __shfl_sync(kFull, p, u);
            if (pu < 0) continue;
            const uint8_t* vr = A.v + ((int64_t)pu * kSubPage + (u & 15)) * slot + h * D;
#pragma unroll
            for (int d = 0; d < DL; ++d) acc[d] = fmaf(w, unpack8<KIND>(vr[lane + 32 * d]), acc[d]);
        }
    }
    if (lane == 0) {
        pm[warp] = m;
        pl[warp] = l;
    }
#pragma unroll
    for (int d = 0; d < DL; ++d) pacc[warp][lane + 32 * d] = acc[d];
    __syncthreads();
    float mx = -INFINITY;
    for (int w = 0; w < kQ8Warps; ++w) mx = fmaxf(mx, pm[w]);
    for (int d = threadIdx.x; d < D; d += kQ8Warps * 32) {
        float den = 0.f, num = 0.f;
        for (int w = 0; w < kQ8Warps; ++w) {
            const float e = pm[w] == -INFINITY ? 0.f : expf(pm[w] - mx);
            den = fmaf(pl[w], e, den);
            num = fmaf(pacc[w][d], e, num);
        }
        // NaN scores stay NaN; an empty context gives zeros
        A.out[(row * A.G + g) * D + d] =
            __bfloat16_as_ushort(__float2bfloat16_rn(den == 0.f ? 0.f : num / den));
    }
}

template <int D>
cudaError_t launch_q8(const Q8Params& A, int64_t rows, bool e4m3, cudaStream_t st) {
    const dim3 grid((unsigned)rows, (unsigned)A.G);
    if (e4m3) attention_q8_kernel<D, __NV_E4M3><<<grid, kQ8Warps * 32, 0, st>>>(A);
    else attention_q8_kernel<D, __NV_E5M2><<<grid, kQ8Warps * 32, 0, st>>>(A);
    return cudaGetLastError();
}

bool sizes_ok(int64_t T, int64_t H, int64_t G, int64_t D) {
    return T >= 0 && H >= 1 && H <= 65536 && T * H <= INT32_MAX && G >= 1 &&
           G <= BSA_MAX_ATTN_Q8_GROUP && (D == 64 || D == 128 || D == 256);
}

}  // namespace
}  // namespace bsa

using namespace bsa;

extern "C" size_t bsa_attention_q8_workspace_bytes(int64_t, int64_t, int64_t, int64_t, int32_t) {
    return 0;
}

extern "C" int bsa_sparse_decode_attention_q8(const void* q, const void* k_cache, const void* v_cache,
                                              int32_t cache_dtype, const float* k_scale,
                                              const float* v_scale, int64_t num_pages,
                                              const int32_t* sparse_bt, const int32_t* sparse_ctx,
                                              int64_t T, int64_t H, int64_t G, int64_t D, int32_t K,
                                              float scale, void* out, void* workspace,
                                              size_t workspace_bytes, void* stream) {
    (void)workspace;
    (void)workspace_bytes;
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
    Q8Params A{};
    A.q = static_cast<const uint16_t*>(q);
    A.k = static_cast<const uint8_t*>(k_cache);
    A.v = static_cast<const uint8_t*>(v_cache);
    A.ks = k_scale;
    A.vs = v_scale;
    A.bt = sparse_bt;
    A.ctx = sparse_ctx;
    A.out = static_cast<uint16_t*>(out);
    A.num_pages = num_pages;
    A.H = (int32_t)H;
    A.G = (int32_t)G;
    A.width = K * kPagesPerBlock;
    A.scale = scale;
    A.status = current_status_word();
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool e4m3 = cache_dtype == BSA_DTYPE_E4M3;
    cudaError_t e;
    if (D == 64) e = launch_q8<64>(A, T * H, e4m3, st);
    else if (D == 128) e = launch_q8<128>(A, T * H, e4m3, st);
    else e = launch_q8<256>(A, T * H, e4m3, st);
    return e == cudaSuccess ? BSA_OK : (int)e;
}
