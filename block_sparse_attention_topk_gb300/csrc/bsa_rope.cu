// bsa_rope.cu -- rotary positions with one or several axes, forward and
// inverse (the inverse rotation is the gradient of the forward one).
//
// One CTA takes a few tokens and all their heads.  The tokens' (cos, sin)
// pairs are formed once in shared memory and serve every head; each thread
// then loads both halves of its pairs before it stores either, so the call
// may run in place.  The work is bound by memory: one read and one write of
// each element.
#include <cuda_runtime.h>
#include <stdint.h>

#include "bsa_internal.h"
#include "bsa_rope.cuh"

namespace bsa {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeTable = 2048;    // (cos, sin) entries per CTA: 16 KB

struct RopeArgs {
    RopeParams r;
    const void* x;
    void* out;
    int64_t xts, xhs, ots, ohs;
    int64_t T;
    int32_t H, D, tile;
};

__device__ __forceinline__ float widen(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ float widen(float f) { return f; }
__device__ __forceinline__ void narrow(float f, float& o) { o = f; }
__device__ __forceinline__ void narrow(float f, uint16_t& o) {
    o = __bfloat16_as_ushort(__float2bfloat16_rn(f));
}

template <typename E>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs A) {
    extern __shared__ __align__(16) float2 cs[];
    unsigned long long* steps = reinterpret_cast<unsigned long long*>(cs + A.tile * A.r.half);
    const int half = A.r.half;
    const int64_t t0 = (int64_t)blockIdx.x * A.tile;
    const int nt = (int)min((int64_t)A.tile, A.T - t0);
    for (int i = threadIdx.x; i < half; i += kRopeThreads) steps[i] = rope_step(__ldg(A.r.inv_freq + i));
    __syncthreads();
    for (int i = threadIdx.x; i < nt * half; i += kRopeThreads) {
        const int t = i / half, f = i - t * half;
        float2 c = rope_turn(__ldg(A.r.positions + rope_axis(A.r, f) * A.T + t0 + t), steps[f]);
        if (A.r.inverse) c.y = -c.y;
        cs[i] = c;
    }
    __syncthreads();
    const int units = A.D - half;      // pairs, then values that pass through
    const E* x = static_cast<const E*>(A.x);
    E* out = static_cast<E*>(A.out);
    for (int i = threadIdx.x; i < nt * A.H * units; i += kRopeThreads) {
        const int u = i % units, th = i / units;
        const int h = th % A.H, t = th / A.H;
        const E* xr = x + (t0 + t) * A.xts + h * A.xhs;
        E* orow = out + (t0 + t) * A.ots + h * A.ohs;
        if (u < half) {
            const int ia = A.r.interleaved ? 2 * u : u;
            const int ib = A.r.interleaved ? 2 * u + 1 : u + half;
            const float a = widen(xr[ia]), b = widen(xr[ib]);
            const float2 c = cs[t * half + u];
            narrow(a * c.x - b * c.y, orow[ia]);
            narrow(b * c.x + a * c.y, orow[ib]);
        } else {
            orow[u + half] = xr[u + half];
        }
    }
}

// Rows (t, h) of D elements at t * ts + h * hs do not overlap.
bool rows_apart(int64_t T, int64_t H, int64_t D, int64_t ts, int64_t hs) {
    if (ts < 0 || hs < 0) return false;
    if (T <= 1 && H <= 1) return true;
    if (T <= 1) return hs >= D;
    if (H <= 1) return ts >= D;
    if (ts >= hs) return hs >= D && ts >= (H - 1) * hs + D;
    return ts >= D && hs >= (T - 1) * ts + D;
}

}  // namespace
}  // namespace bsa

using namespace bsa;

extern "C" int bsa_rope(const void* x, int32_t dtype, int64_t T, int64_t H, int64_t D,
                        int64_t token_stride, int64_t head_stride, const int32_t* positions,
                        int32_t axes, const float* inv_freq, const int32_t* freq_axis,
                        int32_t rot_dim, int32_t flags, void* out, int64_t out_token_stride,
                        int64_t out_head_stride, void* stream) {
    if (dtype != BSA_DTYPE_BF16 && dtype != BSA_DTYPE_FP32) return BSA_ERR_DTYPE;
    if (T < 0 || T > INT32_MAX || H < 0 || H > 65536 || D < 1 || D > BSA_MAX_ROPE_DIM ||
        token_stride < 0 || head_stride < 0)
        return BSA_ERR_SHAPE;
    const int rc = check_rope(D, positions, axes, inv_freq, freq_axis, rot_dim, flags, T > 0);
    if (rc != BSA_OK) return rc;
    if (!rows_apart(T, H, D, out_token_stride, out_head_stride)) return BSA_ERR_SHAPE;
    if (T == 0 || H == 0) return BSA_OK;
    if (x == nullptr || out == nullptr) return BSA_ERR_NULL;
    const uintptr_t size = dtype == BSA_DTYPE_BF16 ? 2 : 4;
    if (reinterpret_cast<uintptr_t>(x) % size != 0 || reinterpret_cast<uintptr_t>(out) % size != 0)
        return BSA_ERR_ALIGN;
    if (x == out && ((T > 1 && token_stride != out_token_stride) || (H > 1 && head_stride != out_head_stride)))
        return BSA_ERR_SHAPE;
    RopeArgs A{};
    A.r = RopeParams{positions, T, inv_freq, freq_axis, axes, rot_dim / 2,
                     (flags & BSA_ROPE_INTERLEAVED) != 0, (flags & BSA_ROPE_INVERSE) != 0};
    A.x = x;
    A.out = out;
    A.xts = token_stride;
    A.xhs = head_stride;
    A.ots = out_token_stride;
    A.ohs = out_head_stride;
    A.T = T;
    A.H = (int32_t)H;
    A.D = (int32_t)D;
    int tile = rot_dim > 0 ? kRopeTable / (rot_dim / 2) : 16;
    if (tile > 16) tile = 16;
    A.tile = tile;
    const size_t smem = (size_t)tile * A.r.half * sizeof(float2) + A.r.half * sizeof(unsigned long long);
    const unsigned grid = (unsigned)((T + tile - 1) / tile);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == BSA_DTYPE_BF16) rope_kernel<uint16_t><<<grid, kRopeThreads, smem, st>>>(A);
    else rope_kernel<float><<<grid, kRopeThreads, smem, st>>>(A);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? BSA_OK : (int)e;
}
