// bsa_rope.cu -- rotary positions with one or several axes, forward and
// inverse (the inverse rotation is the gradient of the forward one).
//
// One CTA takes a few tokens and all their heads.  The tokens' cosines and
// sines are formed once in shared memory and serve every head.  The work is
// bound by memory: one read and one write of each element.
//  rope_slots_kernel   16-byte loads and stores (rows and strides aligned to
//                      16 bytes, D a multiple of two groups), or 8-byte ones of
//                      bf16 where rows or half-split partners are only that
//                      aligned; not in place where a partner may belong to
//                      another thread (kSplitAny).  Many small CTAs
//                      hide the loads: ten of 128 threads per SM with a slot
//                      each in flight take 68 us where four of 256 with two
//                      slots take 73 and two with four slots 85 (24 heads of
//                      128, 32760 tokens, bf16: 5.9 TB/s),
//  rope_kernel         pair by pair: any alignment, in place.
#include <cuda_runtime.h>
#include <stdint.h>

#include "bsa_internal.h"
#include "bsa_overlap.h"
#include "bsa_rope.cuh"

namespace bsa {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeTable = 4096;    // cosines or sines per CTA at most (32 KB both)
constexpr int kRopeTile = 4;        // tokens per CTA, more when they are short
constexpr int kRopeSlots = 512;     // slots per CTA that are enough
constexpr int kRopeCtas = 10;       // per SM

struct RopeArgs {
    RopeParams r;
    const void* x;
    void* out;
    int64_t xts, xhs, ots, ohs;
    int64_t T;
    int32_t H, D, tile;
};

__device__ __forceinline__ void narrow(float f, float& o) { o = f; }
__device__ __forceinline__ void narrow(float f, uint16_t& o) {
    o = __bfloat16_as_ushort(__float2bfloat16_rn(f));
}

// The tile's table (a row's cosines, then its sines).
__device__ __forceinline__ void rope_table(const RopeArgs& A, int64_t t0, int nt, float* cs,
                                           unsigned long long* steps) {
    const int half = A.r.half, pad = rope_pad(half);
    for (int i = threadIdx.x; i < half; i += kRopeThreads) steps[i] = rope_step(__ldg(A.r.inv_freq + i));
    __syncthreads();
    for (int i = threadIdx.x; i < nt * half; i += kRopeThreads) {
        const int t = i / half, f = i - t * half;
        const float2 c = rope_turn(__ldg(A.r.positions + rope_axis(A.r, f) * A.T + t0 + t), steps[f]);
        cs[t * 2 * pad + f] = c.x;
        cs[t * 2 * pad + pad + f] = A.r.inverse ? -c.y : c.y;
    }
    __syncthreads();
}

template <RopeMode MODE, typename E, int GE>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) rope_slots_kernel(const RopeArgs A) {
    using G = Group<E, GE>;
    using V = typename G::V;
    extern __shared__ __align__(16) unsigned char smem[];
    float* cs = reinterpret_cast<float*>(smem);
    const int half = A.r.half;
    const int64_t t0 = (int64_t)blockIdx.x * A.tile;
    const int nt = (int)min((int64_t)A.tile, A.T - t0);
    const E* x = static_cast<const E*>(A.x);
    E* out = static_cast<E*>(A.out);
    const int ks = A.D / (2 * GE);
    const int total = nt * A.H * ks;
    // (token, head, slot) of this thread, advanced by the CTA's width
    int k = threadIdx.x % ks, th = threadIdx.x / ks;
    int h = th % A.H, t = th / A.H;
    const int dk = kRopeThreads % ks, dth = kRopeThreads / ks;
    const int dh = dth % A.H, dt = dth / A.H;
    V a, b;
    auto load = [&]() {
        const E* xr = x + (t0 + t) * A.xts + h * A.xhs;
        int o0, o1;
        slot_groups<MODE, GE>(k, half, o0, o1);
        a = *reinterpret_cast<const V*>(xr + o0);
        b = *reinterpret_cast<const V*>(xr + o1);
    };
    // the first slot is on its way while the table is formed
    if ((int)threadIdx.x < total) load();
    rope_table(A, t0, nt, cs, reinterpret_cast<unsigned long long*>(cs + A.tile * 2 * rope_pad(half)));
    for (int i = threadIdx.x; i < total; i += kRopeThreads) {
        if (i != (int)threadIdx.x) load();
        const E* xr = x + (t0 + t) * A.xts + h * A.xhs;
        E* orow = out + (t0 + t) * A.ots + h * A.ohs;
        float fa[GE], fb[GE];
        G::widen(a, fa);
        G::widen(b, fb);
        slot_rotate<MODE>(xr, k, cs + t * 2 * rope_pad(half), half, fa, fb);
        int o0, o1;
        slot_groups<MODE, GE>(k, half, o0, o1);
        *reinterpret_cast<V*>(orow + o0) = G::narrow(fa);
        *reinterpret_cast<V*>(orow + o1) = G::narrow(fb);
        k += dk;
        h += dh;
        t += dt;
        if (k >= ks) {
            k -= ks;
            ++h;
        }
        if (h >= A.H) {
            h -= A.H;
            ++t;
        }
    }
}

template <typename E>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs A) {
    extern __shared__ __align__(16) unsigned char smem[];
    float* cs = reinterpret_cast<float*>(smem);
    const int half = A.r.half;
    const int64_t t0 = (int64_t)blockIdx.x * A.tile;
    const int nt = (int)min((int64_t)A.tile, A.T - t0);
    rope_table(A, t0, nt, cs, reinterpret_cast<unsigned long long*>(cs + A.tile * 2 * rope_pad(half)));
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
            const float c = cs[t * 2 * rope_pad(half) + u], s = cs[(t * 2 + 1) * rope_pad(half) + u];
            narrow(turn_first(a, b, c, s), orow[ia]);
            narrow(turn_second(a, b, c, s), orow[ib]);
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

template <typename E>
void launch_rope(const RopeArgs& A, cudaStream_t st) {
    constexpr int GE = 16 / (int)sizeof(E);
    const int half = A.r.half;
    const size_t smem = (size_t)A.tile * 2 * rope_pad(half) * sizeof(float) + half * sizeof(unsigned long long);
    const unsigned grid = (unsigned)((A.T + A.tile - 1) / A.tile);
    // the rows lie at multiples of ge elements, and are whole slots of them
    auto rows_of = [&](int ge) {
        return A.D % (2 * ge) == 0 && ((A.xts | A.xhs | A.ots | A.ohs) % ge) == 0 &&
               ((reinterpret_cast<uintptr_t>(A.x) | reinterpret_cast<uintptr_t>(A.out)) & (ge * sizeof(E) - 1)) == 0;
    };
    const bool wide = rows_of(GE);
    const RopeMode mode = rope_mode(A.r, GE);
    if (wide && mode == kSplit) {
        rope_slots_kernel<kSplit, E, GE><<<grid, kRopeThreads, smem, st>>>(A);
        return;
    }
    if (wide && mode == kInterleaved) {
        rope_slots_kernel<kInterleaved, E, GE><<<grid, kRopeThreads, smem, st>>>(A);
        return;
    }
    // Groups of 8 bytes: 24 heads of 72, 19112 tokens, take 36 us half-split and 32
    // interleaved, 79 pair by pair; 24 heads of 128 with 104 rotated half-split,
    // 32760 tokens, 86 where single partners (kSplitAny) take 123.
    if constexpr (GE == 8) {
        const RopeMode narrow_mode = rope_mode(A.r, 4);
        if (rows_of(4) && narrow_mode != kSplitAny) {
            if (narrow_mode == kSplit) rope_slots_kernel<kSplit, E, 4><<<grid, kRopeThreads, smem, st>>>(A);
            else rope_slots_kernel<kInterleaved, E, 4><<<grid, kRopeThreads, smem, st>>>(A);
            return;
        }
    }
    if (wide && A.x != A.out)
        rope_slots_kernel<kSplitAny, E, GE><<<grid, kRopeThreads, smem, st>>>(A);
    else
        rope_kernel<E><<<grid, kRopeThreads, smem, st>>>(A);
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
    const bool same = x == out && (T == 1 || token_stride == out_token_stride) && (H == 1 || head_stride == out_head_stride);
    const int64_t row = D * (int64_t)size, es = (int64_t)size;
    if (!same && rows_overlap(Rows{x, T, H, row, token_stride * es, head_stride * es},
                              Rows{out, T, H, row, out_token_stride * es, out_head_stride * es}))
        return BSA_ERR_SHAPE;
    RopeArgs A{};
    A.r = RopeParams{positions, T, inv_freq, freq_axis, axes, rot_dim / 2,
                     (flags & BSA_ROPE_INTERLEAVED) != 0, (flags & BSA_ROPE_INVERSE) != 0};
    A.x = x;
    A.out = out;
    // strides of dimensions of one entry never matter
    A.xts = T > 1 ? token_stride : 0;
    A.xhs = H > 1 ? head_stride : 0;
    A.ots = T > 1 ? out_token_stride : 0;
    A.ohs = H > 1 ? out_head_stride : 0;
    A.T = T;
    A.H = (int32_t)H;
    A.D = (int32_t)D;
    // tokens per CTA: four, or as many as fill its threads four times over (one
    // 32-wide head a token: 80146 tokens take 24 us in CTAs of four tokens), within the table
    const int64_t row_bytes = H * D * (int64_t)size;
    int64_t tile = kRopeSlots * 32 / row_bytes;
    if (tile < kRopeTile) tile = kRopeTile;
    if (rot_dim > 0 && tile > kRopeTable / (rot_dim / 2)) tile = kRopeTable / (rot_dim / 2);
    if (tile > 256) tile = 256;
    const int64_t want = 4 * (int64_t)device_sm_count();
    while (tile > 1 && (T + tile - 1) / tile < want) tile /= 2;
    A.tile = (int)tile;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == BSA_DTYPE_BF16) launch_rope<uint16_t>(A, st);
    else launch_rope<float>(A, st);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? BSA_OK : (int)e;
}
