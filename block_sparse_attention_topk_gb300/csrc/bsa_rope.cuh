// bsa_rope.cuh -- the rotary rotation shared by bsa_rope and the cache append.
//
// Pair i of a row at position p turns by p * f_i radians.  The product is
// formed in turns as 64-bit fixed point: step_i = frac(f_i / 2 pi) * 2^64,
// rounded from 53 bits, and p * step_i mod 2^64 is the fraction of a turn,
// exact but for the step's own rounding (p * 2^-54 turns at most), at the cost of
// one integer product.  A 32-bit product p * f_i would be off by 0.06 rad at
// p = 10^6.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/bsa_topk.h"

namespace bsa {

struct RopeParams {
    const int32_t* positions;   // [axes, T], or null (the append's own positions)
    int64_t T;
    const float* inv_freq;      // [half]
    const int32_t* freq_axis;   // [half], or null
    int32_t axes, half;         // half = rot_dim / 2
    int32_t interleaved, inverse;
};

#ifdef __CUDACC__
__device__ __forceinline__ unsigned long long rope_step(float f) {
    double t = (double)f * 0.15915494309189533577;   // 1 / (2 pi)
    t -= floor(t);
    return (unsigned long long)(t * 18446744073709551616.0);
}

// (cos, sin) of p turns-steps.  The nearest quarter turn is taken off in fixed point,
// so that what is rounded to fp32's 24 bits is an eighth of a turn at most: the angle is
// off by pi 2^-28 (rounded as it is, up to half a turn, pi 2^-25).
__device__ __forceinline__ float2 rope_turn(int32_t p, unsigned long long step) {
    const unsigned long long phase = (unsigned long long)(long long)p * step;
    const uint32_t k = (uint32_t)((phase + (1ull << 61)) >> 62);
    float c, s;
    sincospif(__ll2float_rn((long long)(phase - ((unsigned long long)k << 62))) * 0x1p-63f, &s, &c);
    const float x = k & 1 ? s : c, y = k & 1 ? c : s;
    return make_float2(k == 1 || k == 2 ? -x : x, k >= 2 ? -y : y);
}

__device__ __forceinline__ int rope_axis(const RopeParams& R, int i) {
    if (R.freq_axis == nullptr) return 0;
    return min(max(__ldg(R.freq_axis + i), 0), R.axes - 1);
}

// ---- 16-byte groups ----------------------------------------------------------
// The kernels move heads as slots of two 16-byte groups of GE elements:
//  kSplit        the two sides of GE pairs (i, i + half), half a multiple of GE,
//  kInterleaved  neighbours, pairs (2i, 2i + 1), any half,
//  kSplitAny     neighbours, pairs (i, i + half), any half: an element's partner
//                lies elsewhere in the row and is loaded by itself.
enum RopeMode { kSplit = 0, kInterleaved = 1, kSplitAny = 2 };
inline RopeMode rope_mode(const RopeParams& R, int ge) {
    if (R.interleaved) return kInterleaved;
    return R.half % ge == 0 ? kSplit : kSplitAny;
}
// A row of the table in shared memory: its cosines, padded to 16 bytes, then
// its sines.
__host__ __device__ inline int rope_pad(int half) { return (half + 3) & ~3; }
__device__ __forceinline__ void widen16(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void widen16(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ uint4 narrow16(const float (&f)[8]) {
    return make_uint4(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7]));
}
__device__ __forceinline__ uint4 narrow16(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
// GE elements as they are loaded and stored: 16 bytes, or 8 bytes of bf16.
template <typename E, int GE>
struct Group {
    using V = uint4;
    __device__ __forceinline__ static void widen(const V& v, float (&f)[GE]) { widen16(v, f); }
    __device__ __forceinline__ static V narrow(const float (&f)[GE]) { return narrow16(f); }
};
template <>
struct Group<uint16_t, 4> {
    using V = uint2;
    __device__ __forceinline__ static void widen(const V& v, float (&f)[4]) {
        f[0] = __uint_as_float(v.x << 16);
        f[1] = __uint_as_float(v.x & 0xFFFF0000u);
        f[2] = __uint_as_float(v.y << 16);
        f[3] = __uint_as_float(v.y & 0xFFFF0000u);
    }
    __device__ __forceinline__ static V narrow(const float (&f)[4]) { return make_uint2(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3])); }
};

__device__ __forceinline__ float widen(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ float widen(float f) { return f; }

// The two sides of a pair after the turn, rounded the same way in every kernel
// (left to the compiler, the contraction of the products differs between them).
__device__ __forceinline__ float turn_first(float a, float b, float c, float s) {
    return fmaf(a, c, -__fmul_rn(b, s));
}
__device__ __forceinline__ float turn_second(float a, float b, float c, float s) {
    return fmaf(b, c, __fmul_rn(a, s));
}

// element offsets of slot k's two groups
template <RopeMode MODE, int GE>
__device__ __forceinline__ void slot_groups(int k, int half, int& o0, int& o1) {
    if (MODE == kSplit && GE * k < half) {
        o0 = GE * k;
        o1 = o0 + half;
    } else {
        o0 = 2 * GE * k;                      // kSplit: half / GE slots cover 2 half elements
        o1 = o0 + GE;
    }
}

// Rotates slot k of a head's row at `x` (its groups' values in a and b; x is
// read again only for partners outside the slot).  cs: the row's cosines, then
// its sines at cs + rope_pad(half).
template <RopeMode MODE, typename E, int GE>
__device__ __forceinline__ void slot_rotate(const E* x, int k, const float* cs, int half, float (&a)[GE],
                                            float (&b)[GE]) {
    const float* sn = cs + rope_pad(half);
    if constexpr (MODE != kSplitAny) {
        if (GE * k >= half) return;
        // an interleaved slot may end past the last pair
        const bool whole = MODE == kSplit || GE * k + GE <= half;
#pragma unroll
        for (int i = 0; i < GE; i += 4) {
            if (!whole && GE * k + i >= half) break;
            const float4 c = *reinterpret_cast<const float4*>(cs + GE * k + i);
            const float4 s = *reinterpret_cast<const float4*>(sn + GE * k + i);
            const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // pair i + j: the groups' elements i + j, or elements 2 (i + j) and the next
                // of the groups in a row
                const int e = 2 * (i + j);
                float& first = MODE == kSplit ? a[i + j] : (e < GE ? a[e % GE] : b[e % GE]);
                float& second = MODE == kSplit ? b[i + j] : (e < GE ? a[e % GE + 1] : b[e % GE + 1]);
                const float u = first, v = second;
                const bool turns = whole || GE * k + i + j < half;
                first = turns ? turn_first(u, v, cc[j], ss[j]) : u;
                second = turns ? turn_second(u, v, cc[j], ss[j]) : v;
            }
        }
    } else {
        const int d0 = 2 * GE * k;
        if (d0 >= 2 * half) return;
        // every load is issued, of the element itself where it has no partner
        float o[2 * GE];
#pragma unroll
        for (int i = 0; i < 2 * GE; ++i) {
            const int d = d0 + i;
            o[i] = widen(x[d < half ? d + half : (d < 2 * half ? d - half : d)]);
        }
#pragma unroll
        for (int i = 0; i < 2 * GE; ++i) {
            const int d = d0 + i;
            const bool first = d < half;
            const int p = min(first ? d : d - half, half - 1);
            const float c = cs[p], s = sn[p];
            float& f = i < GE ? a[i] : b[i - GE];
            const float y = first ? turn_first(f, o[i], c, s) : turn_second(o[i], f, c, s);
            if (d < 2 * half) f = y;
        }
    }
}
#endif

// Checks shared by the entry points: BSA_OK or an error code.
inline int check_rope(int64_t D, const int32_t* positions, int32_t axes, const float* inv_freq,
                      const int32_t* freq_axis, int32_t rot_dim, int32_t flags, bool need_positions) {
    if (rot_dim < 0 || rot_dim > D || rot_dim % 2 != 0) return BSA_ERR_SHAPE;
    if (axes < 1 || axes > BSA_MAX_ROPE_AXES) return BSA_ERR_SHAPE;
    if ((flags & ~(BSA_ROPE_INTERLEAVED | BSA_ROPE_INVERSE)) != 0) return BSA_ERR_SHAPE;
    if (rot_dim > 0) {
        if (inv_freq == nullptr || (positions == nullptr && need_positions)) return BSA_ERR_NULL;
        if (axes > 1 && (freq_axis == nullptr || positions == nullptr)) return BSA_ERR_NULL;
    }
    return BSA_OK;
}

}  // namespace bsa
