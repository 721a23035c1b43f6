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

// (cos, sin) of p turns-steps; the fraction of a turn as [-1, 1) half turns.
__device__ __forceinline__ float2 rope_turn(int32_t p, unsigned long long step) {
    const long long phase = (long long)((unsigned long long)(long long)p * step);
    float2 r;
    sincospif(__ll2float_rn(phase) * 0x1p-63f, &r.y, &r.x);
    return r;
}

__device__ __forceinline__ int rope_axis(const RopeParams& R, int i) {
    if (R.freq_axis == nullptr) return 0;
    return min(max(__ldg(R.freq_axis + i), 0), R.axes - 1);
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
