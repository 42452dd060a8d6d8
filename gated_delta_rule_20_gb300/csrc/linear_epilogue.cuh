// linear_epilogue.cuh -- the arguments of a linear call on the device and its epilogue,
// shared by the FFMA and the tensor-core kernels: scales, bias, activation, gate,
// residual and the one rounding of the output.  All of it in fp32.
#pragma once

#include <cuda_bf16.h>

#include "gdn_device.cuh"
#include "gdn_internal.h"

namespace gdn {

struct LinearArgs {
    const void* x;
    const float* x_scale;  // null unless e4m3
    const void* w;
    const float* w_scale;  // null unless e4m3
    const float* bias;     // may be null
    const void* res;       // may be null; may be out
    void* out;
    int M, N, K;
    int act;       // gdn_activation
    bool out_f32;  // else bf16
    bool gated;
    bool nk;       // weight layout
};

// The tensor-core kernels (linear_tc.cu).  *taken: whether they do the call (they do not for fp32, nor for
// small products of operands that TMA cannot take).
gdn_status launch_linear_tc(const LinearArgs& a, int32_t dtype, int dev, int sms, cudaStream_t s, bool* taken);

__device__ __forceinline__ float activate(int act, float v) {
    switch (act) {  // uniform over the grid
        case GDN_ACT_SILU: return silu_fast(v);
        case GDN_ACT_GELU: return 0.5f * v * (1.f + erff(v * 0.70710678118654752f));
        case GDN_ACT_RELU: return v < 0.f ? 0.f : v;  // NaN stays NaN
        default: return v;
    }
}

// The activation of C values (the choice is uniform over the grid).
template <int C>
__device__ __forceinline__ void activate_all(int act, float (&v)[C]) {
    switch (act) {
        case GDN_ACT_SILU:
#pragma unroll
            for (int j = 0; j < C; ++j) v[j] = activate(GDN_ACT_SILU, v[j]);
            break;
        case GDN_ACT_GELU:
#pragma unroll
            for (int j = 0; j < C; ++j) v[j] = activate(GDN_ACT_GELU, v[j]);
            break;
        case GDN_ACT_RELU:
#pragma unroll
            for (int j = 0; j < C; ++j) v[j] = activate(GDN_ACT_RELU, v[j]);
            break;
    }
}

__device__ __forceinline__ float load_out(const LinearArgs& a, long long i) {
    return a.out_f32 ? static_cast<const float*>(a.res)[i]
                     : __bfloat162float(static_cast<const __nv_bfloat16*>(a.res)[i]);
}
__device__ __forceinline__ void store_out(const LinearArgs& a, long long i, float v) {
    if (a.out_f32)
        static_cast<float*>(a.out)[i] = v;
    else
        static_cast<__nv_bfloat16*>(a.out)[i] = __float2bfloat16_rn(v);
}

// The scaled and biased sum of row m and weight column n (n < 2 N when gated).
__device__ __forceinline__ float affine(const LinearArgs& a, float acc, int m, int n) {
    if (a.x_scale) acc *= a.x_scale[m] * a.w_scale[n];
    return a.bias ? acc + a.bias[n] : acc;
}

}  // namespace gdn
