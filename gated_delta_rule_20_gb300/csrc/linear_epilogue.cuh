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
    int act;       // gdn_activation, or kGeluF32
    bool out_f32;  // else bf16
    bool gated;
    bool nk;       // weight layout
};

// How a product is done (linear_tc.cu): on the tensor cores as it lies, from copies of operands that TMA cannot
// take, from bf16 parts of fp32 operands, or by the FFMA kernel; and the scratch that this takes.
enum class LinearRoute { kTensor, kCopies, kParts, kFfma };
struct LinearPlan {
    LinearRoute route;
    size_t scratch;
};
LinearPlan plan_linear(const LinearArgs& a, int32_t dtype);
// The tensor-core kernel of such a product, its token tile and its splits of K on a device of `sms` SMs.
void linear_tc_tiles(const LinearArgs& a, int32_t dtype, LinearRoute route, int sms, gdn_linear_plan_info* info);

// What fp32 operands by parts are found to be on the device: of `count` blocks, the exponents (biased, as in the number's
// bits; 255 for infinities and NaN, 0 where all is zero) of the largest elements that they met of x, and behind those of
// the weight.  Where parts_fit says no the product by parts does nothing, and the FFMA kernel behind it does it all (else
// that one does nothing).
struct LinearMarks {
    const uint8_t* tops;
    int count;
};

// Whether products of K by parts give what fp32 sums give, for operands under 2^(ex - 126) and 2^(ew - 126):
//   - infinities and NaN do not add up from parts; the largest numbers (ex = 254) round up to an infinite first part;
//   - no sum of the parts' products may pass the range: an infinity of one accumulator could meet another's of the
//     opposite sign.  Every accumulator stays under K 2^(ex + ew - 252), which is held to 2^127;
//   - the least bf16 number, 2^-133, is below 2^-24 of an operand's largest elements by a factor of 2^-8 (ex >= 27), and
//     the largest products are far enough above the least normal number (2^-100; ex + ew >= 154).
__device__ __forceinline__ bool parts_fit(int ex, int ew, int K) {
    const int log_k = 32 - __clz(K - 1);  // (rounded up; 0 for K = 1)
    if (max(ex, ew) >= 254) return false;
    if (min(ex, ew) == 0) return true;  // zeros
    return min(ex, ew) >= 27 && ex + ew >= 154 && ex + ew <= 379 - log_k;
}

// The same from the blocks' tops, for all threads of a CTA of kThreads (room: a word a warp in shared memory).
template <int kThreads>
__device__ __forceinline__ bool parts_fit_all(const uint8_t* tops, int count, int K, uint32_t* room) {
    const uint32_t* words = reinterpret_cast<const uint32_t*>(tops);  // (count is a multiple of 4)
    uint32_t x = 0, w = 0;
    for (int i = threadIdx.x; i < count / 4; i += kThreads) {
        x = __vmaxu4(x, words[i]);
        w = __vmaxu4(w, words[count / 4 + i]);
    }
    auto top = [](uint32_t v) {
        v = __vmaxu4(v, v >> 16);
        return __reduce_max_sync(0xffffffffu, max(v & 0xffu, (v >> 8) & 0xffu));
    };
    const uint32_t ex = top(x), ew = top(w);
    if ((threadIdx.x & 31) == 0) room[threadIdx.x >> 5] = ex | ew << 16;
    __syncthreads();
    uint32_t both = 0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) both = __vmaxu2(both, room[i]);
    return parts_fit((int)(both & 0xffffu), (int)(both >> 16), K);
}

// Enqueues every route but kFfma; marks are set for kParts.
gdn_status launch_linear_tc(const LinearArgs& a, int32_t dtype, LinearRoute route, void* scratch, int dev, int sms,
                            cudaStream_t s, LinearMarks* marks);

// The kernel for few rows on the FMA units (linear_few.cu), for every type, layout, size and alignment.
cudaError_t launch_linear_few(const LinearArgs& a, int32_t dtype, int sms, cudaStream_t s);

// gelu(v) = v Phi(v) for bf16 outputs: Phi(-|v|) = erfc(|v| / sqrt 2) / 2 by the rational approximation 7.1.26 of
// Abramowitz and Stegun's Handbook (Hastings): erfc(z) = (a1 s + ... + a5 s^5) e^(-z^2), s = 1 / (1 + 0.3275911 z), off by
// at most 1.5e-7, so gelu by 0.75e-7 |v|: of the value 5e-5 at v = -3 and 1.6e-3 at -5, where half a step of bf16 is
// 2e-3 to 4e-3.  Half the instructions of erff: M = 16384, K = 512, N = 4096 with GELU takes 96 us, and 122 with erff
// (without an activation 55).
__device__ __forceinline__ float gelu(float v) {
    const float z = fabsf(v) * 0.70710678118654752f;
    const float s = __fdividef(1.f, fmaf(0.3275911f, z, 1.f));
    float p = fmaf(1.061405429f, s, -1.453152027f);
    p = fmaf(p, s, 1.421413741f);
    p = fmaf(p, s, -0.284496736f);
    p = fmaf(p, s, 0.254829592f);
    const float q = 0.5f * p * s * __expf(-z * z);  // Phi(-|v|)
    return v * (v > 0.f ? 1.f - q : q);  // (+infinity stays)
}

// gelu for fp32 outputs, with the relative error of fp32 down to its smallest values: Phi(-a) e^(a^2 / 2) = s (c0 + c1 s
// + ... + c7 s^7), s = 1 / (1 + 0.31 a), a least-maximum fit of the relative error over a = 0 .. 15 (1.6e-7; with the
// roundings 1e-6 of gelu for v > -5 and 4e-6 at -12).  (erfcf instead spills registers in linear_large_kernel.)  M = 16384,
// K = 512, N = 4096 with fp32 output 140 us, 125 by the formula above.
constexpr int kGeluF32 = 16;
__device__ __forceinline__ float gelu_f32(float v) {
    const float s = __fdividef(1.f, fmaf(0.31f, fabsf(v), 1.f));
    float p = fmaf(0.035890512f, s, -0.14181866f);
    p = fmaf(p, s, 0.15545815f);
    p = fmaf(p, s, -0.015285325f);
    p = fmaf(p, s, 0.11032595f);
    p = fmaf(p, s, 0.10770097f);
    p = fmaf(p, s, 0.12407242f);
    p = fmaf(p, s, 0.12365606f);
    const float q = p * s * __expf(-0.5f * v * v);  // Phi(-|v|)
    return v * (v > 0.f ? 1.f - q : q);
}

__device__ __forceinline__ float activate(int act, float v) {
    switch (act) {  // uniform over the grid
        case GDN_ACT_SILU: return silu_fast(v);
        case GDN_ACT_GELU: return gelu(v);
        case kGeluF32: return gelu_f32(v);
        case GDN_ACT_RELU: return v < 0.f ? 0.f : v;  // NaN stays NaN
        default: return v;
    }
}

// The activation of C values (the choice is uniform over the grid).  kBf16: of a kernel for bf16 outputs only.
template <int C, bool kBf16 = false>
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
        case kGeluF32:
            if constexpr (!kBf16) {
#pragma unroll
                for (int j = 0; j < C; ++j) v[j] = activate(kGeluF32, v[j]);
            }
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
