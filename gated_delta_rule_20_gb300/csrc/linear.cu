// linear.cu -- the matrix product with bias, activation and residual in its epilogue
// (gdn_linear): the entry point's checks, the choice of the kernel, and the FFMA kernel
//
//     out[m, n] = act(x_scale[m] w_scale[n] sum_k x[m, k] W[k, n] + bias[n]) + residual[m, n]
//
// (gated: act of the gate's column times the up column).  The FFMA kernel is right for every
// type, layout, size and alignment; it is the path of fp32 compute and of operands whose rows
// TMA cannot take (pointer or row pitch not a multiple of 16 bytes).
//
// FFMA kernel: 256 threads on a tile of 16 TM tokens x 16 TM columns, TM x TM sums a thread,
// K in steps of 16 through shared memory, the next step's elements in registers while this
// one's products run.  A gated tile's columns are 8 TM of the gate and the same 8 TM of the
// up half, so that a thread holds both factors of its outputs.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "gdn_internal.h"
#include "linear_epilogue.cuh"

namespace gdn {
namespace {

constexpr int kBK = 16;

template <typename T, int TM>
__global__ void __launch_bounds__(256) linear_ffma_kernel(const __grid_constant__ LinearArgs a) {
    constexpr int kTile = 16 * TM, kPitch = kTile + 4, kLoads = kTile * kBK / 256;
    __shared__ float xs[kBK][kPitch], wsm[kBK][kPitch];
    const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
    const int cols = a.gated ? kTile / 2 : kTile;  // output columns of the tile
    const long long m0 = (long long)blockIdx.y * kTile, n0 = (long long)blockIdx.x * cols;
    const long long wn = a.gated ? 2LL * a.N : a.N;  // weight columns
    const T* x = static_cast<const T*>(a.x);
    const T* w = static_cast<const T*>(a.w);
    // weight column of the tile's column c, or -1 past the edge
    auto column = [&](int c) -> long long {
        const long long n = n0 + (a.gated && c >= cols ? c - cols : c);
        return n < a.N ? (a.gated && c >= cols ? a.N + n : n) : -1;
    };
    float xr[kLoads], wr[kLoads];
    auto load = [&](int k0) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int k = k0 + tid % kBK;
            const long long m = m0 + tid / kBK + i * (256 / kBK);
            xr[i] = k < a.K && m < a.M ? to_f32(x[m * a.K + k]) : 0.f;
            if (a.nk) {
                const long long n = column(tid / kBK + i * (256 / kBK));
                wr[i] = k < a.K && n >= 0 ? to_f32(w[n * a.K + k]) : 0.f;
            } else {
                const int kk = k0 + (tid + i * 256) / kTile;
                const long long n = column((tid + i * 256) % kTile);
                wr[i] = kk < a.K && n >= 0 ? to_f32(w[kk * wn + n]) : 0.f;
            }
        }
    };
    float acc[TM][TM] = {};
    load(0);
    for (int k0 = 0; k0 < a.K; k0 += kBK) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            xs[tid % kBK][tid / kBK + i * (256 / kBK)] = xr[i];
            if (a.nk)
                wsm[tid % kBK][tid / kBK + i * (256 / kBK)] = wr[i];
            else
                wsm[(tid + i * 256) / kTile][(tid + i * 256) % kTile] = wr[i];
        }
        __syncthreads();
        if (k0 + kBK < a.K) load(k0 + kBK);
#pragma unroll
        for (int k = 0; k < kBK; ++k) {
            float u[TM], v[TM];
#pragma unroll
            for (int i = 0; i < TM; ++i) u[i] = xs[k][ty * TM + i];
            // the thread's columns: TM / 2 of the tile's first half and the same of its second
#pragma unroll
            for (int j = 0; j < TM; ++j) v[j] = wsm[k][(j >= TM / 2 ? kTile / 2 - TM / 2 : 0) + tx * (TM / 2) + j];
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TM; ++j) acc[i][j] = fmaf(u[i], v[j], acc[i][j]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const long long m = m0 + ty * TM + i;
        if (m >= a.M) continue;
#pragma unroll
        for (int j = 0; j < TM; ++j) {
            if (a.gated && j >= TM / 2) continue;
            const long long n = n0 + (j >= TM / 2 ? kTile / 2 - TM / 2 : 0) + tx * (TM / 2) + j;
            if (n >= a.N) continue;
            float v = activate(a.act, affine(a, acc[i][j], (int)m, (int)n));
            if (a.gated) v *= affine(a, acc[i][(j + TM / 2) % TM], (int)m, (int)(a.N + n));
            const long long at = m * a.N + n;
            store_out(a, at, a.res ? v + load_out(a, at) : v);
        }
    }
}

template <typename T>
cudaError_t launch_ffma(const LinearArgs& a, cudaStream_t s) {
    // Small problems take the 64-wide tile, so that there are more blocks than SMs.
    const long long wn = a.gated ? 2LL * a.N : a.N;
    const bool large = ((a.M + 127LL) / 128) * ((wn + 127) / 128) >= 152;
    const int tile = large ? 128 : 64, cols = a.gated ? tile / 2 : tile;
    const dim3 grid((unsigned)((a.N + (long long)cols - 1) / cols), (unsigned)((a.M + (long long)tile - 1) / tile));
    if (large)
        linear_ffma_kernel<T, 8><<<grid, 256, 0, s>>>(a);
    else
        linear_ffma_kernel<T, 4><<<grid, 256, 0, s>>>(a);
    return cudaGetLastError();
}

gdn_status check_linear(const void* x, const float* x_scale, const void* w, const float* w_scale, const float* bias,
                        const void* res, const void* out, const gdn_linear_dims* d) {
    if (!d) return GDN_ERR_NULL;
    const bool f8 = d->dtype == GDN_F8E4M3, f32 = d->dtype == GDN_F32;
    if (!f8 && !f32 && d->dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
    if (d->out_dtype != GDN_F32 && (d->out_dtype != GDN_BF16 || f32)) return GDN_ERR_UNSUPPORTED;
    if (d->activation < GDN_ACT_NONE || d->activation > GDN_ACT_RELU) return GDN_ERR_UNSUPPORTED;
    if (d->flags & ~(uint32_t)(GDN_LINEAR_WEIGHT_NK | GDN_LINEAR_GATED | GDN_LINEAR_FORCE_FFMA))
        return GDN_ERR_UNSUPPORTED;
    if (f8 && !(d->flags & GDN_LINEAR_WEIGHT_NK)) return GDN_ERR_UNSUPPORTED;
    if (d->M < 0 || d->N < 1 || d->K < 1) return GDN_ERR_DIMS;
    const long long lim = INT32_MAX - 256;  // tile origins are 32-bit in the kernels
    if (d->M > 64LL * 65535 || d->N > lim || d->K > lim || ((d->flags & GDN_LINEAR_GATED) && d->N > lim / 2))
        return GDN_ERR_DIMS;  // (the FFMA kernel's grid has at most 65535 tiles of 64 tokens)
    if (d->M == 0) return GDN_OK;
    if (!x || !w || !out || (f8 && (!x_scale || !w_scale))) return GDN_ERR_NULL;
    if (!f8 && (x_scale || w_scale)) return GDN_ERR_UNSUPPORTED;
    auto off = [](const void* p, uintptr_t size) { return (reinterpret_cast<uintptr_t>(p) & (size - 1)) != 0; };
    const uintptr_t e = f8 ? 1 : f32 ? 4 : 2, o = d->out_dtype == GDN_F32 ? 4 : 2;
    if (off(x, e) || off(w, e) || off(res, o) || off(out, o) || off(x_scale, 4) || off(w_scale, 4) || off(bias, 4))
        return GDN_ERR_ALIGN;
    return GDN_OK;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" gdn_status gdn_linear(const void* x, const float* x_scale, const void* weight, const float* weight_scale,
                                 const float* bias, const void* residual, void* out, const gdn_linear_dims* d,
                                 gdn_stream_t stream) {
    const gdn_status st = check_linear(x, x_scale, weight, weight_scale, bias, residual, out, d);
    if (st != GDN_OK || d->M == 0) return st;
    const LinearArgs a{x, x_scale, weight, weight_scale, bias, residual, out, (int)d->M, (int)d->N, (int)d->K,
                       d->activation, d->out_dtype == GDN_F32, (d->flags & GDN_LINEAR_GATED) != 0,
                       (d->flags & GDN_LINEAR_WEIGHT_NK) != 0};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (!(d->flags & GDN_LINEAR_FORCE_FFMA) && linear_tc_supported(a, d->dtype)) return launch_linear_tc(a, d->dtype, s);
    const cudaError_t e = d->dtype == GDN_F32    ? launch_ffma<float>(a, s)
                          : d->dtype == GDN_BF16 ? launch_ffma<__nv_bfloat16>(a, s)
                                                 : launch_ffma<__nv_fp8_e4m3>(a, s);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
