// linear_few.cu -- gdn_linear for few rows on the FMA units: the weight is read once at the rate of
// memory and everything else is kept short.
//
// A thread loads 16-byte pieces of the weight, four ahead of the four that it works on, and has R rows'
// sums in registers.  [K, N'] weights: 8 lanes lie on 128 bytes of a row, the CTA's 32 groups of lanes on
// 32 rows; their sums meet by shuffles and in shared memory.  [N', K] weights: a warp has four columns and
// its 32 lanes lie along K; their sums meet by shuffles.  x is in shared memory in fp32, 1024 of K at a
// time.  K is split over a cluster of up to 8 CTAs until there are about two CTAs an SM; the sums are
// added in the ranks' order.  Rows that 16 bytes do not divide are read by elements, lanes side by side.
//
// Bound by the weight's bytes at one to four rows (16 MB and more: 4.7 TB/s), by its loads' latency below.  fp32, in
// a graph over weights larger than L2, this and the tiled FFMA kernel, us: M = 1, K = N = 2048 6.2 and 18.4, [N, K]
// 5.6 and 22.8; M = 1, K = 2048, N = 8192 14.4 and 64; M = 4 17.4 and 64, M = 8 25 and 64 (every 4 rows read the
// weight again, from L2).  Groups of 8 rows were slower (M = 8: 36): half the warps fit.  16 lanes on a row 13.5 at
// N = 8192, but 19.2 against 14.5 at K = 8192, N = 2048, where there are too few column tiles.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "gdn_internal.h"
#include "linear_epilogue.cuh"
#include "sm100_ptx.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256, kChunk = 1024, kAtOnce = 4;     // threads; K of x in shared memory; pieces of a step
constexpr int kLanes = 8, kSlots = kThreads / kLanes;         // [K, N']: lanes on a row; rows at once

__device__ __forceinline__ void put4(float* to, const float* from) {
    const float4 p = *reinterpret_cast<const float4*>(from);
    to[0] = p.x, to[1] = p.y, to[2] = p.z, to[3] = p.w;
}

// R: rows of the CTA, 1 or 4.
template <typename T, int R, bool kNK, bool kVec>
__global__ void __launch_bounds__(kThreads) linear_few_kernel(const __grid_constant__ LinearArgs a, int splits) {
    constexpr int V = 16 / (int)sizeof(T);            // elements of a piece
    constexpr int kCols = kNK ? 32 : kLanes * V;      // weight columns of the CTA
    constexpr int kStep = kNK ? 32 * V : kSlots * kAtOnce;  // K of a step
    constexpr int kSums = kNK ? kAtOnce : V;          // sums of a row that a thread has
    __shared__ __align__(16) float xs[R * kChunk];    // [K, N']: [k][R]; [N', K]: [R][k]
    __shared__ float part[kNK ? 1 : 8][R][kCols];
    __shared__ float sums[R][kCols];
    struct __align__(16) Piece {
        T e[V];
    };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = splits > 1 ? (int)ptx::cluster_rank() : 0;
    const int cols = a.gated ? kCols / 2 : kCols;  // output columns
    const long long n0 = (long long)(blockIdx.x / splits) * cols;
    const int m0 = (int)blockIdx.y * R;
    const long long wn = a.gated ? 2LL * a.N : a.N;
    const T* x = static_cast<const T*>(a.x);
    const T* w = static_cast<const T*>(a.w);
    const long long steps = ((long long)a.K + kStep - 1) / kStep;
    const long long k_lo = steps * rank / splits * kStep, k_hi = min((long long)a.K, steps * (rank + 1) / splits * kStep);
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();

    // [K, N']: this thread's piece is of columns `col[j]` (kVec: col[0] and on), -1 past N; its rows k + slot + 32 i.
    // [N', K]: columns `col[i]`; its elements from k + lane V on (not kVec: k + lane + 32 j).
    const int slot = tid / kLanes, place = tid % kLanes;
    constexpr int kPlaces = kNK ? kAtOnce : kVec ? 1 : V;
    long long col[kPlaces];
#pragma unroll
    for (int j = 0; j < kPlaces; ++j) {
        int c = kNK ? warp * kAtOnce + j : kVec ? place * V : j * kLanes + place;  // column of the tile: gate columns first
        if (kNK && a.gated) c = j / 2 * cols + warp * 2 + j % 2;
        const bool second = a.gated && c >= cols;
        const long long n = n0 + (second ? c - cols : c);
        col[j] = n < a.N ? (second ? a.N + n : n) : -1;
    }
    auto load = [&](long long k0, Piece (&p)[kAtOnce]) {
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            p[i] = Piece{};
            if constexpr (!kNK) {
                const long long k = k0 + slot + kSlots * i;
                if (k >= k_hi) continue;
                const T* row = w + k * wn;
                if constexpr (kVec) {
                    if (col[0] >= 0) p[i] = *reinterpret_cast<const Piece*>(row + col[0]);
                } else {
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        if (col[j] >= 0) p[i].e[j] = row[col[j]];
                }
            } else if (col[i] >= 0) {
                const T* row = w + col[i] * a.K;
                if constexpr (kVec) {
                    const long long k = k0 + lane * V;
                    if (k < k_hi) p[i] = *reinterpret_cast<const Piece*>(row + k);
                } else {
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const long long k = k0 + lane + 32 * j;
                        if (k < k_hi) p[i].e[j] = row[k];
                    }
                }
            }
        }
    };

    float acc[R][kSums] = {};
    Piece now[kAtOnce], next[kAtOnce];
    load(k_lo, now);
    for (long long k0 = k_lo; k0 < k_hi; k0 += kStep) {
        const int in = (int)((k0 - k_lo) % kChunk);  // (steps divide the chunk)
        if (in == 0) {
            if (k0 > k_lo) __syncthreads();
            const int len = (int)min((long long)kChunk, (k_hi - k0 + kStep - 1) / kStep * kStep);  // with zeros past k_hi
#pragma unroll
            for (int r = 0; r < R; ++r)
                for (int k = tid; k < len; k += kThreads)
                    xs[kNK ? r * kChunk + k : k * R + r] =
                        m0 + r < a.M && k0 + k < k_hi ? to_f32(x[(long long)(m0 + r) * a.K + k0 + k]) : 0.f;
            __syncthreads();
        }
        load(k0 + kStep, next);
        if constexpr (!kNK) {
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                float u[R];
#pragma unroll
                for (int r = 0; r < R; r += 4) {
                    if constexpr (R > 1)
                        put4(u + r, xs + (in + slot + kSlots * i) * R + r);
                    else
                        u[r] = xs[in + slot + kSlots * i];
                }
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float v = to_f32(now[i].e[j]);
#pragma unroll
                    for (int r = 0; r < R; ++r) acc[r][j] = fmaf(u[r], v, acc[r][j]);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < V; j += 4) {
                float u[R][4];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float* xk = xs + r * kChunk + in;
                    if constexpr (kVec) {
                        put4(u[r], xk + lane * V + j);
                    } else {
#pragma unroll
                        for (int q = 0; q < 4; ++q) u[r][q] = xk[lane + 32 * (j + q)];
                    }
                }
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int i = 0; i < kAtOnce; ++i) {
                        const float v = to_f32(now[i].e[j + q]);
#pragma unroll
                        for (int r = 0; r < R; ++r) acc[r][i] = fmaf(u[r][q], v, acc[r][i]);
                    }
            }
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) now[i] = next[i];
    }

    // The CTA's sums.
    if constexpr (kNK) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                float v = acc[r][i];
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
                if (lane == 0) sums[r][a.gated ? i / 2 * cols + warp * 2 + i % 2 : warp * kAtOnce + i] = v;
            }
    } else {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float v = acc[r][j];
#pragma unroll
                for (int d = kLanes; d < 32; d <<= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
                if (lane < kLanes) part[warp][r][kVec ? place * V + j : j * kLanes + place] = v;
            }
        __syncthreads();
        for (int i = tid; i < R * kCols; i += kThreads) {
            float v = 0.f;
#pragma unroll
            for (int q = 0; q < 8; ++q) v += part[q][i / kCols][i % kCols];
            sums[i / kCols][i % kCols] = v;
        }
    }
    if (splits > 1)
        ptx::cluster_sync();
    else
        __syncthreads();
    // All ranks' sums, in their order, and the epilogue: an output a thread, of the rank's share.
    for (int i = rank * kThreads + tid; i < R * cols; i += splits * kThreads) {
        const int r = i / cols, c = i % cols, m = m0 + r;
        const long long n = n0 + c;
        if (m >= a.M || n >= a.N) continue;
        const uint32_t at = ptx::smem_u32(&sums[r][c]);
        float g[8], u[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            if (q >= splits) break;
            const uint32_t peer = splits > 1 ? ptx::map_to_rank(at, q) : at;
            g[q] = ptx::ld_cluster_f32(peer);
            if (a.gated) u[q] = ptx::ld_cluster_f32(peer + cols * 4);
        }
#pragma unroll
        for (int q = 1; q < 8; ++q) {
            if (q >= splits) break;
            g[0] += g[q];
            if (a.gated) u[0] += u[q];
        }
        float v = activate(a.act, affine(a, g[0], m, (int)n));
        if (a.gated) v *= affine(a, u[0], m, (int)(a.N + n));
        const long long o = (long long)m * a.N + n;
        store_out(a, o, a.res ? v + load_out(a, o) : v);
    }
    if (splits > 1) ptx::cluster_sync_relaxed();  // a CTA's shared memory stays until every rank has read it
}

template <typename T, int R, bool kNK, bool kVec>
cudaError_t launch(const LinearArgs& a, int sms, cudaStream_t s) {
    constexpr int V = 16 / (int)sizeof(T), kCols = kNK ? 32 : kLanes * V, kStep = kNK ? 32 * V : kSlots * kAtOnce;
    const int cols = a.gated ? kCols / 2 : kCols;
    const long long tiles = (a.N + (long long)cols - 1) / cols, rows = (a.M + R - 1) / R;
    int splits = 1;
    while (splits < 8 && tiles * rows * splits < 2LL * sms && (long long)kStep * splits * 2 <= a.K) splits *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(tiles * splits), (unsigned)rows);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)splits;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = splits > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, linear_few_kernel<T, R, kNK, kVec>, a, splits);
}

template <typename T, int R>
cudaError_t launch_layout(const LinearArgs& a, int sms, cudaStream_t s) {
    constexpr int V = 16 / (int)sizeof(T);
    const bool vec = (reinterpret_cast<uintptr_t>(a.w) & 15u) == 0 && (a.nk ? a.K : a.N) % V == 0;
    if constexpr (!std::is_same<T, __nv_fp8_e4m3>::value) {  // e4m3 weights are [N', K]
        if (!a.nk) return vec ? launch<T, R, false, true>(a, sms, s) : launch<T, R, false, false>(a, sms, s);
    }
    return vec ? launch<T, R, true, true>(a, sms, s) : launch<T, R, true, false>(a, sms, s);
}

template <typename T>
cudaError_t launch_rows(const LinearArgs& a, int sms, cudaStream_t s) {
    return a.M == 1 ? launch_layout<T, 1>(a, sms, s) : launch_layout<T, 4>(a, sms, s);
}

}  // namespace

cudaError_t launch_linear_few(const LinearArgs& a, int32_t dtype, int sms, cudaStream_t s) {
    return dtype == GDN_F32    ? launch_rows<float>(a, sms, s)
           : dtype == GDN_BF16 ? launch_rows<__nv_bfloat16>(a, sms, s)
                               : launch_rows<__nv_fp8_e4m3>(a, sms, s);
}

}  // namespace gdn
