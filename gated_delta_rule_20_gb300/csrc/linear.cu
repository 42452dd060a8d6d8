// linear.cu -- the matrix product with bias, activation and residual in its epilogue
// (gdn_linear): the entry point's checks, the choice of the kernel, and the FFMA kernel
//
//     out[m, n] = act(x_scale[m] w_scale[n] sum_k x[m, k] W[k, n] + bias[n]) + residual[m, n]
//
// (gated: act of the gate's column times the up column).  The FFMA kernel is right for every
// type, layout, size and alignment; it is the path of fp32 compute and of small products of operands
// whose rows TMA cannot take (pointer or row pitch not a multiple of 16 bytes).  Up to 12 rows linear_few.cu does
// the same.
//
// FFMA kernel: 16 x 16 threads on a tile of 16 TM tokens x 16 TM columns, TM x TM sums a thread as pairs
// of neighbouring columns (fma.rn.f32x2: half the issue slots of single FFMAs, which leaves room for the
// shared-memory loads).  K goes in steps of 16 through two buffers of shared memory: the next steps'
// elements are on their way to registers while this one's products run, and one barrier a step is
// enough.  Rows that 4-element pieces divide are loaded so (kVec), others element by element.  A gated
// tile's columns are 8 TM of the gate and the same 8 TM of the up half, so that a thread holds both
// factors of its outputs.  Small products take the 64-wide tile (TM = 4), load 4 steps ahead and split K
// over a cluster; the ranks' tiles meet in distributed shared memory and are added in the ranks' order.
// (64-wide tiles of two warps with 8 x 8 sums a thread do fewer loads a product, but wait on each of
// them: 102 against 70 us at M = N = K = 1024 in fp32.)
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

constexpr int kBK = 16;

// Four consecutive elements as fp32, in one load (kVec) or one by one where `count` of them exist.
template <typename T, bool kVec>
__device__ __forceinline__ void load4(const T* p, int count, float (&v)[4]) {
    if constexpr (kVec) {
        struct __align__(4 * sizeof(T)) Four {
            T e[4];
        };
        if (count > 0) {
            const Four f = *reinterpret_cast<const Four*>(p);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = to_f32(f.e[j]);
        } else {
            v[0] = v[1] = v[2] = v[3] = 0.f;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = j < count ? to_f32(p[j]) : 0.f;
    }
}

__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t p) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
    return r;
}
__device__ __forceinline__ void fma2(uint64_t& acc, uint64_t u, uint64_t v) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(u), "l"(v));
}

// kNK: the weight is [N', K]; splits: CTAs of the cluster, each with its part of K (TM = 4 only).
template <typename T, int TM, bool kNK, bool kVec>
__global__ void __launch_bounds__(256, 2) linear_ffma_kernel(const __grid_constant__ LinearArgs a, int splits,
                                                             const LinearMarks marks) {
    constexpr int SIDE = 16, kThreads = SIDE * SIDE, kTile = TM * SIDE, kPitch = kTile + 4;
    constexpr int kQuads = kTile * kBK / 4 / kThreads;       // 4-element loads a thread
    constexpr int kAhead = TM == 8 ? 1 : 4;                  // steps loaded ahead
    __shared__ __align__(16) float buf[2][2][kBK][kPitch];  // [turn][x, w]
    const int tid = threadIdx.x, tx = tid % SIDE, ty = tid / SIDE;
    const int cols = a.gated ? kTile / 2 : kTile;  // output columns of the tile
    const int rank = splits > 1 ? (int)ptx::cluster_rank() : 0;
    const long long m0 = (long long)blockIdx.y * kTile, n0 = (long long)(blockIdx.x / splits) * cols;
    const long long wn = a.gated ? 2LL * a.N : a.N;  // weight columns
    const T* x = static_cast<const T*>(a.x);
    const T* w = static_cast<const T*>(a.w);
    const int steps = (a.K + kBK - 1) / kBK;
    const int k_lo = (int)((long long)steps * rank / splits) * kBK;
    const int k_hi = rank + 1 == splits ? a.K : (int)((long long)steps * (rank + 1) / splits) * kBK;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    if (marks.tops) {  // only for operands that the tensor cores' parts do not fit (one answer for the whole grid)
        __shared__ uint32_t tops[kThreads / 32];
        if (parts_fit_all<kThreads>(marks.tops, marks.count, a.K, tops)) return;
    }
    // This thread's pieces: of x (and of a [N', K] weight) 4 elements of K of rows tid / 4 + i kThreads / 4, of a
    // [K, N'] weight 4 columns of one k.  Their addresses at k = 0, and how many elements of the piece's
    // own direction exist (columns: up to 4; rows: all or none).
    const int kq = tid % 4 * 4;
    const T *xp[kQuads], *wp[kQuads];
    bool x_in[kQuads];
    int w_in[kQuads];
#pragma unroll
    for (int i = 0; i < kQuads; ++i) {
        const long long m = m0 + tid / 4 + i * (kThreads / 4);
        x_in[i] = m < a.M;
        xp[i] = x + (x_in[i] ? m * a.K + kq : 0);
        const int c = kNK ? tid / 4 + i * (kThreads / 4) : (tid + i * kThreads) % (kTile / 4) * 4;  // column of the tile
        const bool second = a.gated && c >= cols;
        const long long n = n0 + (second ? c - cols : c), left = a.N - n, col = second ? a.N + n : n;
        w_in[i] = left >= 4 ? 4 : left > 0 ? (int)left : 0;
        wp[i] = w + (w_in[i] == 0 ? 0 : kNK ? col * a.K + kq : (long long)((tid + i * kThreads) / (kTile / 4)) * wn + col);
    }
    float xr[kAhead][kQuads][4], wr[kAhead][kQuads][4];
    auto load = [&](int k0, float (&xr)[kQuads][4], float (&wr)[kQuads][4]) {
        const int left = min(4, k_hi - k0 - kq);  // of this thread's 4 elements of K
#pragma unroll
        for (int i = 0; i < kQuads; ++i) {
            load4<T, kVec>(xp[i] + k0, x_in[i] ? left : 0, xr[i]);
            if constexpr (kNK)
                load4<T, kVec>(wp[i] + k0, w_in[i] > 0 ? left : 0, wr[i]);
            else
                load4<T, kVec>(wp[i] + k0 * wn, k0 + (tid + i * kThreads) / (kTile / 4) < k_hi ? w_in[i] : 0, wr[i]);
        }
    };
    auto store = [&](int turn, const float (&xr)[kQuads][4], const float (&wr)[kQuads][4]) {
#pragma unroll
        for (int i = 0; i < kQuads; ++i) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                buf[turn][0][tid % 4 * 4 + j][tid / 4 + i * (kThreads / 4)] = xr[i][j];
                if constexpr (kNK) buf[turn][1][tid % 4 * 4 + j][tid / 4 + i * (kThreads / 4)] = wr[i][j];
            }
            if constexpr (!kNK) {
                const int row = (tid + i * kThreads) / (kTile / 4), at = (tid + i * kThreads) % (kTile / 4) * 4;
                *reinterpret_cast<float4*>(&buf[turn][1][row][at]) = make_float4(wr[i][0], wr[i][1], wr[i][2], wr[i][3]);
            }
        }
    };
    // The thread's tokens: TM / 2 of the tile's first half and TM / 2 of its second; its columns likewise.
    constexpr int kHalf = TM / 2;
    auto place = [](int t, int i) { return (i >= kHalf ? kTile / 2 - kHalf : 0) + t * kHalf + i; };
    uint64_t acc[TM][kHalf] = {};
    // step i's elements wait in slot i % kAhead of the registers, and in buffer i % 2 of shared memory
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(k_lo + i * kBK, xr[i], wr[i]);
    store(0, xr[0], wr[0]);
    __syncthreads();
    auto step = [&](int k0, int turn, auto slot) {
        constexpr int kSlot = decltype(slot)::value, kNext = (kSlot + 1) % kAhead;
        if (k0 + kAhead * kBK < k_hi) load(k0 + kAhead * kBK, xr[kSlot], wr[kSlot]);
#pragma unroll
        for (int k = 0; k < kBK; ++k) {
            const float* xk = buf[turn][0][k];
            const float* wk = buf[turn][1][k];
            uint64_t v[kHalf];
            float u[TM];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if constexpr (TM == 8) {
                    const float4 p = *reinterpret_cast<const float4*>(xk + h * (kTile / 2) + ty * 4);
                    u[4 * h] = p.x, u[4 * h + 1] = p.y, u[4 * h + 2] = p.z, u[4 * h + 3] = p.w;
                    const float4 q = *reinterpret_cast<const float4*>(wk + h * (kTile / 2) + tx * 4);
                    v[2 * h] = pack2(q.x, q.y), v[2 * h + 1] = pack2(q.z, q.w);
                } else {
                    const float2 p = *reinterpret_cast<const float2*>(xk + h * (kTile / 2) + ty * 2);
                    u[2 * h] = p.x, u[2 * h + 1] = p.y;
                    const float2 q = *reinterpret_cast<const float2*>(wk + h * (kTile / 2) + tx * 2);
                    v[h] = pack2(q.x, q.y);
                }
            }
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const uint64_t uu = pack2(u[i], u[i]);
#pragma unroll
                for (int j = 0; j < kHalf; ++j) fma2(acc[i][j], uu, v[j]);
            }
        }
        if (k0 + kBK < k_hi) store(turn ^ 1, xr[kNext], wr[kNext]);
        __syncthreads();
    };
    for (int k0 = k_lo; k0 < k_hi;) {
        step(k0, 0, std::integral_constant<int, 0>());
        if ((k0 += kBK) >= k_hi) break;
        step(k0, 1, std::integral_constant<int, 1 % kAhead>());
        if ((k0 += kBK) >= k_hi) break;
        if constexpr (kAhead == 4) {
            step(k0, 0, std::integral_constant<int, 2 % kAhead>());
            if ((k0 += kBK) >= k_hi) break;
            step(k0, 1, std::integral_constant<int, 3 % kAhead>());
            k0 += kBK;
        }
    }
    // (column j of the thread: pair j / 2; pairs 0 .. kHalf / 2 - 1 lie in the tile's first half)
    if constexpr (TM == 4) {
        // The tile through shared memory, [token][column]: a thread then finishes 4 neighbouring columns, of
        // the tokens that its rank owns, over all ranks' sums.  (Outputs finished from the
        // registers are a copy of the epilogue each, whose code took 5 us to fetch, and 64 of them 20 us.)
        float* tile = &buf[0][0][0][0];
        static_assert(sizeof(buf) >= (size_t)kTile * kTile * sizeof(float), "the tile fits the buffers");
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                *reinterpret_cast<float2*>(tile + place(ty, i) * kTile + h * (kTile / 2) + tx * 2) = unpack2(acc[i][h]);
            }
        if (splits > 1)
            ptx::cluster_sync();
        else
            __syncthreads();
        const int width = cols / 4;  // threads of a token
        const long long n = n0 + tid % width * 4;
        const int there = (int)max(0LL, min(4LL, a.N - n));  // columns that exist
        const uint32_t at = ptx::smem_u32(tile) + tid % width * 16;
#pragma unroll 1
        for (int r = rank + splits * (tid / width); r < kTile; r += splits * (kThreads / width)) {
            const long long m = m0 + r;
            if (m >= a.M || there == 0) break;
            float4 g[8], u[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                if (q >= splits) break;
                const uint32_t peer = ptx::map_to_rank(at + r * kTile * 4, q);
                g[q] = ptx::ld_cluster_f32x4(peer);
                if (a.gated) u[q] = ptx::ld_cluster_f32x4(peer + kTile / 2 * 4);
            }
#pragma unroll
            for (int q = 1; q < 8; ++q) {  // the ranks' order
                if (q >= splits) break;
                g[0].x += g[q].x, g[0].y += g[q].y, g[0].z += g[q].z, g[0].w += g[q].w;
                if (a.gated) u[0].x += u[q].x, u[0].y += u[q].y, u[0].z += u[q].z, u[0].w += u[q].w;
            }
            float v[4] = {g[0].x, g[0].y, g[0].z, g[0].w};
            const float w4[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = affine(a, v[j], (int)m, (int)(n + min(j, there - 1)));
            activate_all<4>(a.act, v);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (j >= there) break;
                if (a.gated) v[j] *= affine(a, w4[j], (int)m, (int)(a.N + n + j));
                const long long o = m * a.N + n + j;
                store_out(a, o, a.res ? v[j] + load_out(a, o) : v[j]);
            }
        }
        if (splits > 1) ptx::cluster_sync_relaxed();  // a CTA's shared memory stays until every rank has read it
    } else {
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const long long m = m0 + place(ty, i);
            float v[TM];
#pragma unroll
            for (int j = 0; j < kHalf; ++j) {
                const float2 p = unpack2(acc[i][j]);
                v[2 * j] = p.x;
                v[2 * j + 1] = p.y;
            }
            if (m >= a.M) continue;
            const int outs = a.gated ? kHalf : TM;
#pragma unroll
            for (int j = 0; j < TM; ++j) {
                const long long n = n0 + (a.gated ? place(tx, j % kHalf) : place(tx, j));
                if (n < a.N) v[j] = affine(a, v[j], (int)m, (int)(a.gated && j >= kHalf ? a.N + n : n));
            }
            float f[TM];
#pragma unroll
            for (int j = 0; j < TM; ++j) f[j] = v[j];
            activate_all<TM>(a.act, f);
#pragma unroll
            for (int j = 0; j < TM; ++j) {
                const long long n = n0 + place(tx, j);
                if (j >= outs || n >= a.N) continue;
                const float y = a.gated ? f[j] * v[(j + kHalf) % TM] : f[j];
                const long long at = m * a.N + n;
                store_out(a, at, a.res ? y + load_out(a, at) : y);
            }
        }
    }
}

template <typename T, int TM, bool kNK, bool kVec>
cudaError_t launch_tile(const LinearArgs& a, int splits, const LinearMarks& marks, cudaStream_t s) {
    const int tile = 16 * TM, cols = a.gated ? tile / 2 : tile;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((a.N + (long long)cols - 1) / cols * splits),
                       (unsigned)((a.M + (long long)tile - 1) / tile));
    cfg.blockDim = dim3(256);
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
    return cudaLaunchKernelEx(&cfg, linear_ffma_kernel<T, TM, kNK, kVec>, a, splits, marks);
}

template <typename T, int TM>
cudaError_t launch_layout(const LinearArgs& a, int splits, const LinearMarks& marks, cudaStream_t s) {
    // pieces of 4 elements: rows that they divide, from an address that they divide
    auto four = [](const void* p) { return reinterpret_cast<uintptr_t>(p) % (4 * sizeof(T)) == 0; };
    const long long wn = a.gated ? 2LL * a.N : a.N;
    const bool vec = four(a.x) && four(a.w) && a.K % 4 == 0 && (a.nk || (wn % 4 == 0 && a.N % 4 == 0));
    if constexpr (!std::is_same<T, __nv_fp8_e4m3>::value) {  // e4m3 weights are [N', K]
        if (!a.nk)
            return vec ? launch_tile<T, TM, false, true>(a, splits, marks, s)
                       : launch_tile<T, TM, false, false>(a, splits, marks, s);
    }
    return vec ? launch_tile<T, TM, true, true>(a, splits, marks, s) : launch_tile<T, TM, true, false>(a, splits, marks, s);
}

// Few rows: a kernel that reads the weight once for every 4.  It and the tiles of launch_ffma, us: fp32 K = N = 2048 M = 12
// 13.9 and 18.8, M = 16 13.8 and 18.9 but K = 4097, N = 2001 51 and 38; e4m3 K = 4097, N = 2001 M = 8 50 and 50, M = 12
// 57 and 50.
bool few_rows(const LinearArgs& a, int32_t dtype) { return a.M <= (dtype == GDN_F8E4M3 ? 8 : 12); }

template <typename T>
cudaError_t launch_ffma(const LinearArgs& a, int32_t dtype, int sms, const LinearMarks& marks, cudaStream_t s) {
    if (few_rows(a, dtype) && !marks.tops) return launch_linear_few(a, dtype, sms, s);
    const long long wn = a.gated ? 2LL * a.N : a.N;
    auto tiles = [&](int t) { return ((a.M + (long long)t - 1) / t) * ((wn + t - 1) / t); };
    if (tiles(128) >= sms) return launch_layout<T, 8>(a, 1, marks, s);
    // Small products: 64-wide tiles, and K over as many CTAs as give two an SM (4 steps of K each at least).
    int splits = 1;
    while (splits < 8 && tiles(64) * splits * 2 <= 2LL * sms && a.K >= kBK * 4 * 2 * splits) splits *= 2;
    return launch_layout<T, 4>(a, splits, marks, s);
}

gdn_status check_dims(const gdn_linear_dims* d) {
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
    return GDN_OK;
}

gdn_status check_linear(const void* x, const float* x_scale, const void* w, const float* w_scale, const float* bias,
                        const void* res, const void* out, const gdn_linear_dims* d) {
    const gdn_status st = check_dims(d);
    if (st != GDN_OK || d->M == 0) return st;
    const bool f8 = d->dtype == GDN_F8E4M3, f32 = d->dtype == GDN_F32;
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

namespace {

LinearArgs args_of(const void* x, const float* x_scale, const void* weight, const float* weight_scale, const float* bias,
                   const void* residual, void* out, const gdn_linear_dims* d) {
    const bool f32 = d->out_dtype == GDN_F32;
    const int act = f32 && d->activation == GDN_ACT_GELU ? kGeluF32 : d->activation;
    return LinearArgs{x, x_scale, weight, weight_scale, bias, residual, out, (int)d->M, (int)d->N, (int)d->K, act, f32,
                      (d->flags & GDN_LINEAR_GATED) != 0, (d->flags & GDN_LINEAR_WEIGHT_NK) != 0};
}

LinearPlan plan_of(const LinearArgs& a, const gdn_linear_dims* d) {
    if (d->flags & GDN_LINEAR_FORCE_FFMA) return LinearPlan{LinearRoute::kFfma, 0};
    return plan_linear(a, d->dtype);
}

}  // namespace

extern "C" size_t gdn_linear_workspace_bytes(const void* x, const void* weight, const gdn_linear_dims* d) {
    if (check_dims(d) != GDN_OK || d->M == 0) return 0;
    return plan_of(args_of(x, nullptr, weight, nullptr, nullptr, nullptr, nullptr, d), d).scratch;
}

extern "C" gdn_status gdn_linear_plan(const void* x, const void* weight, const gdn_linear_dims* d, int32_t sm_count,
                                      gdn_linear_plan_info* info) {
    const gdn_status st = check_dims(d);
    if (st != GDN_OK) return st;
    if (!info) return GDN_ERR_NULL;
    if (sm_count < 1) return GDN_ERR_DIMS;
    *info = gdn_linear_plan_info{GDN_LINEAR_KERNEL_NONE, GDN_LINEAR_OPERANDS_AS_THEY_LIE, 0, 0};
    if (d->M == 0) return GDN_OK;
    const LinearArgs a = args_of(x, nullptr, weight, nullptr, nullptr, nullptr, nullptr, d);
    const LinearPlan how = plan_of(a, d);
    if (how.route == LinearRoute::kFfma) {
        info->kernel = few_rows(a, d->dtype) ? GDN_LINEAR_KERNEL_FEW : GDN_LINEAR_KERNEL_FFMA;
        return GDN_OK;
    }
    if (how.route == LinearRoute::kCopies) info->operands = GDN_LINEAR_OPERANDS_COPIED;
    if (how.route == LinearRoute::kParts) info->operands = GDN_LINEAR_OPERANDS_IN_PARTS;
    linear_tc_tiles(a, d->dtype, how.route, sm_count, info);
    return GDN_OK;
}

extern "C" gdn_status gdn_linear_ws(const void* x, const float* x_scale, const void* weight, const float* weight_scale,
                                    const float* bias, const void* residual, void* out, const gdn_linear_dims* d,
                                    void* workspace, size_t workspace_bytes, gdn_stream_t stream) {
    gdn_status st = check_linear(x, x_scale, weight, weight_scale, bias, residual, out, d);
    if (st != GDN_OK) return st;
    if (reinterpret_cast<uintptr_t>(workspace) & 15u) return GDN_ERR_ALIGN;
    if (d->M == 0) return GDN_OK;
    const LinearArgs a = args_of(x, x_scale, weight, weight_scale, bias, residual, out, d);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    LinearPlan how = plan_of(a, d);
    if (workspace && workspace_bytes < how.scratch) return GDN_ERR_WORKSPACE;
    // An output over an operand would be read after other rows and columns are written.
    const long long e = d->dtype == GDN_F32 ? 4 : d->dtype == GDN_BF16 ? 2 : 1, wn = a.gated ? 2 * d->N : d->N;
    const long long out_bytes = d->M * d->N * (a.out_f32 ? 4 : 2);
    if (overlap(out, out_bytes, x, d->M * d->K * e) || overlap(out, out_bytes, weight, wn * d->K * e) ||
        overlap_in_part(out, out_bytes, residual, out_bytes))
        return GDN_ERR_UNSUPPORTED;
    int dev = 0, sms = 0;
    if (current_device_sms(&dev, &sms) != GDN_OK) return GDN_ERR_CUDA;
    void* own = nullptr;
    if (how.scratch > 0 && !workspace && cudaMallocAsync(&own, how.scratch, s) != cudaSuccess) {
        (void)cudaGetLastError();
        how.route = LinearRoute::kFfma;  // needs none
    }
    LinearMarks marks{nullptr, 0};
    if (how.route != LinearRoute::kFfma)
        st = launch_linear_tc(a, d->dtype, how.route, own ? own : workspace, dev, sms, s, &marks);
    if (st == GDN_OK && (how.route == LinearRoute::kFfma || how.route == LinearRoute::kParts)) {
        const cudaError_t e = d->dtype == GDN_F32    ? launch_ffma<float>(a, d->dtype, sms, marks, s)
                              : d->dtype == GDN_BF16 ? launch_ffma<__nv_bfloat16>(a, d->dtype, sms, marks, s)
                                                     : launch_ffma<__nv_fp8_e4m3>(a, d->dtype, sms, marks, s);
        if (e != cudaSuccess) st = GDN_ERR_CUDA;
    }
    if (own && cudaFreeAsync(own, s) != cudaSuccess && st == GDN_OK) st = GDN_ERR_CUDA;
    if (st == GDN_ERR_CUDA) (void)cudaGetLastError();  // reported here, and not by the thread's next call again
    return st;
}

extern "C" gdn_status gdn_linear(const void* x, const float* x_scale, const void* weight, const float* weight_scale,
                                 const float* bias, const void* residual, void* out, const gdn_linear_dims* d,
                                 gdn_stream_t stream) {
    return gdn_linear_ws(x, x_scale, weight, weight_scale, bias, residual, out, d, nullptr, 0, stream);
}
