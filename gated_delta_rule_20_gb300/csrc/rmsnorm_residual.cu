// rmsnorm_residual.cu -- RMS norm behind the residual's addition, over rows of D
// elements, with the normalised row in the compute dtype or in 8 bits (e4m3)
// with one scale a row:
//
//     h[r, :] = x[r, :] + residual[r, :]               (fp32; written back rounded to the compute dtype)
//     y[r, :] = h[r, :] / sqrt(mean(h[r, :]^2) + eps) * w
//     out     = y rounded once, or
//     scale[r] = max(max_i |y[r, i]|, GDN_FP8_AMAX_MIN) / 448,  out[r, i] = e4m3(y[r, i] / scale[r])
//
// One pass over HBM: the row stays in registers (or in shared memory, second
// kernel) between its statistics and its output.  The row's maximum needs no
// second reduction behind the norm: with s = 1 / sqrt(mean + eps), a positive
// factor of the whole row, max |y| = s max |h w|, so the sum of squares and
// max |h w| are reduced together.
//
// The statistics take the unrounded fp32 h; the only roundings are those of
// the two outputs.  A NaN in a row makes mean(h^2) one, and by it the row's y,
// maximum and scale, as in the formula; an infinity makes its own y NaN and the
// row's others 0 (finite / infinity), and in 8 bits the whole row and its scale
// NaN.  A row of numbers whose sum of squares passes fp32's range (|h| of 1e19
// and more) comes out as zeros.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <type_traits>

#include "gdn_device.cuh"
#include "gdn_internal.h"
#include "sm100_ptx.cuh"

namespace gdn {
namespace {

struct NormArgs {
    const void* x;
    const void* res;   // may be null
    const float* w;
    void* h;           // may be null; may be res
    void* out;         // may be x
    float* scale;      // e4m3 output only
    long long rows;
    int D;
    float eps;
};

struct F8 {};  // tag: e4m3 output with a scale a row

// (sum of squares, max |h w|) over the GROUP threads of a row.  Groups above a warp are whole
// blocks; `part` is used in turns (`turn` = 0, 1), so that one barrier a row is enough: a
// slot is written again only after the barrier of the row in between.
template <int GROUP>
__device__ __forceinline__ float2 reduce_row(float ss, float mx, float2 (*part)[GROUP / 32], int turn) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
        mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    }
    if constexpr (GROUP > 32) {
        if ((threadIdx.x & 31) == 0) part[turn][threadIdx.x >> 5] = make_float2(ss, mx);
        __syncthreads();
        ss = 0.f;
        mx = 0.f;
#pragma unroll
        for (int i = 0; i < GROUP / 32; ++i) {  // the same order in every thread
            const float2 p = part[turn][i];
            ss += p.x;
            mx = max_nan(mx, p.y);
        }
    }
    return make_float2(ss, mx);
}

// What turns h w into the output, (h w x) y: the norm's factor, over the row's scale for e4m3 (x = 1).  Where that
// passes fp32's range (rows of the least scale with a small eps, zeros among them: from 1 / sqrt(eps) = 7.6e5 on), the
// factor and the scale's inverse are applied one after the other.
template <typename O>
__device__ __forceinline__ float2 row_factor(float2 stat, const NormArgs& a, long long r, bool first) {
    const float rinv = rsqrtf(stat.x / (float)a.D + a.eps);
    if constexpr (std::is_same<O, F8>::value) {
        float m = stat.y * rinv;
        m = m < GDN_FP8_AMAX_MIN ? GDN_FP8_AMAX_MIN : m;  // a NaN stays one
        if (m > 3.4e38f) m = __int_as_float(0x7fc00000);  // an infinite weight: no scale stands for the row
        const float scale = m / 448.f;
        if (first) a.scale[r] = scale;
        const float f = rinv / scale;
        return f > 3.4e38f && rinv < 3.4e38f ? make_float2(rinv, 1.f / scale) : make_float2(1.f, f);
    } else {
        return make_float2(1.f, rinv);
    }
}
// h w, scaled as row_factor says.
template <typename O>
__device__ __forceinline__ float scaled(float hw, float2 f) {
    if constexpr (std::is_same<O, F8>::value) hw *= f.x;
    return hw * f.y;
}

// V elements as a 16-byte piece of the flat array.  One that reaches past the array's end (its last piece,
// kOdd only) is put together from the elements that exist.  (A piece over a row's end holds elements of
// the neighbouring row too, which another block may be writing: they are replaced by zeros, see below.)
template <typename T, bool kOdd>
__device__ __forceinline__ uint4 load_piece(const T* p, long long piece, long long elements) {
    constexpr int V = 16 / (int)sizeof(T);
    if (!kOdd || (piece + 1) * V <= elements) return __ldcs(reinterpret_cast<const uint4*>(p) + piece);
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    T* e = reinterpret_cast<T*>(&v);
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (piece * V + j < elements) e[j] = p[piece * V + j];
    return v;
}
// V elements of a row (`col`: the column of the first) stored as a piece, or one by one where the piece
// reaches past the row's ends; W: a word of V elements of E.
template <typename E, typename W, bool kOdd>
__device__ __forceinline__ void store_piece(E* p, long long piece, int col, int D, W v) {
    constexpr int V = (int)(sizeof(W) / sizeof(E));
    if (!kOdd || (col >= 0 && col + V <= D)) {
        reinterpret_cast<W*>(p)[piece] = v;
        return;
    }
    const E* e = reinterpret_cast<const E*>(&v);
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (col + j >= 0 && col + j < D) p[piece * V + j] = e[j];
}

// Arrays on 16 bytes: GROUP threads a row, P pieces of 16 bytes a thread.  The next row's pieces are loaded
// before this row's statistics are reduced, so that the barrier does not leave HBM idle.
// Rows of whole pieces keep their weights in registers.  Rows that are not (kOdd) start anywhere in a
// piece: the pieces are still those of the flat array, the ones at a row's ends go element by element, and
// the weights, whose place in the pieces changes from row to row, are read from shared memory, one word in
// V left out so that the threads' words lie in different banks.
template <typename T, typename O, int GROUP, int P, bool kOdd>
__global__ void __launch_bounds__(GROUP == 32 ? 256 : GROUP) rmsnorm_residual_vec_kernel(const __grid_constant__ NormArgs a) {
    constexpr int V = 16 / (int)sizeof(T);
    constexpr int kBlock = GROUP == 32 ? 256 : GROUP;
    constexpr int kRows = kBlock / GROUP;  // rows of a block at a time
    __shared__ float2 part[2][GROUP / 32];
    extern __shared__ float w_smem[];  // kOdd: [D + D / V]
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();  // the preceding kernel's results (see launch)
    const int t = threadIdx.x % GROUP, D = a.D;
    const T* x = static_cast<const T*>(a.x);
    const T* res = static_cast<const T*>(a.res);
    long long r = (long long)blockIdx.x * kRows + threadIdx.x / GROUP;
    const long long step = (long long)gridDim.x * kRows;
    uint4 xv[P], rv[P];
    // columns between a row's first piece and its start; pieces of the row
    auto shift_of = [&](long long row) { return kOdd ? (int)(row * D % V) : 0; };
    auto load = [&](long long row, int shift) {
        const long long first = (row * D - shift) / V;
        const int pieces = (shift + D + V - 1) / V;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int i = t + p * GROUP;
            if (i < pieces) {
                xv[p] = load_piece<T, kOdd>(x, first + i, a.rows * D);
                if (res) rv[p] = load_piece<T, kOdd>(res, first + i, a.rows * D);
            }
        }
    };
#pragma unroll
    for (int p = 0; p < P; ++p) xv[p] = rv[p] = make_uint4(0u, 0u, 0u, 0u);
    if (r < a.rows) load(r, shift_of(r));
    float w[kOdd ? 1 : P][V];
    if constexpr (kOdd) {
        for (int i = threadIdx.x; i < D; i += kBlock) w_smem[i + i / V] = a.w[i];
        __syncthreads();
    } else {
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int j = 0; j < V; j += 4) {
                const int i = t + p * GROUP;
                const float4 f =
                    i < D / V ? *reinterpret_cast<const float4*>(a.w + i * V + j) : make_float4(0.f, 0.f, 0.f, 0.f);
                w[p][j] = f.x;
                w[p][j + 1] = f.y;
                w[p][j + 2] = f.z;
                w[p][j + 3] = f.w;
            }
    }
    // blocks of several rows have one warp a row and no barrier in the loop; a block of one row leaves it as one
    for (int turn = 0; r < a.rows; r += step, turn ^= 1) {
        const int shift = shift_of(r), pieces = (shift + D + V - 1) / V;
        const long long first = (r * D - shift) / V;
        float h[P][V], ss = 0.f, mx = 0.f;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const T* xe = reinterpret_cast<const T*>(&xv[p]);
            const T* re = reinterpret_cast<const T*>(&rv[p]);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                h[p][j] = to_f32(xe[j]);
                if (res) h[p][j] += to_f32(re[j]);
            }
            if constexpr (kOdd) {  // zeros for what is not the row's
                const int col = (t + p * GROUP) * V - shift;
                if (col < 0 || col + V > D) {
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        if (col + j < 0 || col + j >= D) h[p][j] = 0.f;
                }
            }
#pragma unroll
            for (int j = 0; j < V; ++j) ss += h[p][j] * h[p][j];
        }
        const long long next = r + step;
        if (next < a.rows) load(next, shift_of(next));
        if (a.h) {
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const int i = t + p * GROUP;
                uint4 o;
                T* oe = reinterpret_cast<T*>(&o);
#pragma unroll
                for (int j = 0; j < V; ++j) oe[j] = from_f32<T>(h[p][j]);
                if (i < pieces) store_piece<T, uint4, kOdd>(static_cast<T*>(a.h), first + i, i * V - shift, D, o);
            }
        }
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if constexpr (kOdd) {
                    // column c = i V - shift + j of piece i lies at c + c / V, that is i (V + 1) - shift + j, and one
                    // before where j < shift; columns past the row's ends read some other weight, for an h of 0
                    const int i = t + p * GROUP;
                    const int at = i * (V + 1) - shift + j - (j < shift ? 1 : 0);
                    h[p][j] *= w_smem[min(max(at, 0), D + D / V - 1)];
                } else {
                    h[p][j] *= w[p][j];
                }
                if constexpr (std::is_same<O, F8>::value) mx = max_nan(mx, fabsf(h[p][j]));
            }
        const float2 f = row_factor<O>(reduce_row<GROUP>(ss, mx, part, turn), a, r, t == 0);
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int i = t + p * GROUP;
            if (i >= pieces) continue;
            if constexpr (std::is_same<O, F8>::value) {
                uint32_t q[V / 4];
#pragma unroll
                for (int j = 0; j < V; j += 4)
                    q[j / 4] = pack_e4m3x4(scaled<O>(h[p][j], f), scaled<O>(h[p][j + 1], f), scaled<O>(h[p][j + 2], f),
                                           scaled<O>(h[p][j + 3], f));
                if constexpr (V == 8)
                    store_piece<uint8_t, uint2, kOdd>(static_cast<uint8_t*>(a.out), first + i, i * V - shift, D,
                                                      make_uint2(q[0], q[1]));
                else
                    store_piece<uint8_t, uint32_t, kOdd>(static_cast<uint8_t*>(a.out), first + i, i * V - shift, D, q[0]);
            } else {
                uint4 o;
                T* oe = reinterpret_cast<T*>(&o);
#pragma unroll
                for (int j = 0; j < V; ++j) oe[j] = from_f32<T>(scaled<O>(h[p][j], f));
                store_piece<T, uint4, kOdd>(static_cast<T*>(a.out), first + i, i * V - shift, D, o);
            }
        }
    }
}

// Any D and any element alignment: the fp32 row waits in shared memory (D floats a row) for its
// statistics.  Loads and stores of one element a thread, kUnroll of them in flight.
template <typename T, typename O, int GROUP>
__global__ void __launch_bounds__(GROUP == 32 ? 256 : GROUP) rmsnorm_residual_any_kernel(const __grid_constant__ NormArgs a) {
    constexpr int kBlock = GROUP == 32 ? 256 : GROUP, kRows = kBlock / GROUP, kUnroll = 4;
    extern __shared__ float row_smem[];
    __shared__ float2 part[2][GROUP / 32];
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int t = threadIdx.x % GROUP;
    const long long r = (long long)blockIdx.x * kRows + threadIdx.x / GROUP;
    if (r >= a.rows) return;  // a whole warp (GROUP == 32), or none of the block
    float* row = row_smem + (threadIdx.x / GROUP) * a.D;
    const T* x = static_cast<const T*>(a.x) + r * a.D;
    const T* res = a.res ? static_cast<const T*>(a.res) + r * a.D : nullptr;
    T* ho = a.h ? static_cast<T*>(a.h) + r * a.D : nullptr;
    float ss = 0.f, mx = 0.f;
    for (int i0 = t; i0 < a.D; i0 += GROUP * kUnroll) {
        float v[kUnroll], u[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const int i = i0 + k * GROUP;
            v[k] = i < a.D ? to_f32(x[i]) : 0.f;
            u[k] = res && i < a.D ? to_f32(res[i]) : 0.f;
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const int i = i0 + k * GROUP;
            if (i >= a.D) continue;
            const float h = res ? v[k] + u[k] : v[k];
            if (ho) ho[i] = from_f32<T>(h);
            ss += h * h;
            const float hw = h * a.w[i];
            row[i] = hw;  // read back by this thread only
            if constexpr (std::is_same<O, F8>::value) mx = max_nan(mx, fabsf(hw));
        }
    }
    const float2 f = row_factor<O>(reduce_row<GROUP>(ss, mx, part, 0), a, r, t == 0);
    for (int i = t; i < a.D; i += GROUP) {
        if constexpr (std::is_same<O, F8>::value)
            static_cast<uint8_t*>(a.out)[r * a.D + i] = to_e4m3(scaled<O>(row[i], f));
        else
            static_cast<T*>(a.out)[r * a.D + i] = from_f32<T>(scaled<O>(row[i], f));
    }
}

// The kernels' CTAs may be set up while the stream's preceding kernel ends (programmatic stream
// serialization); they wait for it before they read anything.
cudaError_t launch(void (*kernel)(NormArgs), unsigned grid, int threads, size_t smem, cudaStream_t s, const NormArgs& a) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <typename T, typename O, int GROUP, int P, bool kOdd>
cudaError_t launch_rows(const NormArgs& a, int dev, int sms, cudaStream_t s) {
    constexpr int kBlock = GROUP == 32 ? 256 : GROUP, kRows = kBlock / GROUP;
    static const int fit = [] {  // blocks an SM of this instantiation, the same on every device the library is built for
        int n = 0;
        const cudaError_t e =
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, rmsnorm_residual_vec_kernel<T, O, GROUP, P, kOdd>, kBlock, 0);
        return e == cudaSuccess && n > 0 ? n : 1;
    }();
    constexpr int V = 16 / (int)sizeof(T);
    const size_t smem = kOdd ? (a.D + a.D / V) * sizeof(float) : 0;
    int per_sm = fit;
    if (kOdd && per_sm > (int)(220 * 1024 / (smem + 2048))) per_sm = (int)(220 * 1024 / (smem + 2048));
    constexpr int kMost = GROUP * P * (V + 1) * (int)sizeof(float);  // the longest row's weights and the words left out
    if constexpr (kOdd && kMost > 40 * 1024) {
        static std::atomic<bool> done[kMaxDevices];
        const cudaError_t e = allow_smem(rmsnorm_residual_vec_kernel<T, O, GROUP, P, kOdd>, kMost, done, dev);
        if (e != cudaSuccess) return e;
    }
    const long long need = (a.rows + kRows - 1) / kRows, room = (long long)sms * per_sm;
    const unsigned grid = (unsigned)(need < room ? need : room);
    return launch(rmsnorm_residual_vec_kernel<T, O, GROUP, P, kOdd>, grid, kBlock, smem, s, a);
}

template <typename T, typename O, int GROUP, int P>
cudaError_t launch_vec(const NormArgs& a, int dev, int sms, cudaStream_t s) {
    return a.D % (16 / (int)sizeof(T)) == 0 ? launch_rows<T, O, GROUP, P, false>(a, dev, sms, s)
                                            : launch_rows<T, O, GROUP, P, true>(a, dev, sms, s);
}

template <typename T, typename O, int GROUP>
cudaError_t launch_any(const NormArgs& a, int dev, cudaStream_t s) {
    constexpr int kBlock = GROUP == 32 ? 256 : GROUP, kRows = kBlock / GROUP;
    const size_t smem = (size_t)kRows * a.D * sizeof(float);
    if constexpr (GROUP == 1024) {  // (the others' rows take 32 KB at the most)
        static std::atomic<bool> done[kMaxDevices];
        const cudaError_t e =
            allow_smem(rmsnorm_residual_any_kernel<T, O, GROUP>, GDN_NORM_MAX_D * (int)sizeof(float), done, dev);
        if (e != cudaSuccess) return e;
    }
    return launch(rmsnorm_residual_any_kernel<T, O, GROUP>, (unsigned)((a.rows + kRows - 1) / kRows), kBlock, smem, s, a);
}

// The group is the smallest that holds the row in 2 or 3 pieces a thread (4 for warps, whose rows
// need no barrier, and for the widest rows).
template <typename T, typename O>
cudaError_t launch_norm(const NormArgs& a, cudaStream_t s) {
    constexpr int V = 16 / (int)sizeof(T);
    const uintptr_t wide = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.res) |
                           reinterpret_cast<uintptr_t>(a.h) | reinterpret_cast<uintptr_t>(a.out) |
                           reinterpret_cast<uintptr_t>(a.w);
    // pieces of a row (rows that are not whole pieces: with those that reach past their ends)
    const int nv = (wide & 15u) != 0 ? INT32_MAX : a.D % V == 0 ? a.D / V : (a.D + 2 * V - 2) / V;
    int dev = 0, sms = 0;
    if (current_device_sms(&dev, &sms) != GDN_OK) return cudaErrorInvalidDevice;
    if (nv <= 32) return launch_vec<T, O, 32, 1>(a, dev, sms, s);
    if (nv <= 64) return launch_vec<T, O, 32, 2>(a, dev, sms, s);
    if (nv <= 128) return launch_vec<T, O, 32, 4>(a, dev, sms, s);
    if (nv <= 256) return launch_vec<T, O, 128, 2>(a, dev, sms, s);
    if (nv <= 384) return launch_vec<T, O, 128, 3>(a, dev, sms, s);
    if (nv <= 512) return launch_vec<T, O, 256, 2>(a, dev, sms, s);
    if (nv <= 768) return launch_vec<T, O, 256, 3>(a, dev, sms, s);
    if (nv <= 1024) return launch_vec<T, O, 512, 2>(a, dev, sms, s);
    if (nv <= 1536) return launch_vec<T, O, 512, 3>(a, dev, sms, s);
    if (nv <= 2048) return launch_vec<T, O, 512, 4>(a, dev, sms, s);
    if (a.D <= 1024) return launch_any<T, O, 32>(a, dev, s);
    if (a.D <= 8192) return launch_any<T, O, 256>(a, dev, s);
    return launch_any<T, O, 1024>(a, dev, s);
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" gdn_status gdn_rmsnorm_residual(const void* x, const void* residual, const float* norm_weight,
                                           void* residual_out, void* out, float* out_scale, int64_t rows, int64_t D,
                                           int32_t dtype, int32_t out_dtype, float eps, gdn_stream_t stream) {
    if ((dtype != GDN_F32 && dtype != GDN_BF16) || (out_dtype != dtype && out_dtype != GDN_F8E4M3))
        return GDN_ERR_UNSUPPORTED;
    if (rows < 0 || D < 1 || D > GDN_NORM_MAX_D || rows > INT32_MAX || !(eps >= 0.f)) return GDN_ERR_DIMS;
    if (rows == 0) return GDN_OK;
    const bool f8 = out_dtype == GDN_F8E4M3;
    if (!x || !norm_weight || !out || (f8 && !out_scale)) return GDN_ERR_NULL;
    if (residual_out == out) return GDN_ERR_UNSUPPORTED;  // two results in one buffer
    const uintptr_t esz = dtype == GDN_BF16 ? 2 : 4;
    if (((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(residual) |
          reinterpret_cast<uintptr_t>(residual_out) | (f8 ? 0 : reinterpret_cast<uintptr_t>(out))) & (esz - 1)) ||
        ((reinterpret_cast<uintptr_t>(norm_weight) | (f8 ? reinterpret_cast<uintptr_t>(out_scale) : 0)) & 3u))
        return GDN_ERR_ALIGN;
    // in place: element by element, or not at all
    const long long in_bytes = rows * D * (long long)esz, out_bytes = f8 ? rows * D : in_bytes;
    if (overlap(out, out_bytes, residual_out, in_bytes) || overlap_in_part(out, out_bytes, x, in_bytes) ||
        overlap_in_part(out, out_bytes, residual, in_bytes) || overlap_in_part(residual_out, in_bytes, x, in_bytes) ||
        overlap_in_part(residual_out, in_bytes, residual, in_bytes))
        return GDN_ERR_UNSUPPORTED;
    const NormArgs a{x, residual, norm_weight, residual_out, out, out_scale, rows, (int)D, eps};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (dtype == GDN_BF16)
        e = f8 ? launch_norm<__nv_bfloat16, F8>(a, s) : launch_norm<__nv_bfloat16, __nv_bfloat16>(a, s);
    else
        e = f8 ? launch_norm<float, F8>(a, s) : launch_norm<float, float>(a, s);
    if (e == cudaSuccess) return GDN_OK;
    (void)cudaGetLastError();  // reported here, and not by the thread's next call again
    return GDN_ERR_CUDA;
}
