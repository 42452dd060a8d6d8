// linear_attn.cu -- linear attention with a decay for each head: entry points, the single-token step and the
// prefill on the FMA units.
//
//     S_t = e^{g_t} S_{t-1} + k_t v_t^T,     o_t = scale * S_t^T q_t        S fp32 [Dk, Dv] per (batch, value head)
//
// Step.  One pass over the state: S' = e^g S + k v^T is written as it is read and o = scale q^T S' summed on the
// way, so the state's bytes bound it.  A thread has all of its loads (32 numbers, in registers) on their way at once and makes
// its stores before the sums over rows go through shared memory; 64 registers a thread let an SM hold 128 KB of loads.
// Measured (128 x 128): 64 x 32 heads 41 us, 6.6 TB/s of the 6.8 that a copy reaches; 4 x 32 heads 3.2 us, 1 x 32 heads 2.0 us.
//
// Prefill on the FMA units (fp32 compute, and small bf16 calls of head dims off the tensor-core kernel): the recurrence itself, token by
// token, with the state in registers.  Its 2 Dk Dv multiply-adds a token are the fewest of any form (a chunked one adds
// C (Dk + Dv) / 2), and every one is an fp32 FMA on operands that lie in shared memory.  A warp owns 16
// columns: lane (d, e) = (lane % 8, lane / 8) holds rows 32 m + 4 d + {0..3} of columns 4 e + {0..3}, so that the 8 lanes of a
// column read 128 contiguous bytes of q and of k, and o is summed over them with 4 shuffles.  Rows go in pairs
// (fma.rn.f32x2).  The state is kept as S~_t = e^{-c_t} S_t, with c the sum of the log-decays since the first of 16
// staged tokens: S~ += (e^{-c_t} k_t) v_t^T, o_t = e^{c_t} scale S~^T q_t, and one product by e^{c_16} a block.  That is a third
// fewer operations than a decay a token, and one rounding of a decay in 16: with decays near 1 the functions' errors
// would add up (1.5e-6 after 290 tokens at e^-0.0005).  c is an fp32 sum, whose roundings are the largest error left
// (1.4e-7 of the outputs' norm, 1.9e-7 of the state's, at e^-0.25 a token); kept as two numbers (1.1e-7 and 0.7e-7) it takes
// up to 8 % longer.  Blocks that decay by more than e^-8 take a product a token; they forget within a few tokens.  64 packed
// FMAs a warp and token are 128 cycles of a scheduler; with the loads, the sums over lanes and what prepares v it issues some
// 200 instructions, and 32 heads of 8 warps leave a scheduler one warp or two, whose latencies show: 4 x 32 heads x 512 x 128 x
// 128 in fp32 249 us in one pass, 224 in two segments (the FMAs alone: 58); 2 x 16 heads x 2048 218 us in segments and 1022 in
// one pass.
#include <cuda_bf16.h>

#include <atomic>

#include "gdn_device.cuh"
#include "gdn_internal.h"
#include "linear_attn.h"
#include "sm100_ptx.cuh"

namespace gdn {
namespace {

constexpr int kMaxD = 128;

// ------------------------------------------------------------------ single-token step
// How a CTA's threads lie over its slice of V C columns: thread = V neighbouring columns of every rgs-th row, so that
// whole rows are read and written as one piece of memory.  kFlat (whole rows that are no multiple of 16 bytes, of heads that
// are): rgs rows are cut into C pieces of 4, whichever rows these begin and end in; as rgs Dv is a multiple of 4, a thread's
// pieces lie in the same columns all the same.
struct StepShape {
    int C, rgs;   // threads of a row (kFlat: of rgs rows); rows at once
    int group;    // value heads of a key head
    uint32_t by;  // tid / C = tid by >> 16
};
template <int V>
struct alignas(4 * V) StepPiece {
    float e[V];
};

// kRows: a thread's rows at most, all of them on their way at once.
template <typename T, int V, bool kFlat, int kRows, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) linear_attn_step_kernel(LinearAttn p, StepShape w) {
    using P = StepPiece<V>;
    __shared__ float s_q[kMaxD + 1], s_k[kMaxD + 1];
    __shared__ __align__(16) float s_red[V * kThreads];
    const int bh = blockIdx.x, C = w.C, rgs = w.rgs, tid = threadIdx.x, Dk = p.Dk, Dv = p.Dv;
    const int cols = kFlat ? Dv : V * C, base = blockIdx.y * cols;
    const int rg = kFlat ? V * tid / Dv : (int)(tid * w.by >> 16), c = base + V * tid - rg * cols;
    const bool live = kFlat ? tid < C : rg < rgs;
    const int rows = live && c < Dv ? Dk : 0;  // (the last few threads may have none)
    const size_t at = (size_t)bh * Dk * Dv + (size_t)rg * Dv + c;
    const int down = rgs * Dv;  // to a thread's next row
    ptx::griddep_wait();

    P S[kRows] = {};
    if (p.state_in) {
        const float* from = p.state_in + at;
#pragma unroll
        for (int i = 0; i < kRows; ++i, from += down) {
            if (rg + i * rgs < rows) {
                if constexpr (V == 4)
                    *reinterpret_cast<float4*>(&S[i]) = __ldcs(reinterpret_cast<const float4*>(from));
                else
                    S[i].e[0] = *from;
            }
        }
    }
    const int b = bh / p.Hv, h = bh - b * p.Hv, hk = h / w.group;
    float v[V] = {}, o[V] = {};
    if (rows) {
#pragma unroll
        for (int j = 0; j < V; ++j)
            v[j] = to_f32(static_cast<const T*>(p.v)[(size_t)bh * Dv + c + j - (kFlat && c + j >= Dv ? Dv : 0)]);
    }
    for (int i = tid; i < Dk; i += blockDim.x) {
        const size_t row = ((size_t)b * p.Hk + hk) * Dk + i;
        s_q[i] = to_f32(static_cast<const T*>(p.q)[row]);
        s_k[i] = to_f32(static_cast<const T*>(p.k)[row]);
    }
    const float a = expf(least_decay(p.g_log[p.head_decay ? h : bh]));
    __syncthreads();

    float* to = p.state_out + at;
#pragma unroll
    for (int i = 0; i < kRows; ++i, to += down) {
        const int r = rg + i * rgs;
        if (r < rows) {
            const float k0 = s_k[r], q0 = s_q[r], k1 = kFlat ? s_k[r + 1] : 0.f, q1 = kFlat ? s_q[r + 1] : 0.f;
            P x;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const bool next = kFlat && c + j >= Dv;
                const float k = next ? k1 : k0, q = next ? q1 : q0;
                x.e[j] = fmaf(a, S[i].e[j], k * v[j]);
                o[j] = fmaf(q, x.e[j], o[j]);
            }
            if constexpr (V == 4)
                __stcs(reinterpret_cast<float4*>(to), *reinterpret_cast<const float4*>(&x));
            else
                *to = x.e[0];
        }
    }
    ptx::griddep_launch_dependents();
    if (live) {
#pragma unroll
        for (int j = 0; j < V; ++j) s_red[V * tid + j] = o[j];
    }
    __syncthreads();
    for (int i = tid; i < cols && base + i < Dv; i += blockDim.x) {
        float sum = 0.f;
#pragma unroll 8
        for (int g = 0; g < rgs; ++g) sum += s_red[g * cols + i];
        static_cast<T*>(p.out)[(size_t)bh * Dv + base + i] = from_f32<T>(p.scale * sum);
    }
}

template <typename K, typename... A>
cudaError_t launch_after(K* kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream, const A&... a) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a...);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename T, int V, bool kFlat>
cudaError_t launch_step_shape(const LinearAttn& p, const StepShape& w, int slices, int threads, cudaStream_t stream) {
    constexpr int kMost = 32 / V;  // rows of a thread
    const dim3 grid((unsigned)(p.B * p.Hv), (unsigned)slices);
    if (threads > 256) return launch_after(linear_attn_step_kernel<T, V, kFlat, kMost, 512>, grid, threads, 0, stream, p, w);
    if (p.Dk > kMost / 2 * w.rgs)
        return launch_after(linear_attn_step_kernel<T, V, kFlat, kMost, 256>, grid, threads, 0, stream, p, w);
    return launch_after(linear_attn_step_kernel<T, V, kFlat, kMost / 2, 256>, grid, threads, 0, stream, p, w);
}

template <typename T, int V>
cudaError_t launch_step_rows(const LinearAttn& p, int sms, cudaStream_t stream) {
    const long long heads = (long long)p.B * p.Hv;
    // Columns of a head are independent: a CTA takes a slice of them.  Slices of 32 columns spread a few heads over the card (32
    // heads of 128 x 128 2.0 us, whole 3.1; 160 heads 3.7 and 4.7); of many heads, slices that keep to lines of 128 bytes finish
    // more evenly than whole heads (2048 heads of 128 x 96 in 32s 32 us, whole 33), others are slower (128 x 100: 46 and 29).
    const int width = heads < 2 * sms ? 32 : p.Dv % 64 == 0 ? 64 : p.Dv % 32 == 0 ? 32 : 128;
    const int slices = (p.Dv + width - 1) / width;
    StepShape w;
    w.C = ((p.Dv + slices - 1) / slices + V - 1) / V;
    w.group = p.Hv / p.Hk;
    w.by = 65536u / w.C + 1;
    // CTAs as small as leave a thread 32 numbers: an SM holds the more of them (2048 heads of 32 x 32: 3.8 us in 64 threads, 6.2 in
    // 256).
    const auto fits = [&](int threads) { return threads / w.C * (32 / V) >= p.Dk; };
    int threads = fits(256) ? 256 : 512;
    if (heads * slices >= 2 * sms)
        while (threads > 64 && fits(threads / 2)) threads /= 2;
    w.rgs = threads / w.C;
    return launch_step_shape<T, V, false>(p, w, slices, threads, stream);
}

template <typename T>
cudaError_t launch_step(const LinearAttn& p, int sms, cudaStream_t stream) {
    const bool aligned = aligned16(p.state_in) && aligned16(p.state_out);
    if (aligned && p.Dv % 4 == 0) return launch_step_rows<T, 4>(p, sms, stream);
    if (aligned && p.Dk * p.Dv % 4 == 0 && p.Dv >= 4 && (long long)p.B * p.Hv >= 2 * sms) {
        // (2048 heads of 96 x 75: 21 us instead of 24 by single numbers, of 128 x 33 14 and 17)
        const int unit = p.Dv % 2 ? 4 : 2;  // of rows that are pieces of 16 bytes together
        StepShape w;
        w.rgs = ((p.Dk + 7) / 8 + unit - 1) / unit * unit;
        w.C = w.rgs * p.Dv / 4;
        w.group = p.Hv / p.Hk;
        w.by = 0;
        return launch_step_shape<T, 4, true>(p, w, 1, (w.C + 31) / 32 * 32, stream);
    }
    return launch_step_rows<T, 1>(p, sms, stream);
}

// ------------------------------------------------------------------ prefill on the FMA units
constexpr int kTok = 16;           // tokens staged at once
constexpr float kMostBlock = 8.f;  // largest log-decay of a block that is taken off its keys

union Pair {
    float2 f;
    unsigned long long u;
};
__device__ __forceinline__ Pair pair_of(float x, float y) {
    Pair r;
    r.f = make_float2(x, y);
    return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.u) : "l"(a.u), "l"(b.u), "l"(c.u));
    return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
    Pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.u) : "l"(a.u), "l"(b.u));
    return r;
}

template <int MB>
__device__ __forceinline__ void scale_state(Pair (&S)[MB][2][4], float a) {
    const Pair aa = pair_of(a, a);
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int j = 0; j < 4; ++j) S[m][u][j] = mul2(aa, S[m][u][j]);
}

// Shared memory of a CTA: two buffers of kTok tokens' k, v and q, and the outputs, in fp32.
template <int MB, bool kStatesOnly>
struct FfmaBuffers {
    static constexpr int kDk = 32 * MB;
    __host__ __device__ static int floats(int cols) {  // of one buffer
        return kTok * ((kStatesOnly ? 1 : 2) * kDk + cols);
    }
    static size_t bytes(int cols) { return sizeof(float) * (2 * floats(cols) + (kStatesOnly ? 0 : kTok * cols)); }
};

// MB: blocks of 32 rows of the state.  kStatesOnly (the first pass of a split): segments 0 .. P - 2, end states and decays to
// the split's arrays, no outputs.  kAsync (fp32 with rows of whole 16 bytes): the next tokens are copied into the other
// buffer while these are computed; else they are loaded, and widened, between.
template <typename T, int MB, bool kStatesOnly, bool kAsync>
__global__ void __launch_bounds__(256, 2) linear_attn_ffma_kernel(LinearAttn p, LinearAttnSplit split) {
    using Buf = FfmaBuffers<MB, kStatesOnly>;
    constexpr int kDk = Buf::kDk;
    extern __shared__ __align__(16) float s_mem[];
    __shared__ float4 s_a[2][kTok];  // what a token's state is multiplied by before it, its values, and its output
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, d = lane & 7, e = lane >> 3, warps = blockDim.x >> 5;
    const int cols = 16 * warps, base = blockIdx.y * cols;
    const int mine = warp * 16 + e * 4;  // this lane's first column of the slice
    const long long heads = (long long)p.B * p.Hv, bh = blockIdx.x;
    const int seg = blockIdx.z;
    const int b = (int)(bh / p.Hv), h = (int)(bh - (long long)b * p.Hv), hk = h / (p.Hv / p.Hk);
    const int Dk = p.Dk, Dv = p.Dv, size = Buf::floats(cols);
    float* const s_o = s_mem + 2 * size;
    const long long n_state = (long long)Dk * Dv;
    ptx::griddep_wait();
    int len = p.S;
    if (p.lengths) len = max(0, min(p.S, p.lengths[b]));
    const int t0 = split.P > 1 ? seg * split.len : 0, t1 = split.P > 1 && len - t0 > split.len ? t0 + split.len : len;

    // the start state
    const float* src = p.state_in ? p.state_in + bh * n_state : nullptr;
    if (split.P > 1 && !kStatesOnly) src = split.start(seg, bh, heads, n_state);
    if (kStatesOnly && seg > 0) src = nullptr;
    float* copy = kStatesOnly && seg == 0 ? split.parts + ((split.P - 1) * heads + bh) * n_state : nullptr;
    Pair S[MB][2][4];
#pragma unroll
    for (int m = 0; m < MB; ++m) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float x[2][4];
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const int r = 32 * m + 4 * d + 2 * u + w, at = r * Dv + base + mine;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool in = r < Dk && base + mine + j < Dv;
                    x[w][j] = src && in ? src[at + j] : 0.f;
                    if (copy && in) copy[at + j] = x[w][j];
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) S[m][u][j] = pair_of(x[0][j], x[1][j]);
        }
        asm volatile("" ::: "memory");  // (no more addresses at once)
    }
    const T* qr = static_cast<const T*>(p.q) + ((size_t)b * p.Hk + hk) * p.S * Dk;
    const T* kr = static_cast<const T*>(p.k) + ((size_t)b * p.Hk + hk) * p.S * Dk;
    const T* vr = static_cast<const T*>(p.v) + (size_t)bh * p.S * Dv + base;
    T* orow = static_cast<T*>(p.out) + (size_t)bh * p.S * Dv + base;
    const float* gr = p.g_log + (p.head_decay ? h : (size_t)bh * p.S);
    const int here = min(cols, Dv - base);  // of the slice's columns

    // channels past Dk are zeros; nothing else that is not there is used
    for (int i = tid; i < 2 * size; i += blockDim.x) s_mem[i] = 0.f;
    __syncthreads();
    // tokens t .. t + n - 1 into a buffer; a warp takes every `warps`-th token
    const auto stage = [&](float* buf, int t, int n) {
        float* sk = buf;
        float* sv = buf + kTok * kDk;
        float* sq = sv + kTok * cols;
        if (kAsync) {
            for (int tok = warp; tok < n; tok += warps) {
                const size_t row = (size_t)(t + tok) * Dk + 4 * lane;
                if (4 * lane < Dk) {
                    ptx::cp_async_16(sk + tok * kDk + 4 * lane, kr + row);
                    if (!kStatesOnly) ptx::cp_async_16(sq + tok * kDk + 4 * lane, qr + row);
                }
                if (4 * lane < here)
                    ptx::cp_async_16(sv + tok * cols + 4 * lane, vr + (size_t)(t + tok) * Dv + 4 * lane);
            }
        } else {
#pragma unroll 4
            for (int i = 0; i < kTok; ++i) {
                const int tok = warp + i * warps;
                if (tok < n) {
                    const size_t row = (size_t)(t + tok) * Dk;
#pragma unroll
                    for (int m = 0; m < MB; ++m) {
                        const int c = 32 * m + lane;
                        if (c < Dk) {
                            sk[tok * kDk + c] = to_f32(kr[row + c]);
                            if (!kStatesOnly) sq[tok * kDk + c] = to_f32(qr[row + c]);
                        }
                    }
                    for (int c = lane; c < here; c += 32) sv[tok * cols + c] = to_f32(vr[(size_t)(t + tok) * Dv + c]);
                }
            }
        }
    };
    if (kAsync && t0 < t1) {
        stage(s_mem, t0, min(kTok, t1 - t0));
        ptx::cp_async_commit();
    }
    float decay = 1.f, g_next = 0.f;
    if (t0 + lane < t1 && lane < kTok) g_next = gr[p.head_decay ? 0 : t0 + lane];

    int turn = 0;
    for (int t = t0; t < t1; t += kTok, ++turn) {
        const int n = min(kTok, t1 - t);
        float* buf = s_mem + (kAsync ? (turn & 1) * size : 0);
        if (!kAsync) stage(buf, t, n);
        // every warp sums the log-decays: lane i has token i's
        const float g = lane < n ? least_decay(g_next) : 0.f;
        if (t + kTok + lane < t1 && lane < kTok) g_next = gr[p.head_decay ? 0 : t + kTok + lane];
        float c_in = g;
#pragma unroll
        for (int o = 1; o < kTok; o <<= 1) {
            const float y = __shfl_up_sync(0xffffffffu, c_in, o);
            if (lane >= o) c_in += y;
        }
        const bool blockwise = __all_sync(0xffffffffu, !(fabsf(c_in) > kMostBlock) || lane >= kTok);
        const float total = __shfl_sync(0xffffffffu, c_in, kTok - 1);
        if (warp == 0 && lane < kTok)
            s_a[turn & 1][lane] =
                blockwise ? make_float4(1.f, expf(-c_in), expf(c_in), 0.f) : make_float4(expf(g), 1.f, 1.f, 0.f);
        if (kAsync) ptx::cp_async_wait_all();
        __syncthreads();  // the buffer and s_a are there; the other buffer has been read
        if (kAsync && t + kTok < t1) {
            stage(s_mem + ((turn + 1) & 1) * size, t + kTok, min(kTok, t1 - t - kTok));
            ptx::cp_async_commit();
        }
        if (kStatesOnly) decay *= expf(total);
        const float* sk = buf + 4 * d;
        const float* sv = buf + kTok * kDk + mine;
        const float* sq = buf + kTok * (kDk + cols) + 4 * d;
#pragma unroll 1  // (two tokens a turn take 3 to 5 % longer)
        for (int i = 0; i < n; ++i, sk += kDk, sv += cols, sq += kDk) {
            const float4 a = s_a[turn & 1][i];
            if (!blockwise) scale_state(S, a.x);
            const float4 v4 = *reinterpret_cast<const float4*>(sv);
            const Pair vv[4] = {pair_of(a.y * v4.x, a.y * v4.x), pair_of(a.y * v4.y, a.y * v4.y),
                                pair_of(a.y * v4.z, a.y * v4.z), pair_of(a.y * v4.w, a.y * v4.w)};
            Pair o[4];
#pragma unroll
            for (int m = 0; m < MB; ++m) {
                const float4 k4 = *reinterpret_cast<const float4*>(sk + 32 * m);
                const Pair kk[2] = {pair_of(k4.x, k4.y), pair_of(k4.z, k4.w)};
                Pair qq[2] = {};
                if (!kStatesOnly) {
                    const float4 q4 = *reinterpret_cast<const float4*>(sq + 32 * m);
                    qq[0] = pair_of(q4.x, q4.y);
                    qq[1] = pair_of(q4.z, q4.w);
                }
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        S[m][u][j] = fma2(kk[u], vv[j], S[m][u][j]);
                        if (!kStatesOnly) o[j] = m + u ? fma2(qq[u], S[m][u][j], o[j]) : mul2(qq[u], S[m][u][j]);
                    }
            }
            if (!kStatesOnly) {
                // the sum over the 8 lanes of a column group: each keeps two columns, then one
                float x[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = o[j].f.x + o[j].f.y;
                const bool up = d & 4, up2 = d & 2;
                const float y0 = (up ? x[2] : x[0]) + __shfl_xor_sync(0xffffffffu, up ? x[0] : x[2], 4);
                const float y1 = (up ? x[3] : x[1]) + __shfl_xor_sync(0xffffffffu, up ? x[1] : x[3], 4);
                float z = (up2 ? y1 : y0) + __shfl_xor_sync(0xffffffffu, up2 ? y0 : y1, 2);
                z += __shfl_xor_sync(0xffffffffu, z, 1);
                if (!(d & 1)) s_o[i * cols + mine + (up ? 2 : 0) + (up2 ? 1 : 0)] = a.z * z;
            }
        }
        if (blockwise) scale_state(S, expf(total));
        if (!kStatesOnly || !kAsync) __syncthreads();  // the outputs are there, and the buffer has been read
        if (!kStatesOnly)
            for (int tok = warp; tok < n; tok += warps)
                for (int c = lane; c < here; c += 32)
                    orow[(size_t)(t + tok) * Dv + c] = from_f32<T>(p.scale * s_o[tok * cols + c]);
    }
    ptx::griddep_launch_dependents();

    float* dst = nullptr;
    if (kStatesOnly) {
        dst = split.parts + (seg * heads + bh) * n_state;
        if (tid == 0 && blockIdx.y == 0) split.decays[seg * heads + bh] = decay;
    } else if (seg == split.P - 1) {
        dst = p.state_out + bh * n_state;
    }
    if (!dst) return;
#pragma unroll
    for (int m = 0; m < MB; ++m) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const int r = 32 * m + 4 * d + 2 * u + w, at = r * Dv + base + mine;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (r < Dk && base + mine + j < Dv) dst[at + j] = w ? S[m][u][j].f.y : S[m][u][j].f.x;
            }
        asm volatile("" ::: "memory");
    }
}

template <typename T, int MB, bool kStatesOnly, bool kAsync>
cudaError_t launch_ffma_kernel(const LinearAttn& p, const LinearAttnSplit& s, int warps, int dev, cudaStream_t stream) {
    using Buf = FfmaBuffers<MB, kStatesOnly>;
    static std::atomic<bool> allowed[kMaxDevices];
    auto* kernel = linear_attn_ffma_kernel<T, MB, kStatesOnly, kAsync>;
    if (Buf::bytes(kMaxD) + 1024 > 48 * 1024) {  // (with s_a)
        const cudaError_t e = allow_smem(kernel, (int)Buf::bytes(kMaxD), allowed, dev);
        if (e != cudaSuccess) return e;
    }
    const dim3 grid((unsigned)(p.B * p.Hv), (unsigned)((p.Dv + 16 * warps - 1) / (16 * warps)),
                    (unsigned)(kStatesOnly ? s.P - 1 : s.P));
    return launch_after(kernel, grid, 32 * warps, Buf::bytes(16 * warps), stream, p, s);
}

template <typename T, int MB, bool kAsync>
cudaError_t launch_ffma_rows(const LinearAttn& p, const LinearAttnSplit& s, int dev, int sms, cudaStream_t stream) {
    // as many columns a CTA as leave every SM two CTAs (its warps share the staged q and k)
    const long long heads = (long long)p.B * p.Hv;
    int warps = 8;
    while (warps > 1 && (16 * (warps / 2) >= p.Dv || heads * s.P * ((p.Dv + 16 * warps - 1) / (16 * warps)) < 2 * sms))
        warps /= 2;
    if (s.P > 1) {
        cudaError_t e = launch_ffma_kernel<T, MB, true, kAsync>(p, s, warps, dev, stream);
        if (e == cudaSuccess) e = launch_linear_attn_combine(p, s, stream);
        if (e != cudaSuccess) return e;
    }
    return launch_ffma_kernel<T, MB, false, kAsync>(p, s, warps, dev, stream);
}

template <typename T, bool kAsync>
cudaError_t launch_ffma(const LinearAttn& p, const LinearAttnSplit& s, int dev, int sms, cudaStream_t stream) {
    switch ((p.Dk + 31) / 32) {
        case 1: return launch_ffma_rows<T, 1, kAsync>(p, s, dev, sms, stream);
        case 2: return launch_ffma_rows<T, 2, kAsync>(p, s, dev, sms, stream);
        case 3: return launch_ffma_rows<T, 3, kAsync>(p, s, dev, sms, stream);
        default: return launch_ffma_rows<T, 4, kAsync>(p, s, dev, sms, stream);
    }
}

// ------------------------------------------------------------------ the states of a split
// X_j += F_j X_{j-1} for j = 1 .. P - 2: a thread V elements of a state, the loads of eight segments at once in front of their
// sums.  n elements of a state are `slices` CTAs' work.  Bound by bytes, of which the first pass left most in L2: 9 segments of
// 32 heads 8 us less in all than with one number and segment at a time (271 -> 261 us for 32768 tokens).
template <int V>
__global__ void __launch_bounds__(256) linear_attn_combine_kernel(LinearAttnSplit s, int heads, int slices, int n) {
    struct alignas(4 * V) Some {
        float e[V];
    };
    const int bh = blockIdx.x / slices, at = ((blockIdx.x - bh * slices) * 256 + threadIdx.x) * V;
    ptx::griddep_wait();
    if (at < n) {
        float* part = s.parts + (long long)bh * n + at;
        const float* decay = s.decays + bh;
        const long long next = (long long)heads * n;
        Some x = *reinterpret_cast<const Some*>(part);
#pragma unroll 1
        for (int left = s.P - 2; left > 0; left -= 8) {
            Some y[8];
            float f[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (u < left) {
                    y[u] = *reinterpret_cast<const Some*>(part + (u + 1) * next);
                    f[u] = decay[(long long)(u + 1) * heads];
                }
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (u < left) {
#pragma unroll
                    for (int i = 0; i < V; ++i) x.e[i] = fmaf(f[u], x.e[i], y[u].e[i]);
                    *reinterpret_cast<Some*>(part + (u + 1) * next) = x;
                }
            part += 8 * next;
            decay += 8ll * heads;
        }
    }
    ptx::griddep_launch_dependents();
}

}  // namespace

cudaError_t launch_linear_attn_combine(const LinearAttn& p, const LinearAttnSplit& s, cudaStream_t stream) {
    if (s.P <= 2) return cudaSuccess;
    const int heads = p.B * p.Hv, n = p.Dk * p.Dv, V = n % 4 == 0 ? 4 : 1, slices = (n + 256 * V - 1) / (256 * V);
    const dim3 grid((unsigned)(heads * slices));  // (a split's states fit in memory: far fewer than 2^31)
    if (V == 4) return launch_after(linear_attn_combine_kernel<4>, grid, 256, 0, stream, s, heads, slices, n);
    return launch_after(linear_attn_combine_kernel<1>, grid, 256, 0, stream, s, heads, slices, n);
}

namespace {

// ------------------------------------------------------------------ rows for the tensor-core kernel
// q and k, or v, with their channels padded with zeros to multiples of 8 (rows that TMA can read).  A thread 8 channels of a row;
// rows behind a length are left out.  Bound by bytes.
struct PadRows {
    const __nv_bfloat16* src[3];  // q, k, v
    __nv_bfloat16* dst[3];        // (null: not padded)
    int heads[3], D[3], P[3];
    Divisor pieces[3], tokens[3], batch[3];  // of a row; by S; by heads S
    const int32_t* lengths;
    int B, S;
};
__global__ void __launch_bounds__(256) linear_attn_pad_kernel(const __grid_constant__ PadRows a) {
    ptx::griddep_wait();
    const int w = blockIdx.y;
    if (a.dst[w]) {
        const int D = a.D[w], P = a.P[w], all = a.B * a.heads[w] * a.S * (P / 8);
        for (long long n0 = (long long)blockIdx.x * 256 + threadIdx.x; n0 < all; n0 += (long long)gridDim.x * 256) {
            const int n = (int)n0, row = a.pieces[w].of(n), c = 8 * (n - row * (P / 8));
            if (a.lengths && row - a.tokens[w].of(row) * a.S >= a.lengths[a.batch[w].of(row)]) continue;
            const unsigned short* from = reinterpret_cast<const unsigned short*>(a.src[w]) + (long long)row * D + c;
            uint32_t x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = c + i < D ? from[i] : 0;
            *reinterpret_cast<uint4*>(a.dst[w] + (long long)row * P + c) =
                make_uint4(x[0] | x[1] << 16, x[2] | x[3] << 16, x[4] | x[5] << 16, x[6] | x[7] << 16);
        }
    }
    ptx::griddep_launch_dependents();
}

// Outputs out of padded rows: a thread 8 elements of a head's [S, Dv] that are 16 aligned bytes; rows behind a length are left as
// they are, or zeroed.  `blocks` CTAs a head.
__global__ void __launch_bounds__(256) linear_attn_unpad_kernel(LinearAttn p, const unsigned short* padded, Divisor row_of, int blocks) {
    ptx::griddep_wait();
    const int bh = blockIdx.x / blocks, all = p.S * p.Dv;
    unsigned short* out = static_cast<unsigned short*>(p.out) + (long long)bh * all;
    const int before = (int)((reinterpret_cast<uintptr_t>(out) & 15) / 2);  // elements from 16 aligned bytes to the head's first
    int len = p.S;
    if (p.lengths) len = max(0, min(p.S, p.lengths[bh / p.Hv]));
    const int written = p.zero_rest ? all : len * p.Dv, given = len * p.Dv;
    const unsigned short* from = padded + (long long)bh * p.S * p.Pv;
    for (int e0 = ((blockIdx.x - bh * blocks) * 256 + threadIdx.x) * 8 - before; e0 < written; e0 += blocks * 2048) {
        uint32_t x[8];
        int row = row_of.of(max(e0, 0)), c = max(e0, 0) - row * p.Dv;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = e0 + i;
            x[i] = e >= 0 && e < given ? from[(long long)row * p.Pv + c] : 0;
            if (e >= 0 && ++c == p.Dv) {
                c = 0;
                ++row;
            }
        }
        if (e0 >= 0 && e0 + 8 <= written) {
            *reinterpret_cast<uint4*>(out + e0) =
                make_uint4(x[0] | x[1] << 16, x[2] | x[3] << 16, x[4] | x[5] << 16, x[6] | x[7] << 16);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (e0 + i >= 0 && e0 + i < written) out[e0 + i] = (unsigned short)x[i];
        }
    }
    ptx::griddep_launch_dependents();
}

// ------------------------------------------------------------------ host side
constexpr uint32_t kKnownFlags = GDN_FORCE_FFMA | GDN_SINGLE_PASS | GDN_HEAD_DECAY;  // (and GDN_ZERO_PADDING of a prompt)

gdn_status check_dims(const gdn_dims* d, bool step) {
    if (!d) return GDN_ERR_NULL;
    if (d->dtype != GDN_F32 && d->dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
    if (d->flags & ~(kKnownFlags | (step ? 0u : (uint32_t)GDN_ZERO_PADDING))) return GDN_ERR_UNSUPPORTED;
    if (d->B < 0 || d->Hk < 1 || d->Hv < 1 || d->S < 0 || d->Dk < 1 || d->Dv < 1) return GDN_ERR_DIMS;
    if (d->Dk > kMaxD || d->Dv > kMaxD || d->Hv % d->Hk != 0 || (step && d->S != 1)) return GDN_ERR_DIMS;
    // (tokens are counted in 32 bits, to the end of the last chunk of 128)
    if (d->B > INT32_MAX || d->Hv > INT32_MAX || d->S > INT32_MAX - 4096 || d->B * d->Hv > INT32_MAX) return GDN_ERR_DIMS;
    if (d->B * d->Hv > (int64_t(1) << 48) / (d->S + 1)) return GDN_ERR_DIMS;  // byte counts stay within 64 bits
    return GDN_OK;
}

gdn_status check(const void* q, const void* k, const void* v, const float* g_log, const int32_t* lengths, float scale,
                 const float* state_in, float* state_out, void* out, const gdn_dims* d, bool step, LinearAttn* p) {
    const gdn_status s = check_dims(d, step);
    if (s != GDN_OK) return s;
    if (d->B == 0) {
        p->B = 0;
        return GDN_OK;
    }
    const bool empty = d->S == 0;
    if (!state_out || (!empty && (!q || !k || !v || !g_log || !out))) return GDN_ERR_NULL;
    const uintptr_t el = d->dtype == GDN_BF16 ? 2 : 4;
    const auto off = [](const void* a, uintptr_t n) { return (reinterpret_cast<uintptr_t>(a) & (n - 1)) != 0; };
    if (off(q, el) || off(k, el) || off(v, el) || off(out, el) || off(g_log, 4) || off(lengths, 4) || off(state_in, 4) ||
        off(state_out, 4))
        return GDN_ERR_ALIGN;
    const long long qk = d->B * d->Hk * d->S * d->Dk * (long long)el, vo = d->B * d->Hv * d->S * d->Dv * (long long)el;
    const long long st = d->B * d->Hv * d->Dk * d->Dv * 4;
    const long long gs = (d->flags & GDN_HEAD_DECAY ? d->Hv : d->B * d->Hv * d->S) * 4;
    // what is written lies over nothing that is read, but for the state in its own place
    if (overlap(out, vo, q, qk) || overlap(out, vo, k, qk) || overlap(out, vo, v, vo) || overlap(out, vo, g_log, gs) ||
        overlap(out, vo, state_in, st) || overlap(out, vo, state_out, st) || overlap(out, vo, lengths, 4 * d->B) ||
        overlap(state_out, st, q, qk) || overlap(state_out, st, k, qk) || overlap(state_out, st, v, vo) ||
        overlap(state_out, st, g_log, gs) || overlap(state_out, st, lengths, 4 * d->B) ||
        overlap_in_part(state_out, st, state_in, st))
        return GDN_ERR_UNSUPPORTED;
    *p = LinearAttn{q, k, v, g_log, lengths, state_in, state_out, out, scale, (int)d->B, (int)d->Hk, (int)d->Hv, (int)d->S,
                    (int)d->Dk, (int)d->Dv, d->dtype == GDN_BF16, (d->flags & GDN_HEAD_DECAY) != 0, lengths && (d->flags & GDN_ZERO_PADDING), (int)d->Dk, (int)d->Dv};
    return GDN_OK;
}

// Heads that the tensor-core kernel takes.  Its CTAs walk theirs one by one, 1.2 to 4 us for one without a token, while other
// roles wait, and waits are bounded (2 s): 2^24 heads are 0.14 s for an SM.  (Of 2^28 without tokens, 8 x 8 each, the waits would
// run out.)  So many heads have some hundreds of tokens at the most in any memory, and fare as well on the FMA units: 2^22 heads of
// 1 token 91 ms on the tensor cores and 5.4, 2^20 of 130 tokens 32 and 38.
constexpr int64_t kMostHeads = 1 << 24;
bool tensor_core_call(const gdn_dims* d) {
    return d->dtype == GDN_BF16 && !(d->flags & GDN_FORCE_FFMA) && d->B * d->Hv <= kMostHeads;
}

// Whether rows are padded for the tensor cores: bf16 with channels that are no multiple of 8.  Small calls keep the recurrence on
// the FMA units (two more launches), and so do heads of a few tokens: a chunk of 128 takes the tensor cores 2.5 us an SM however
// few of them there are.  us, FMA units and tensor cores: 4 x 32 heads x 4096 x 77 x 75 1824, 176; 1 x 8 x 500 x 77 x 75 36, 18;
// 8 x 4 x 100 x 33 x 35 23, 10; 64 x 32 x 2 x 100 x 100 82, 62; but 64 x 32 x 20 x 30 x 30 28, 56.
constexpr double kPadWork = 3e6;    // state elements over all tokens
constexpr int64_t kPadHead = 24576;  // and over a head's, as the FMA units take them: 32 rows and 16 columns at once
bool padded(const gdn_dims* d) {
    return tensor_core_call(d) && (d->Dk % 8 || d->Dv % 8) &&
           (double)d->B * d->Hv * d->S * d->Dk * d->Dv > kPadWork &&
           d->S * ((d->Dk + 31) / 32 * 32) * ((d->Dv + 15) / 16 * 16) > kPadHead &&
           d->B * d->Hv * d->S < INT32_MAX / 16 - 4096 && d->S * d->Dv < INT32_MAX / 2;  // (what these launches count in 32 bits)
}
bool tensor_core_dims(const gdn_dims* d) {
    return tensor_core_call(d) && ((d->Dk % 8 == 0 && d->Dv % 8 == 0) || padded(d));
}
// Bytes of the padded q and k (each), and v and out.
struct PadBytes {
    size_t qk, vo;
    size_t all() const { return 2 * (qk + vo); }
};
PadBytes pad_bytes(const gdn_dims* d) {
    if (!padded(d)) return {0, 0};
    const auto of = [&](int64_t heads, int64_t D) {
        return D % 8 ? ((size_t)(d->B * heads * d->S * ((D + 7) / 8 * 8)) * 2 + 255) / 256 * 256 : 0;
    };
    return {of(d->Hk, d->Dk), of(d->Hv, d->Dv)};
}

// Segments that a sequence is cut into, of *len tokens: as many as make the call shortest by an estimate of its launches, and
// only if that saves a tenth (by dims alone: operands off 16 bytes, which run on the FMA units, are cut alike).
// A unit (128 tokens on the tensor cores, 16 on the FMA units) takes `whole` us in the last launch and `states` in the first;
// a launch of a split costs `launch` more, and a combine step and a state's way to and from memory `state`.  Measured on the
// tensor cores: a unit 2.2 us where 32 CTAs have HBM to themselves and 2.6 where 128 share it, and 1.6 in the first launch;
// the others are estimates.  With 2.6 and 1.6 instead of 2.5 and 1.5 none of twelve shapes (1 to 128 heads, 1000 to 131072
// tokens) is cut otherwise, with 2.2 and 1.6 one (36 heads x 1237, whole).  Of forced splits of 1 x 32 heads x 32768 tokens into 4
// to 37 segments the 9 that it picks are the fastest, 262 us (4: 271, 14: 266, 10: 291, one pass: 562); of 8192 tokens 4
// segments, 81 us (one pass 147, 8 segments 88); 4 x 32 heads x 4096 stay whole, 86 us (2 segments: 122).  (All in a graph.)
int segments(const gdn_dims* d, int sms, int* len) {
    *len = (int)d->S;
    const bool tc = tensor_core_dims(d);
    const int unit = tc ? 128 : kTok;
    const double whole = tc ? 2.5 : 8.0, states = tc ? 1.5 : 5.0, launch = 4.0, state = 0.05;
    const long long heads = (long long)d->B * d->Hv, units = (d->S + unit - 1) / unit, room = tc ? sms : 2ll * sms;
    if ((d->flags & GDN_SINGLE_PASS) || units < 2) return 1;
    const auto rounds = [&](long long items) { return (double)((items + room - 1) / room); };
    double best = 0.9 * rounds(heads) * (units * whole + launch);
    int P = 1;
    for (int n = 2; n <= 64 && n <= units; ++n) {
        const long long each = (units + n - 1) / n;
        if ((n - 1) * each >= units) continue;  // (the last segment would be empty)
        const double t = rounds(heads * (n - 1)) * (each * states + launch) + rounds(heads * n) * (each * whole + launch) +
                         launch + state * n;
        if (t < best) {
            best = t;
            P = n;
            *len = (int)(each * unit);
        }
    }
    return P;
}

// CTAs that run parts of the heads left over by whole rounds of all SMs (see Items in linear_attn_tc.cu), of *len tokens; 0: none.
// A head is cut into as many parts as there are rounds in front of the last and CTAs for, if that saves 4 chunks of 128 tokens:
// the hand-over costs some 8 us.
int handed_parts(const gdn_dims* d, int sms, int* len) {
    const long long heads = (long long)d->B * d->Hv, units = (d->S + 127) / 128, whole = heads / sms, rest = heads % sms;
    if ((d->flags & GDN_SINGLE_PASS) || !tensor_core_dims(d)) return 0;
    if (whole < 1 || rest < 1) return 0;
    long long n = sms / rest < whole + 1 ? sms / rest : whole + 1;
    while (n > 1 && (n - 1) * ((units + n - 1) / n) >= units) --n;  // (the last part would be empty)
    if (n < 2 || units - (units + n - 1) / n < 4) return 0;
    *len = (int)((units + n - 1) / n * 128);
    return (int)(n * rest);
}

// q, k and v into padded rows at `to`, and *r the call on these.
gdn_status pad_rows(const LinearAttn& p, const PadBytes& pb, uint8_t* to, int sms, cudaStream_t stream, LinearAttn* r) {
    PadRows a{};
    const void* src[3] = {p.q, p.k, p.v};
    const size_t at[3] = {0, pb.qk, 2 * pb.qk};
    const auto up = [](int D) { return (D + 7) / 8 * 8; };
    long long most = 0;
    for (int w = 0; w < 3; ++w) {
        const bool vo = w == 2;
        a.src[w] = static_cast<const __nv_bfloat16*>(src[w]);
        a.dst[w] = (vo ? pb.vo : pb.qk) ? reinterpret_cast<__nv_bfloat16*>(to + at[w]) : nullptr;
        a.heads[w] = vo ? p.Hv : p.Hk;
        a.D[w] = vo ? p.Dv : p.Dk;
        a.P[w] = up(a.D[w]);
        a.pieces[w] = divisor(a.P[w] / 8);
        a.tokens[w] = divisor(p.S);
        a.batch[w] = divisor(a.heads[w] * p.S);
        const long long n = (long long)p.B * a.heads[w] * p.S * (a.P[w] / 8);
        if (a.dst[w] && n > most) most = n;
    }
    a.lengths = p.lengths;
    a.B = p.B;
    a.S = p.S;
    const long long blocks = (most + 255) / 256;
    const dim3 grid((unsigned)(blocks < 16ll * sms ? blocks : 16ll * sms), 3);
    if (launch_after(linear_attn_pad_kernel, grid, 256, 0, stream, a) != cudaSuccess) return GDN_ERR_CUDA;
    if (pb.qk) {
        r->q = a.dst[0];
        r->k = a.dst[1];
        r->Pk = a.P[0];
    }
    if (pb.vo) {
        r->v = a.dst[2];
        r->out = to + 2 * pb.qk + pb.vo;
        r->Pv = a.P[2];
        r->zero_rest = false;
    }
    return GDN_OK;
}
gdn_status unpad_rows(const LinearAttn& p, const LinearAttn& r, cudaStream_t stream) {
    LinearAttn o = p;
    o.Pv = r.Pv;
    const long long pieces = ((long long)p.S * p.Dv + 7) / 8 + 1, per_head = (pieces + 1023) / 1024, heads = (long long)p.B * p.Hv;
    const int blocks = (int)(heads * per_head > INT32_MAX ? 1 : per_head);
    return launch_after(linear_attn_unpad_kernel, dim3((unsigned)(heads * blocks)), 256, 0, stream, o,
                        static_cast<const unsigned short*>(r.out), divisor(p.Dv), blocks) == cudaSuccess
               ? GDN_OK
               : GDN_ERR_CUDA;
}

}  // namespace
}  // namespace gdn

extern "C" {

gdn_status gdn_linear_attn_prefill(const void* q, const void* k, const void* v, const float* g_log, const int32_t* lengths,
                                   float scale, const float* state_in, float* state_out, void* out, const gdn_dims* dims,
                                   void* workspace, size_t workspace_bytes, gdn_stream_t stream) {
    gdn::LinearAttn p{};
    gdn_status s = gdn::check(q, k, v, g_log, lengths, scale, state_in, state_out, out, dims, false, &p);
    if (s != GDN_OK || p.B == 0) return s;
    if (!gdn::aligned16(workspace)) return GDN_ERR_ALIGN;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (p.S == 0) {  // no tokens: the state is the one that came in
        const size_t bytes = (size_t)p.B * p.Hv * p.Dk * p.Dv * sizeof(float);
        if (state_in == state_out) return GDN_OK;
        const cudaError_t e = state_in ? cudaMemcpyAsync(state_out, state_in, bytes, cudaMemcpyDeviceToDevice, st)
                                       : cudaMemsetAsync(state_out, 0, bytes, st);
        return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
    }
    int dev = 0, sms = 0;
    s = gdn::current_device_sms(&dev, &sms);
    if (s != GDN_OK) return s;
    // the rows that the tensor cores read and write: the caller's, or padded ones
    const gdn::PadBytes pb = gdn::pad_bytes(dims);
    const bool pad = pb.all() > 0;
    bool tc = gdn::tensor_core_dims(dims) && (pb.qk || (gdn::aligned16(q) && gdn::aligned16(k))) &&
              (pb.vo || (gdn::aligned16(v) && gdn::aligned16(out)));
    gdn::LinearAttnSplit split{1, p.S, nullptr, nullptr, 0, nullptr};
    int len = 0;
    const int P = gdn::segments(dims, sms, &len), handed = P == 1 && tc ? gdn::handed_parts(dims, sms, &len) : 0;
    const size_t base = P > 1 ? gdn::linear_attn_split_bytes(p, P) : gdn::linear_attn_flag_bytes(handed);
    const size_t at = (base + 255) / 256 * 256, need = tc && pad ? at + pb.all() : base;
    bool own = false;
    void* ws = nullptr;
    if (need) {
        if (workspace) {
            if (workspace_bytes < need) return GDN_ERR_WORKSPACE;
            ws = workspace;
        } else if (cudaMallocAsync(&ws, need, st) == cudaSuccess) {
            own = true;
        } else {
            (void)cudaGetLastError();  // one pass instead, of the rows as they are
            ws = nullptr;
            if (pad) tc = false;
        }
        if (ws && handed) {
            split.len = len;
            split.handed = handed;
            split.flags = static_cast<uint32_t*>(ws);
        } else if (ws && P > 1) {
            float* f = static_cast<float*>(ws);
            split = {P, len, f, f + (size_t)P * p.B * p.Hv * p.Dk * p.Dv, 0, nullptr};
        }
    }
    if (tc) {
        int32_t* status = nullptr;
        s = gdn::status_word_for_current_device(&status);
        gdn::LinearAttn r = p;
        if (s == GDN_OK && pad) s = gdn::pad_rows(p, pb, static_cast<uint8_t*>(ws) + at, sms, st, &r);
        if (s == GDN_OK) s = gdn::launch_linear_attn_tc(r, split, dev, sms, status, st);
        if (s == GDN_OK && pb.vo) s = gdn::unpad_rows(p, r, st);
    } else {
        const bool async =
            !p.bf16 && p.Dk % 4 == 0 && p.Dv % 4 == 0 && gdn::aligned16(q) && gdn::aligned16(k) && gdn::aligned16(v);
        cudaError_t e = cudaSuccess;
        if (p.zero_rest) e = cudaMemsetAsync(out, 0, (size_t)p.B * p.Hv * p.S * p.Dv * (p.bf16 ? 2 : 4), st);
        if (e == cudaSuccess)
            e = p.bf16  ? gdn::launch_ffma<__nv_bfloat16, false>(p, split, dev, sms, st)
                : async ? gdn::launch_ffma<float, true>(p, split, dev, sms, st)
                        : gdn::launch_ffma<float, false>(p, split, dev, sms, st);
        s = e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
    }
    if (s != GDN_OK) (void)cudaGetLastError();
    if (own && cudaFreeAsync(ws, st) != cudaSuccess && s == GDN_OK) s = GDN_ERR_CUDA;
    return s;
}

gdn_status gdn_linear_attn_step(const void* q, const void* k, const void* v, const float* g_log, float scale,
                                const float* state_in, float* state_out, void* out, const gdn_dims* dims,
                                gdn_stream_t stream) {
    gdn::LinearAttn p{};
    gdn_status s = gdn::check(q, k, v, g_log, nullptr, scale, state_in, state_out, out, dims, true, &p);
    if (s != GDN_OK || p.B == 0) return s;
    int dev = 0, sms = 0;
    s = gdn::current_device_sms(&dev, &sms);
    if (s != GDN_OK) return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = p.bf16 ? gdn::launch_step<__nv_bfloat16>(p, sms, st) : gdn::launch_step<float>(p, sms, st);
    if (e == cudaSuccess) return GDN_OK;
    (void)cudaGetLastError();
    return GDN_ERR_CUDA;
}

int32_t gdn_linear_attn_segments(const gdn_dims* dims, int32_t sm_count) {
    if (gdn::check_dims(dims, false) != GDN_OK || sm_count < 1) return 0;
    int len = 0;
    if (dims->B == 0 || dims->S == 0) return 1;
    return gdn::segments(dims, sm_count, &len);
}

size_t gdn_linear_attn_workspace_bytes(const gdn_dims* dims) {
    int dev = 0, sms = 0;
    if (gdn::check_dims(dims, false) != GDN_OK) return 0;
    if (gdn::current_device_sms(&dev, &sms) != GDN_OK) {
        (void)cudaGetLastError();
        return 0;
    }
    gdn::LinearAttn p{};
    p.B = (int)dims->B;
    p.Hv = (int)dims->Hv;
    p.Dk = (int)dims->Dk;
    p.Dv = (int)dims->Dv;
    const int P = gdn_linear_attn_segments(dims, sms);
    int len = 0;
    const size_t base =
        P > 1 ? gdn::linear_attn_split_bytes(p, P) : gdn::linear_attn_flag_bytes(gdn::handed_parts(dims, sms, &len));
    const size_t pad = gdn::pad_bytes(dims).all();
    return pad ? (base + 255) / 256 * 256 + pad : base;
}

}  // extern "C"
