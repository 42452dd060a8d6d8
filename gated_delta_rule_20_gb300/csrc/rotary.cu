// rotary.cu -- rotary positions of q and k.
//
//     theta = position * inv_freq[i]:   (a, b) -> amplitude (a cos - b sin, b cos + a sin)
//
// on channel pairs (i, i + R/2) or (2i, 2i + 1) of the first R channels; the rest is copied.
//
// The angle is kept in turns, as a 64-bit binary fraction of one: f = inv_freq / 2 pi mod 1, and position * f wraps
// around as whole turns do.  That product is exact, so that far positions keep the accuracy of near ones: the angle's
// error is that of f, 1.5 * 2^-64 of a turn at the most, times the position, where an fp32 product loses 2^-24 of the
// angle itself (a radian at position 10^7).  (Frequencies above 1 radian, which no model has, take whole turns out of the 64
// bits of 2 / pi: their f is off by as many times as much.)
//
// Bound by bytes: a row is read and written once.  A thread takes one piece of a token's head (16 bytes, or two of them half
// the turned channels apart), makes that piece's sines and cosines, and goes through the heads with them: the trigonometry
// is done once a token, and a head costs two pointer additions.  Measured (bf16): 4 x 4096 tokens x 32 heads x 128 out of packed
// rows 45 us, 5.9 TB/s; 32768 tokens x 40 heads, 32 of 128 channels turned, 102 us, 6.6 TB/s of the 6.8 that a copy reaches.
#include <cuda_bf16.h>

#include "gdn_device.cuh"
#include "gdn_internal.h"
#include "sm100_ptx.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 128;
constexpr int kBlocks = 7;  // of an SM: 896 threads with 64 bytes each on their way (8 in fewer registers: spills)

struct RotaryTensor {
    const void* x;
    void* y;
    int64_t xs[3], ys[3];  // strides in elements: batch, head, token
    int heads;
};
struct RotaryArgs {
    RotaryTensor t[2];  // q, k
    const double* inv_freq;
    const void* positions;  // null: first + token
    long long pos_batch;    // its batch stride
    long long first;
    int B, S, R, D;
    int heads_thread;  // heads that a thread goes through, q's and k's counted through
    int rot_slots;     // threads of a token whose piece is turned
    int slots;         // and all of them (the rest copy)
    bool pos32, inverse;
    float amplitude;
};

// inv_freq / 2 pi mod 1 in units of 2^-64 of a turn.  2^64 / (2 pi) = kInv2Pi / 4 with kInv2Pi = 2^66 / (2 pi)
// rounded down; the double's 53 bits are multiplied as integers (a double's units are few on this chip).
constexpr unsigned long long kInv2Pi = 0xA2F9836E4E441529ull;  // 2 / pi in units of 2^-64
__device__ __forceinline__ unsigned long long turns_of(double f) {
    const unsigned long long bits = (unsigned long long)__double_as_longlong(f);
    const int e = (int)((bits >> 52) & 0x7ff);
    if (e == 0 || e == 0x7ff) return 0;  // zero (and below 2^-1022); infinities and NaN turn nothing
    // f = m 2^(e - 1023 - 63), m in [2^63, 2^64);  turns = f (2 / pi) / 4
    const unsigned long long m = (bits << 11) | (1ull << 63);
    const unsigned long long hi = __umul64hi(m, kInv2Pi), lo = m * kInv2Pi;  // m (2 / pi) 2^64
    const int sh = e - 1024;  // turns 2^64 = (hi : lo) 2^(e - 1023 - 63 - 2), its integer part from hi on at e = 1024
    unsigned long long t;
    if (sh >= 0)
        t = sh < 64 ? (sh ? (hi << sh) | (lo >> (64 - sh)) : hi) : sh < 128 ? lo << (sh - 64) : 0;
    else
        t = sh > -64 ? hi >> -sh : 0;
    return (long long)bits < 0 ? 0ull - t : t;
}

template <typename T, int V>
struct alignas(sizeof(T) * V) Piece {
    T e[V];
};

// 16-byte pieces are read and written once and marked so (ld.cs, st.cs: 45 us instead of 54 for 4 x 4096 tokens x 32 heads).
template <typename P, typename T>
__device__ __forceinline__ P load_piece(const T* from) {
    P r;
    if constexpr (sizeof(P) == 16)
        *reinterpret_cast<uint4*>(&r) = __ldcs(reinterpret_cast<const uint4*>(from));
    else
        r = *reinterpret_cast<const P*>(from);
    return r;
}
template <typename P, typename T>
__device__ __forceinline__ void store_piece(T* to, const P& x) {
    if constexpr (sizeof(P) == 16)
        __stcs(reinterpret_cast<uint4*>(to), *reinterpret_cast<const uint4*>(&x));
    else
        *reinterpret_cast<P*>(to) = x;
}

// V elements an access.  Half layout: two accesses a thread and head, `apart` channels apart.  Interleaved: one piece of V
// elements (V = 1: the pair's two), so that the threads of a token, turning and copying, read its row as it lies.
template <typename T, int V, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, kBlocks) rotary_kernel(const __grid_constant__ RotaryArgs a) {
    using P = Piece<T, V>;
    constexpr bool kOne = kInterleaved && V > 1;                      // one access a thread and head where it turns
    constexpr int kPairs = kInterleaved ? (V > 1 ? V / 2 : 1) : V;    // pairs of a thread
    constexpr int kUnroll = kOne ? 4 : 2;                             // heads on their way
    const int id = blockIdx.x * kThreads + threadIdx.x, token = id / a.slots, slot = id - token * a.slots;
    if (token >= a.B * a.S) return;
    const int b = token / a.S, s = token - b * a.S, half = a.R / 2;
    const bool turn = slot < a.rot_slots;
    // the thread's first channel, how far its second piece is, and whether it has one
    int c, apart;
    bool two = true;
    if (turn) {
        c = slot * (kOne ? V : kInterleaved ? 2 : V);
        apart = kInterleaved ? 1 : half;
        two = !kOne;
    } else {
        const int copies = a.slots - a.rot_slots;
        c = a.R + (slot - a.rot_slots) * V;
        apart = copies * V;
        two = !kOne && c + apart < a.D;
    }
    ptx::griddep_wait();
    float cs[kPairs], sn[kPairs];
    if (turn) {
        long long pos = a.first + s;
        if (a.positions) {
            const long long at = b * a.pos_batch + s;
            pos = a.pos32 ? (long long)static_cast<const int32_t*>(a.positions)[at]
                          : static_cast<const long long*>(a.positions)[at];
        }
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            const unsigned long long f = turns_of(a.inv_freq[slot * kPairs + i]);
            const long long angle = (long long)((unsigned long long)pos * f);
            float x, y;
            sincospif(__ll2float_rn(angle) * 0x1p-63f, &x, &y);  // half turns in [-1, 1]
            sn[i] = a.amplitude * (a.inverse ? -x : x);
            cs[i] = a.amplitude * y;
        }
    }
    const int lo = blockIdx.y * a.heads_thread, hi = min(lo + a.heads_thread, a.t[0].heads + a.t[1].heads);
#pragma unroll 1
    for (int w = 0; w < 2; ++w) {
        const RotaryTensor& t = a.t[w];
        const int before = w ? a.t[0].heads : 0, h0 = max(lo, before), h1 = min(hi, before + t.heads);
        if (h0 >= h1) continue;
        const T* x = static_cast<const T*>(t.x) + b * t.xs[0] + (h0 - before) * t.xs[1] + s * t.xs[2] + c;
        T* y = static_cast<T*>(t.y) + b * t.ys[0] + (h0 - before) * t.ys[1] + s * t.ys[2] + c;
        const long long dx = t.xs[1], dy = t.ys[1];
#pragma unroll 1
        for (int h = h0; h < h1; h += kUnroll, x += kUnroll * dx, y += kUnroll * dy) {
            P p[kUnroll], q[kOne ? 1 : kUnroll];
            const int n = h1 - h;
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                if (u < n) {
                    p[u] = load_piece<P>(x + u * dx);
                    if (!kOne && two) q[u] = load_piece<P>(x + u * dx + apart);
                }
            if (turn) {
#pragma unroll
                for (int u = 0; u < kUnroll; ++u)
#pragma unroll
                    for (int i = 0; i < kPairs; ++i) {
                        T& ea = p[u].e[kOne ? 2 * i : i];
                        T& eb = kOne ? p[u].e[(2 * i + 1) % V] : q[kOne ? 0 : u].e[kOne ? 0 : i];
                        const float fa = to_f32(ea), fb = to_f32(eb);
                        ea = from_f32<T>(fa * cs[i] - fb * sn[i]);
                        eb = from_f32<T>(fb * cs[i] + fa * sn[i]);
                    }
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                if (u < n) {
                    store_piece(y + u * dy, p[u]);
                    if (!kOne && two) store_piece(y + u * dy + apart, q[u]);
                }
        }
    }
    ptx::griddep_launch_dependents();
}

template <typename T, int V, bool kInterleaved>
cudaError_t launch(RotaryArgs a, int sms, cudaStream_t stream) {
    a.rot_slots = a.R / 2 / (kInterleaved ? (V > 1 ? V / 2 : 1) : V);
    const bool copies = a.t[0].x != a.t[0].y || (a.t[1].heads && a.t[1].x != a.t[1].y);
    a.slots = a.rot_slots + (!copies ? 0 : kInterleaved && V > 1 ? (a.D - a.R) / V : ((a.D - a.R) / V + 1) / 2);
    // heads of a thread: all, so that its sines serve them all, unless that leaves an SM fewer than 1024 threads; then
    // half as many, down to one or to the most parts that a grid has
    constexpr int kMostParts = 65535;
    const int heads = a.t[0].heads + a.t[1].heads;
    const long long threads = (long long)a.B * a.S * a.slots;
    a.heads_thread = heads;
    const auto parts = [&](int each) { return (heads + each - 1) / each; };
    while (a.heads_thread > 1 && threads * parts(a.heads_thread) < 1024ll * sms && parts((a.heads_thread + 1) / 2) <= kMostParts)
        a.heads_thread = (a.heads_thread + 1) / 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((threads + kThreads - 1) / kThreads), (unsigned)parts(a.heads_thread));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rotary_kernel<T, V, kInterleaved>, a);
}

template <typename T, bool kInterleaved>
cudaError_t launch_width(const RotaryArgs& a, int v, int sms, cudaStream_t stream) {
    if constexpr (sizeof(T) == 2)
        if (v == 8) return launch<T, 8, kInterleaved>(a, sms, stream);
    if (v >= 4) return launch<T, 4, kInterleaved>(a, sms, stream);
    if (v == 2) return launch<T, 2, kInterleaved>(a, sms, stream);
    return launch<T, 1, kInterleaved>(a, sms, stream);
}

// Elements from the lowest to behind the highest that the strides reach.
long long extent(const gdn_rotary_dims* d, int64_t heads, const int64_t* st) {
    return (d->B - 1) * st[0] + (heads - 1) * st[1] + (d->S - 1) * st[2] + d->D;
}

// Whether rows of D elements at these strides lie over one another: each stride has to pass all that the
// smaller ones reach.
bool rows_meet(const int64_t* sizes, const int64_t* st, int64_t D) {
    bool done[3] = {};
    long long reach = D;
    for (int n = 0; n < 3; ++n) {
        int least = -1;
        for (int j = 0; j < 3; ++j)
            if (!done[j] && sizes[j] > 1 && (least < 0 || st[j] < st[least])) least = j;
        if (least < 0) return false;
        if (st[least] < reach) return true;
        reach += (sizes[least] - 1) * st[least];
        done[least] = true;
    }
    return false;
}

// Whether rows a and b (D elements each) share no memory though what they span does: there is a period that all longer
// strides of both are multiples of, and in it what the shorter ones of a reach ends before b's begins, and the other way
// round.  (q and k in packed rows: the period is a token's stride, a head's, or a batch's.)
bool apart(const void* a, const int64_t* na, const int64_t* sa, const void* b, const int64_t* nb, const int64_t* sb, int64_t D,
           int el) {
    const int64_t from = (int64_t)(reinterpret_cast<intptr_t>(b) - reinterpret_cast<intptr_t>(a)) / el;
    for (int c = 0; c < 6; ++c) {
        const int64_t period = c < 3 ? sa[c] : sb[c - 3];
        if (period == 0) continue;
        const auto reach = [&](const int64_t* n, const int64_t* st) {  // -1: a longer stride is not a multiple
            int64_t r = D;
            for (int j = 0; j < 3; ++j) {
                if (st[j] < period)
                    r += (n[j] - 1) * st[j];
                else if (st[j] % period)
                    return (int64_t)-1;
            }
            return r;
        };
        const int64_t ra = reach(na, sa), rb = reach(nb, sb), at = (from % period + period) % period;
        if (ra > 0 && rb > 0 && at >= ra && at + rb <= period) return true;
    }
    return false;
}

}  // namespace
}  // namespace gdn

extern "C" gdn_status gdn_rotary(const void* q, const void* k, const double* inv_freq, const void* positions, void* q_out,
                                 void* k_out, const gdn_rotary_dims* d, gdn_stream_t stream) {
    using namespace gdn;
    if (!d) return GDN_ERR_NULL;
    if (d->dtype != GDN_F32 && d->dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
    constexpr uint32_t kFlags = GDN_ROTARY_INTERLEAVED | GDN_ROTARY_INVERSE | GDN_ROTARY_POSITIONS_I32;
    if (d->flags & ~kFlags) return GDN_ERR_UNSUPPORTED;
    if (d->B < 0 || d->S < 0 || d->Hq < 0 || d->Hk < 0 || d->D < 1 || d->R < 2 || d->R > d->D || d->R % 2 ||
        d->D > GDN_ROTARY_MAX_D || d->Hq > 65536 || d->Hk > 65536)
        return GDN_ERR_DIMS;
    // (a thread a piece of a token's channels, counted in 32 bits)
    if (d->B > INT32_MAX || d->S > INT32_MAX || d->B * d->S > (INT32_MAX - 4096) / d->D) return GDN_ERR_DIMS;
    if (d->B == 0 || d->S == 0 || d->Hq + d->Hk == 0) return GDN_OK;
    if (!inv_freq || (d->Hq && (!q || !q_out)) || (d->Hk && (!k || !k_out))) return GDN_ERR_NULL;
    const int el = d->dtype == GDN_BF16 ? 2 : 4;
    constexpr int64_t kSpan = int64_t(1) << 56;  // elements that a dim's rows may lie apart (byte counts stay within 64 bits)
    const bool i32 = (d->flags & GDN_ROTARY_POSITIONS_I32) != 0;
    if ((reinterpret_cast<uintptr_t>(inv_freq) & 7) || (reinterpret_cast<uintptr_t>(positions) & (i32 ? 3 : 7)))
        return GDN_ERR_ALIGN;
    RotaryArgs a{};
    const bool inter = (d->flags & GDN_ROTARY_INTERLEAVED) != 0;
    // elements of an access: the most that the pointers, the strides and the channel counts are multiples of
    uint64_t odd = (inter ? (uint64_t)d->R : (uint64_t)d->R / 2) | (uint64_t)(d->D - d->R);
    const void* xs[2] = {q, k};
    void* ys[2] = {q_out, k_out};
    const int64_t* xst[2] = {d->q_strides, d->k_strides};
    const int64_t* yst[2] = {d->q_out_strides, d->k_out_strides};
    const int64_t heads[2] = {d->Hq, d->Hk}, sizes[2][3] = {{d->B, d->Hq, d->S}, {d->B, d->Hk, d->S}};
    long long nx[2], ny[2];
    bool in_place[2];
    if (d->position_stride < 0 || (d->B > 1 && d->position_stride > kSpan / (d->B - 1))) return GDN_ERR_DIMS;
    const long long np = ((d->B - 1) * d->position_stride + d->S) * (i32 ? 4 : 8);
    for (int i = 0; i < 2; ++i) {
        a.t[i].heads = (int)heads[i];
        if (!heads[i]) continue;
        const uintptr_t px = reinterpret_cast<uintptr_t>(xs[i]), py = reinterpret_cast<uintptr_t>(ys[i]);
        if ((px | py) & (el - 1)) return GDN_ERR_ALIGN;
        a.t[i].x = xs[i];
        a.t[i].y = ys[i];
        bool same = true;
        for (int j = 0; j < 3; ++j) {
            const bool used = sizes[i][j] > 1;  // a stride that is never taken may be anything
            if (xst[i][j] < 0 || yst[i][j] < 0) return GDN_ERR_DIMS;
            if (used && (xst[i][j] > kSpan / (sizes[i][j] - 1) || yst[i][j] > kSpan / (sizes[i][j] - 1))) return GDN_ERR_DIMS;
            a.t[i].xs[j] = used ? xst[i][j] : 0;
            a.t[i].ys[j] = used ? yst[i][j] : 0;
            odd |= (uint64_t)a.t[i].xs[j] | (uint64_t)a.t[i].ys[j];
            same = same && a.t[i].xs[j] == a.t[i].ys[j];
        }
        if (rows_meet(sizes[i], a.t[i].ys, d->D)) return GDN_ERR_DIMS;
        odd |= (px | py) / el;
        nx[i] = extent(d, heads[i], a.t[i].xs) * el;
        ny[i] = extent(d, heads[i], a.t[i].ys) * el;
        in_place[i] = px == py && same;
        if (overlap(ys[i], ny[i], inv_freq, d->R * 4) || overlap(ys[i], ny[i], positions, np)) return GDN_ERR_UNSUPPORTED;
    }
    // an output shares no memory with the other one, nor with an input but its own in place
    for (int i = 0; i < 2; ++i) {
        for (int j = 0; j < 2; ++j) {
            if (!heads[i] || !heads[j]) continue;
            if (!(i == j && in_place[i]) && overlap(ys[i], ny[i], xs[j], nx[j]) &&
                !apart(ys[i], sizes[i], a.t[i].ys, xs[j], sizes[j], a.t[j].xs, d->D, el))
                return GDN_ERR_UNSUPPORTED;
            if (i < j && overlap(ys[i], ny[i], ys[j], ny[j]) &&
                !apart(ys[i], sizes[i], a.t[i].ys, ys[j], sizes[j], a.t[j].ys, d->D, el))
                return GDN_ERR_UNSUPPORTED;
        }
    }
    int v = 16 / el;
    while (v > 1 && odd % v) v /= 2;
    a.inv_freq = inv_freq;
    a.positions = positions;
    a.pos_batch = d->position_stride;
    a.first = d->first_position;
    a.B = (int)d->B;
    a.S = (int)d->S;
    a.R = (int)d->R;
    a.D = (int)d->D;
    a.pos32 = i32;
    a.inverse = (d->flags & GDN_ROTARY_INVERSE) != 0;
    a.amplitude = d->amplitude;
    int dev = 0, sms = 0;
    const gdn_status s = current_device_sms(&dev, &sms);
    if (s != GDN_OK) return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (d->dtype == GDN_BF16)
        e = inter ? launch_width<__nv_bfloat16, true>(a, v, sms, st) : launch_width<__nv_bfloat16, false>(a, v, sms, st);
    else
        e = inter ? launch_width<float, true>(a, v, sms, st) : launch_width<float, false>(a, v, sms, st);
    if (e == cudaSuccess) return GDN_OK;
    (void)cudaGetLastError();
    return GDN_ERR_CUDA;
}
