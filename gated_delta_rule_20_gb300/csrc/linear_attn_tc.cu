// linear_attn_tc.cu -- prefill of linear attention with a decay for each head on the tensor cores (bf16).
//
// Chunks of 128 tokens, c_i the sum of the log-decays of a chunk up to token i, S the state in front of it:
//     o_i = scale ( e^{c_i} q_i S + sum_{j <= i} e^{c_i - c_j} (q_i . k_j) v_j )
//     S'  = e^{c_128} S + sum_j k_j (e^{c_128 - c_j} v_j)^T
//
// Products, 128 x 128 x 128 each (Dk = Dv = 128), all issued by one thread in this order a chunk:
//   QK   scores[i, j]        A = Q, B = K                  (shared memory)
//   QS   O = Q S             A = Q, B = S^T in bf16        (shared memory)
//   KV   X[dv, dk] = (e^. V)^T K in three parts: A = part of (e^. V)^T (TMEM), B = K
//   PV   O += P V            A = P (TMEM, over the scores), B = V
// The state is fp32: X is added to it on the FMA units, and e^. v is cut into three bf16 parts that add up to its 24
// bits, so that the state is as exact as an fp32 recurrence's.  O sums both terms in one accumulator: a row is kept divided
// by e^{m_i}, m_i = max(c_i, -64), which is 1 in front of Q S, and its scores are e^{c_i - c_j - m_i}: at most
// e^64, inside bf16's range.  The output's last product is scale e^{m_i}.  (Rows past c_i = -64 so keep e^-64 of S instead of
// less: 1.6e-28.)
//
// Exponents.  c is summed within blocks of 32 tokens: no difference of two large sums is ever taken.  With block sums T_b,
// a score off the diagonal blocks takes e^{c_i - R} e^{R - c_j}, R the end of j's block, a factor of its row and one of its
// column, and only the 32 x 32 diagonal blocks take an exponential an element.
//
// Roles (768 threads): 4 warps turn scores into P, 8 hold the state (a thread: 64 rows of a column dv in fp32 registers), 4
// make the parts of e^. V, 4 write the outputs; one warp each for TMA, the products and the decays.  A CTA walks its
// sequences' chunks without a break: the pipeline runs through from one sequence to the next.
#include <cuda_bf16.h>

#include <atomic>

#include "gdn_device.cuh"
#include "gdn_internal.h"
#include "linear_attn.h"
#include "sm100_ptx.cuh"

namespace gdn {
namespace {

using namespace ptx;

constexpr int kC = 128;  // tokens of a chunk
constexpr int kThreads = 768;
constexpr uint32_t kHalf = 16384, kTile = 2 * kHalf;  // 128 rows x 64 channels, and 128
constexpr uint32_t kOffQ = 0, kOffK = 2 * kTile, kOffV = 4 * kTile, kOffS = 6 * kTile, kOffSmall = 7 * kTile;
constexpr int kSub = 16, kSlots = 5;  // tokens a slot of the parts of e^. V, and slots
// TMEM columns: scores (P over their first 64), O, X, the parts' slots of 3 x 8
constexpr uint32_t kColP = 0, kColO = 128, kColX = 256, kColV = 384, kSlotCols = 24;
constexpr float kMinRow = -64.f * kLog2e;  // least m_i, in powers of two

// Registers a thread of each role; what the block is launched with covers their sum (launch checks it).
constexpr int kRegsP = 80, kRegsS = 120, kRegsV = 64, kRegsO = 48, kRegsCtl = 48;
constexpr int kRegsSum = (kRegsP + 2 * kRegsS + kRegsV + kRegsO + kRegsCtl) * 128;

struct Small {
    float c[2][kC];      // sums of log2-decays within blocks of 32
    float h[2][kC];      // e^(the log-decays behind the token in its block)
    float T[2][4];       // the blocks' log2-decays
    float w[2][4];       // e^(the log-decays behind the block)
    float total[2];      // e^(the chunk's)
    uint64_t kvfull[2], kvfree[2], qfull[2], qfree[2], decfull[2], decfree[2];
    uint64_t vfull[kSlots], vfree[kSlots];
    uint64_t sfull, xfull, qkfull, pfull, ofull, ofree, drain;
    uint32_t tmem;
    int abort;
};
constexpr uint32_t kSmem = kOffSmall + sizeof(Small);
static_assert(kSmem <= 232448, "shared memory of a CTA");

template <int N>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// 16 lanes from the address's lane on, 8 columns (.16x128b, 2 repeats): r[2k], r[2k + 1] = column 4 k + t % 4 of
// lanes t / 4 and t / 4 + 8.
__device__ __forceinline__ void tmem_st16x128_x2(uint32_t taddr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(r0), "r"(r1), "r"(r2),
                 "r"(r3)
                 : "memory");
}

// 32 lanes x 16 consecutive columns.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
        : "r"(taddr));
}

// Waits as ptx::mbar_wait_or_abort's, but inline: a kernel that shares out its registers cannot call functions.
__device__ __forceinline__ bool wait_inline(uint64_t* bar, uint32_t parity, volatile int* abort) {
    if (mbar_try_wait(bar, parity)) return true;
    uint64_t t0 = 0;
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 15u) == 0) {
            if (abort && *abort) return false;
            const uint64_t t = globaltimer_ns();
            if (t0 == 0) t0 = t;
            if (t - t0 > 1000000000ull) {
                if (abort) *abort = 1;
                return false;
            }
        }
    }
}
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort) {
    return __all_sync(0xffffffffu, wait_inline(bar, parity, abort));
}
// What is in flight when a role gives up: waited for with the time limit alone.
__device__ __forceinline__ void wait_drain(uint64_t* bar, uint32_t parity) { (void)wait_inline(bar, parity, nullptr); }

struct Chunks {  // the walk over a CTA's items: (segment, head), and the chunks of each
    int seg, b, h, bh, t0, t1, n;
};
__device__ __forceinline__ Chunks chunks_of(const LinearAttn& p, const LinearAttnSplit& s, int item) {
    Chunks c;
    const int heads = p.B * p.Hv;
    c.seg = item / heads;
    c.bh = item - c.seg * heads;
    c.b = c.bh / p.Hv;
    c.h = c.bh - c.b * p.Hv;
    int len = p.S;
    if (p.lengths) len = max(0, min(p.S, p.lengths[c.b]));
    c.t0 = s.P > 1 ? c.seg * s.len : 0;
    c.t1 = s.P > 1 ? min(len, c.t0 + s.len) : len;
    c.n = c.t1 > c.t0 ? (c.t1 - c.t0 + kC - 1) / kC : 0;
    return c;
}

// kStatesOnly: the first pass of a split (end states and decays of segments 0 .. P - 2; only KV is formed).
template <bool kStatesOnly>
__global__ void __launch_bounds__(kThreads, 1)
    linear_attn_tc_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                          const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap to,
                          const __grid_constant__ LinearAttn p, const __grid_constant__ LinearAttnSplit split,
                          int32_t* status) {
    extern __shared__ __align__(1024) uint8_t sm[];
    Small& sh = *reinterpret_cast<Small*>(sm + kOffSmall);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = warp & 3;
    volatile int* abort = &sh.abort;
    const uint32_t sbase = smem_u32(sm);
    const long long heads = p.B * p.Hv;
    const int items = (int)heads * (kStatesOnly ? split.P - 1 : split.P);

    if (tid == 0) {
        // (the tiles' descriptors need 1024-byte alignment, which a launch without static shared memory has)
        sh.abort = (sbase & 1023u) ? 1 : 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.kvfull[i], 1);
            mbar_init(&sh.kvfree[i], 1);
            mbar_init(&sh.qfull[i], 1);
            mbar_init(&sh.qfree[i], 1);
            mbar_init(&sh.decfull[i], 32);
            mbar_init(&sh.decfree[i], kStatesOnly ? 384 : 640);
        }
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&sh.vfull[i], 128);
            mbar_init(&sh.vfree[i], 1);
        }
        mbar_init(&sh.sfull, 256);
        mbar_init(&sh.xfull, 1);
        mbar_init(&sh.qkfull, 1);
        mbar_init(&sh.pfull, 128);
        mbar_init(&sh.ofull, 1);
        mbar_init(&sh.ofree, 128);
        mbar_init(&sh.drain, 1);
        fence_mbar_init();
    }
    if (warp == 21) tmem_alloc(&sh.tmem, 512);
    if (warp == 20 && elect_one()) {
        tma_prefetch_desc(&tk);
        tma_prefetch_desc(&tv);
        if (!kStatesOnly) {
            tma_prefetch_desc(&tq);
            tma_prefetch_desc(&to);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    const uint32_t tq4 = tmem + ((uint32_t)(quad * 32) << 16);  // this warp's lanes
    griddep_wait();

    int cn = 0;  // chunks so far, over all items
    if (warp < 4) {
        // ------------------------------------------------------------ scores -> P
        if (!kStatesOnly) {
            for (int item = blockIdx.x; item < items; item += gridDim.x) {
                const Chunks w = chunks_of(p, split, item);
                bool fail = false;
                for (int c = 0; c < w.n; ++c, ++cn) {
                    const int s = cn & 1;
                    fail = !wait_warp(&sh.decfull[s], (cn >> 1) & 1, abort);
                    if (fail) break;
                    const int a = quad;
                    float R = 0.f;
                    for (int m = 0; m < a; ++m) R += sh.T[s][m];
                    const float ci = sh.c[s][32 * a + lane], shift = ci - fmaxf(R + ci, kMinRow);
                    float u[3];  // off the diagonal: 2^(c_i - m_i - (end of block b))
#pragma unroll
                    for (int b = 0; b < 3; ++b) {
                        float x = shift;
                        for (int m = b + 1; m < a; ++m) x += sh.T[s][m];
                        u[b] = exp2_approx(x);
                    }
                    fail = !wait_warp(&sh.qkfull, cn & 1, abort);
                    if (fail) break;
                    tc_fence_after();
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        uint32_t pk[16];
                        if (b > a) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) pk[j] = 0;
                        } else {
                            float x[32];
                            tmem_ld32(tq4 + kColP + 32 * b, x);
                            tmem_wait_ld();
                            if (b < a) {
                                const float ub = u[b < 3 ? b : 0];
#pragma unroll
                                for (int j = 0; j < 32; j += 4) {
                                    const float4 h = *reinterpret_cast<const float4*>(&sh.h[s][32 * b + j]);
                                    pk[j / 2] = pack_bf16x2(x[j] * (ub * h.x), x[j + 1] * (ub * h.y));
                                    pk[j / 2 + 1] = pack_bf16x2(x[j + 2] * (ub * h.z), x[j + 3] * (ub * h.w));
                                }
                            } else {
#pragma unroll
                                for (int j = 0; j < 32; j += 4) {
                                    const float4 cj = *reinterpret_cast<const float4*>(&sh.c[s][32 * b + j]);
                                    const float y0 = j <= lane ? x[j] * exp2_approx(shift - cj.x) : 0.f;
                                    const float y1 = j + 1 <= lane ? x[j + 1] * exp2_approx(shift - cj.y) : 0.f;
                                    const float y2 = j + 2 <= lane ? x[j + 2] * exp2_approx(shift - cj.z) : 0.f;
                                    const float y3 = j + 3 <= lane ? x[j + 3] * exp2_approx(shift - cj.w) : 0.f;
                                    pk[j / 2] = pack_bf16x2(y0, y1);
                                    pk[j / 2 + 1] = pack_bf16x2(y2, y3);
                                }
                            }
                        }
                        // (over score columns that this warp has read: 16 b + 15 < 32 (b + 1))
                        tmem_st16u(tq4 + kColP + 16 * b, pk);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    mbar_arrive(&sh.pfull);
                    mbar_arrive(&sh.decfree[s]);
                }
                if (fail) break;
            }
        }
    } else if (warp < 12) {
        // ------------------------------------------------------------ the state: thread = 64 rows of column dv
        regs_inc<kRegsS>();
        const int dv = quad * 32 + lane, half = (warp - 4) >> 2;
        const int rows = dv < p.Dv ? min(64, p.Dk - 64 * half) : 0;  // of the 64 that are there (<= 0: none)
        const long long ns = (long long)p.Dk * p.Dv;
        float S[64];
        bool fail = false;
        for (int item = blockIdx.x; item < items && !fail; item += gridDim.x) {
            const Chunks w = chunks_of(p, split, item);
            int pitch = p.Dv;
            asm volatile("" : "+r"(pitch));  // (64 rows' offsets are not kept in registers over the chunks)
            const int first = 64 * half * pitch + dv;
            const float* src = p.state_in ? p.state_in + w.bh * ns : nullptr;
            if (!kStatesOnly && split.P > 1) src = split.parts + (w.seg ? w.bh : (split.P - 1) * heads + w.bh) * ns;
            if (kStatesOnly && w.seg) src = nullptr;
#pragma unroll
            for (int i = 0; i < 64; ++i) {
                S[i] = src && i < rows ? src[first + i * pitch] : 0.f;
                if (i % 16 == 15) asm volatile("" ::: "memory");  // (no more loads' addresses at once)
            }
            if (!kStatesOnly && split.P > 1) {
                for (int m = 1; m < w.seg; ++m) {
                    const float f = split.decays[m * heads + w.bh];
                    const float* x = split.parts + (m * heads + w.bh) * ns;
#pragma unroll
                    for (int i = 0; i < 64; ++i) {
                        if (i < rows) S[i] = fmaf(f, S[i], x[first + i * pitch]);
                        if (i % 16 == 15) asm volatile("" ::: "memory");
                    }
                }
            }
            if (kStatesOnly && w.seg == 0) {  // the copy of state_in
                float* x = split.parts + ((split.P - 1) * heads + w.bh) * ns;
#pragma unroll
                for (int i = 0; i < 64; ++i) {
                    if (i < rows) x[first + i * pitch] = S[i];
                    if (i % 16 == 15) asm volatile("" ::: "memory");
                }
            }
            float decay = 1.f;
            for (int c = 0; c < w.n; ++c, ++cn) {
                const int s = cn & 1;
                if (!kStatesOnly) {
                    // S^T in bf16, rows dv: the products that read the previous one are done (xfull)
#pragma unroll
                    for (int ch = 0; ch < 8; ++ch) {
                        const float* x = S + 8 * ch;
                        *reinterpret_cast<uint4*>(sm + kOffS + half * kHalf + sw128_offset(dv, ch * 16)) =
                            make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                       pack_bf16x2(x[6], x[7]));
                    }
                    fence_proxy_async_smem();
                }
                mbar_arrive(&sh.sfull);
                fail = !wait_warp(&sh.decfull[s], (cn >> 1) & 1, abort);
                if (fail) break;
                const float e = sh.total[s];
                decay *= e;
                fail = !wait_warp(&sh.xfull, cn & 1, abort);
                if (fail) break;
                tc_fence_after();
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    if (64 * half + 16 * b < p.Dk) {
                        float x[16];
                        tmem_ld16(tq4 + kColX + 64 * half + 16 * b, x);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) S[16 * b + i] = fmaf(e, S[16 * b + i], x[i]);
                    }
                }
                tc_fence_before();
                mbar_arrive(&sh.decfree[s]);
            }
            if (fail) break;
            float* dst = nullptr;
            if (kStatesOnly) {
                dst = split.parts + (w.seg * heads + w.bh) * ns;
                if (tid == 128) split.decays[w.seg * heads + w.bh] = decay;
            } else if (w.seg == split.P - 1) {
                dst = p.state_out + w.bh * ns;
            }
            if (dst) {
                asm volatile("" : "+r"(pitch));
#pragma unroll
                for (int i = 0; i < 64; ++i) {
                    if (i < rows) dst[first + i * pitch] = S[i];
                    if (i % 16 == 15) asm volatile("" ::: "memory");
                }
            }
        }
    } else if (warp < 16) {
        // ------------------------------------------------------------ parts of e^. V
        regs_dec<kRegsV>();
        int vi = 0;  // slots so far
        bool fail = false;
        for (int item = blockIdx.x; item < items && !fail; item += gridDim.x) {
            const Chunks w = chunks_of(p, split, item);
            for (int c = 0; c < w.n && !fail; ++c, ++cn) {
                const int s = cn & 1, n = min(kC, w.t1 - w.t0 - c * kC), subs = (n + kSub - 1) / kSub;
                fail = !wait_warp(&sh.decfull[s], (cn >> 1) & 1, abort) ||
                       !wait_warp(&sh.kvfull[s], (cn >> 1) & 1, abort);
                if (fail) break;
                uint8_t* vt = sm + kOffV + s * kTile;
                if (n < subs * kSub && p.lengths) {
                    // rows behind the last token in the last 16: whatever they hold is not multiplied, not even by zero.
                    // A warp clears the columns that it reads itself, of V and of K
                    const int rows = subs * kSub - n;
                    for (int i = lane; i < rows * 8; i += 32) {
                        const uint32_t at =
                            (quad >> 1) * kHalf + sw128_offset(n + (i >> 3), (quad & 1) * 64 + (i & 3) * 16);
                        *reinterpret_cast<uint4*>((i & 4 ? vt : sm + kOffK + s * kTile) + at) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                const uint32_t vh = smem_u32(vt) + (quad >> 1) * kHalf;
                for (int u = 0; u < subs; ++u, ++vi) {
                    const int slot = vi % kSlots, turn = vi / kSlots;
                    if (turn > 0) {
                        fail = !wait_warp(&sh.vfree[slot], (turn - 1) & 1, abort);
                        if (fail) break;
                    }
                    if (quad * 32 < p.Dv) {
                        tc_fence_after();
                        const float wb = sh.w[s][u >> 1];
                        uint32_t part[3][2][4];  // [part][8 tokens][8 columns dv]
#pragma unroll
                        for (int o = 0; o < 2; ++o) {
                            const int tok = u * kSub + o * 8;
                            uint32_t m[4];
                            ldmatrix_x4_trans(
                                vh + sw128_offset(tok + (lane & 7), (quad & 1) * 64 + (lane >> 3) * 16), m);
                            const float2 h = *reinterpret_cast<const float2*>(&sh.h[s][tok + 2 * (lane & 3)]);
                            const float d0 = h.x * wb, d1 = h.y * wb;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                float x0 = bf16lo_to_f32(m[i]) * d0, x1 = bf16hi_to_f32(m[i]) * d1;
#pragma unroll
                                for (int q = 0; q < 3; ++q) {
                                    const uint32_t r = pack_bf16x2(x0, x1);
                                    part[q][o][i] = r;
                                    x0 -= bf16lo_to_f32(r);
                                    x1 -= bf16hi_to_f32(r);
                                }
                            }
                        }
                        const uint32_t at = tq4 + kColV + slot * kSlotCols;
#pragma unroll
                        for (int q = 0; q < 3; ++q) {
                            tmem_st16x128_x2(at + 8 * q, part[q][0][0], part[q][0][1], part[q][1][0], part[q][1][1]);
                            tmem_st16x128_x2(at + 8 * q + (16u << 16), part[q][0][2], part[q][0][3], part[q][1][2],
                                             part[q][1][3]);
                        }
                        tmem_wait_st();
                        tc_fence_before();
                    }
                    mbar_arrive(&sh.vfull[slot]);
                }
                if (!fail) mbar_arrive(&sh.decfree[s]);
            }
        }
    } else if (warp < 20) {
        // ------------------------------------------------------------ outputs
        regs_dec<kRegsO>();
        if (!kStatesOnly) {
            const int r = quad * 32 + lane;
            bool stop = false;
            for (int item = blockIdx.x; item < items && !stop; item += gridDim.x) {
                const Chunks w = chunks_of(p, split, item);
                for (int c = 0; c < w.n; ++c, ++cn) {
                    const int s = cn & 1, t = w.t0 + c * kC, n = min(kC, w.t1 - t);
                    bool fail = !wait_warp(&sh.decfull[s], (cn >> 1) & 1, abort);
                    float f = 0.f;
                    if (!fail) {
                        float R = 0.f;
                        for (int m = 0; m < quad; ++m) R += sh.T[s][m];
                        f = p.scale * exp2_approx(fmaxf(R + sh.c[s][r], kMinRow));
                        fail = !wait_warp(&sh.ofull, cn & 1, abort);
                    }
                    if (named_bar_any(2, 128, fail)) {
                        stop = true;
                        break;
                    }
                    tc_fence_after();
                    // whole chunks and the end of the tensor by TMA, out of q's tile; rows that a length ends by themselves
                    const bool tma = n == kC || t + n == p.S;
                    uint8_t* tile = sm + kOffQ + s * kTile;
                    uint8_t* row = static_cast<uint8_t*>(p.out) + ((long long)w.bh * p.S + t + r) * (long long)p.Dv * 2;
#pragma unroll
                    for (int b = 0; b < 8; ++b) {
                        if (16 * b < p.Dv) {
                            float x[16];
                            tmem_ld16(tq4 + kColO + 16 * b, x);
                            tmem_wait_ld();
                            if (16 * (b + 1) >= p.Dv) {  // the last columns have been read
                                tc_fence_before();
                                mbar_arrive(&sh.ofree);
                            }
#pragma unroll
                            for (int ch = 0; ch < 2; ++ch) {
                                const float* y = x + 8 * ch;
                                const uint4 o = make_uint4(pack_bf16x2(f * y[0], f * y[1]), pack_bf16x2(f * y[2], f * y[3]),
                                                           pack_bf16x2(f * y[4], f * y[5]), pack_bf16x2(f * y[6], f * y[7]));
                                if (tma)
                                    *reinterpret_cast<uint4*>(tile + (b >> 2) * kHalf +
                                                              sw128_offset(r, (b & 3) * 32 + ch * 16)) = o;
                                else if (r < n && 16 * b + 8 * ch < p.Dv)
                                    *reinterpret_cast<uint4*>(row + 32 * b + 16 * ch) = o;
                            }
                        }
                    }
                    mbar_arrive(&sh.decfree[s]);
                    if (tma) {
                        fence_proxy_async_smem();
                        named_bar_sync(2, 128);
                    }
                    if (warp == 16 && elect_one()) {
                        if (tma) {
                            tma_store_3d(&to, tile, 0, t, w.bh);
                            if (p.Dv > 64) tma_store_3d(&to, tile + kHalf, 64, t, w.bh);
                            tma_store_commit();
                            tma_store_wait_read0();
                        }
                        mbar_arrive(&sh.qfree[s]);
                    }
                    __syncwarp();
                }
            }
            if (warp == 16) tma_store_wait_all0();
        }
    } else {
        regs_dec<kRegsCtl>();
        if (warp == 20) {
            // -------------------------------------------------------- TMA
            const uint32_t kb = p.Dk > 64 ? kTile : kHalf, vb = p.Dv > 64 ? kTile : kHalf;
            int kv_issued = 0, q_issued = 0;
            bool fail = false;
            for (int item = blockIdx.x; item < items && !fail; item += gridDim.x) {
                const Chunks w = chunks_of(p, split, item);
                const int bhk = w.b * p.Hk + w.h / (p.Hv / p.Hk);
                for (int c = 0; c < w.n; ++c, ++cn) {
                    const int s = cn & 1, t = w.t0 + c * kC;
                    if (cn >= 2) {
                        fail = !wait_warp(&sh.kvfree[s], ((cn >> 1) - 1) & 1, abort);
                        if (fail) break;
                    }
                    if (elect_one()) {
                        uint8_t* kt = sm + kOffK + s * kTile;
                        uint8_t* vt = sm + kOffV + s * kTile;
                        mbar_arrive_expect_tx(&sh.kvfull[s], kb + vb);
                        tma_load_3d(kt, &tk, &sh.kvfull[s], 0, t, bhk);
                        if (p.Dk > 64) tma_load_3d(kt + kHalf, &tk, &sh.kvfull[s], 64, t, bhk);
                        tma_load_3d(vt, &tv, &sh.kvfull[s], 0, t, w.bh);
                        if (p.Dv > 64) tma_load_3d(vt + kHalf, &tv, &sh.kvfull[s], 64, t, w.bh);
                    }
                    __syncwarp();
                    kv_issued = cn + 1;
                    if (!kStatesOnly) {
                        if (cn >= 2) {
                            fail = !wait_warp(&sh.qfree[s], ((cn >> 1) - 1) & 1, abort);
                            if (fail) break;
                        }
                        if (elect_one()) {
                            uint8_t* qt = sm + kOffQ + s * kTile;
                            mbar_arrive_expect_tx(&sh.qfull[s], kb);
                            tma_load_3d(qt, &tq, &sh.qfull[s], 0, t, bhk);
                            if (p.Dk > 64) tma_load_3d(qt + kHalf, &tq, &sh.qfull[s], 64, t, bhk);
                        }
                        __syncwarp();
                        q_issued = cn + 1;
                    }
                }
            }
            // every load has landed before the CTA ends (bounded)
            for (int i = max(0, kv_issued - 2); i < kv_issued; ++i) wait_drain(&sh.kvfull[i & 1], (i >> 1) & 1);
            for (int i = max(0, q_issued - 2); i < q_issued; ++i) wait_drain(&sh.qfull[i & 1], (i >> 1) & 1);
        } else if (warp == 21) {
            // -------------------------------------------------------- products
            const int Nk = (p.Dk + 15) & ~15, Nv = (p.Dv + 15) & ~15, ksteps = Nk / 16;
            constexpr uint32_t kIdQK = make_idesc_bf16(128, 128, 0, 0);
            const uint32_t id_qs = make_idesc_bf16(128, Nv, 0, 0), id_pv = make_idesc_bf16(128, Nv, 0, 1),
                           id_kv = make_idesc_bf16(128, Nk, 0, 1);
            int vi = 0, last = -1;  // (last: the last chunk with a commit to wait for)
            bool fail = false;
            const uint64_t ds = make_sdesc(sbase + kOffS, 16, 1024);
            for (int item = blockIdx.x; item < items && !fail; item += gridDim.x) {
                const Chunks w = chunks_of(p, split, item);
                for (int c = 0; c < w.n && !fail; ++c, ++cn) {
                    const int s = cn & 1, n = min(kC, w.t1 - w.t0 - c * kC), subs = (n + kSub - 1) / kSub;
                    const uint32_t kt = sbase + kOffK + s * kTile, vt = sbase + kOffV + s * kTile;
                    const uint64_t dq = make_sdesc(sbase + kOffQ + s * kTile, 16, 1024), dk = make_sdesc(kt, 16, 1024),
                                   dkm = make_sdesc(kt, kHalf, 1024), dvm = make_sdesc(vt, kHalf, 1024);
                    fail = !wait_warp(&sh.kvfull[s], (cn >> 1) & 1, abort);
                    if (fail) break;
                    if (!kStatesOnly) {
                        fail = !wait_warp(&sh.qfull[s], (cn >> 1) & 1, abort);
                        if (fail) break;
                        tc_fence_after();
                        if (elect_one()) {
                            for (int k = 0; k < ksteps; ++k) {
                                const uint32_t at = (k >> 2) * kHalf + (k & 3) * 32;
                                mma_bf16(tmem + kColP, sdesc_add(dq, at), sdesc_add(dk, at), kIdQK, k > 0);
                            }
                            mma_commit(&sh.qkfull);
                        }
                        __syncwarp();
                        fail = (cn > 0 && !wait_warp(&sh.ofree, (cn - 1) & 1, abort));
                        if (fail) break;
                    }
                    fail = !wait_warp(&sh.sfull, cn & 1, abort);
                    if (fail) break;
                    tc_fence_after();
                    if (!kStatesOnly && elect_one()) {
                        for (int k = 0; k < ksteps; ++k) {
                            const uint32_t at = (k >> 2) * kHalf + (k & 3) * 32;
                            mma_bf16(tmem + kColO, sdesc_add(dq, at), sdesc_add(ds, at), id_qs, k > 0);
                        }
                    }
                    __syncwarp();
                    for (int u = 0; u < subs; ++u, ++vi) {
                        const int slot = vi % kSlots;
                        fail = !wait_warp(&sh.vfull[slot], (vi / kSlots) & 1, abort);
                        if (fail) break;
                        tc_fence_after();
                        if (elect_one()) {
                            const uint32_t a = tmem + kColV + slot * kSlotCols;
                            const uint64_t b = sdesc_add(dkm, u * 2048);
                            mma_bf16_tmem_a(tmem + kColX, a, b, id_kv, u > 0);
                            mma_bf16_tmem_a(tmem + kColX, a + 8, b, id_kv, 1);
                            mma_bf16_tmem_a(tmem + kColX, a + 16, b, id_kv, 1);
                            mma_commit(&sh.vfree[slot]);
                            if (u == subs - 1) {
                                mma_commit(&sh.xfull);
                                if (kStatesOnly) mma_commit(&sh.kvfree[s]);
                            }
                        }
                        __syncwarp();
                    }
                    if (fail) break;
                    if (!kStatesOnly) {
                        fail = !wait_warp(&sh.pfull, cn & 1, abort);
                        if (fail) break;
                        tc_fence_after();
                        if (elect_one()) {
                            for (int k = 0; k < subs; ++k)
                                mma_bf16_tmem_a(tmem + kColO, tmem + kColP + 8 * k, sdesc_add(dvm, k * 2048), id_pv, 1);
                            mma_commit(&sh.ofull);
                            mma_commit(&sh.kvfree[s]);
                        }
                        __syncwarp();
                    }
                    last = cn;
                }
            }
            if (fail) {
                // products in flight end before the tensor memory is freed: a commit behind all of them (bounded).
                if (elect_one()) {
                    mma_commit(&sh.drain);
                    wait_drain(&sh.drain, 0);
                }
                __syncwarp();
            } else if (last >= 0) {
                wait_drain(&sh.kvfree[last & 1], (last >> 1) & 1);
            }
        } else if (warp == 22) {
            // -------------------------------------------------------- decays
            bool fail = false;
            for (int item = blockIdx.x; item < items && !fail; item += gridDim.x) {
                const Chunks w = chunks_of(p, split, item);
                const float* g = p.head_decay ? p.g_log + w.h : p.g_log + (long long)w.bh * p.S;
                for (int c = 0; c < w.n; ++c, ++cn) {
                    const int s = cn & 1, t = w.t0 + c * kC;
                    float x[4];
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const int tok = t + 32 * b + lane;
                        x[b] = 0.f;
                        if (tok < w.t1) x[b] = least_decay(p.head_decay ? *g : g[tok]);
                    }
                    if (cn >= 2) {
                        fail = !wait_warp(&sh.decfree[s], ((cn >> 1) - 1) & 1, abort);
                        if (fail) break;
                    }
                    float T[4], behind = 0.f;
#pragma unroll
                    for (int b = 3; b >= 0; --b) {
                        float up = x[b], down = x[b];
#pragma unroll
                        for (int o = 1; o < 32; o <<= 1) {
                            const float y = __shfl_up_sync(0xffffffffu, up, o), z = __shfl_down_sync(0xffffffffu, down, o);
                            if (lane >= o) up += y;
                            if (lane + o < 32) down += z;
                        }
                        const float after = __shfl_down_sync(0xffffffffu, down, 1);
                        sh.c[s][32 * b + lane] = kLog2e * up;
                        sh.h[s][32 * b + lane] = expf(lane < 31 ? after : 0.f);
                        T[b] = __shfl_sync(0xffffffffu, down, 0);
                        if (lane == 0) {
                            sh.T[s][b] = kLog2e * T[b];
                            sh.w[s][b] = expf(behind);
                        }
                        behind += T[b];
                    }
                    if (lane == 0) sh.total[s] = expf(behind);
                    mbar_arrive(&sh.decfull[s]);
                }
            }
        }
    }
    griddep_launch_dependents();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 21) {
        tmem_relinquish();
        tmem_dealloc(tmem, 512);
    }
    if (tid == 0 && sh.abort && status) atomicExch(status, (int32_t)GDN_ERR_TIMEOUT);
}

// ------------------------------------------------------------------ host side
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static const EncodeTiledFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        return cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
                       q == cudaDriverEntryPointSuccess
                   ? reinterpret_cast<EncodeTiledFn>(p)
                   : nullptr;
    }();
    return fn;
}

// [heads, S, D] bf16 in boxes of 128 tokens x 64 channels; what lies outside reads as zeros and is not written.
bool encode(CUtensorMap* map, const void* ptr, long long heads, int S, int D) {
    const EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)S, (cuuint64_t)heads};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)S * D * 2};
    cuuint32_t box[3] = {64, kC, 1}, estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kStatesOnly>
gdn_status launch(const CUtensorMap (&m)[4], const LinearAttn& p, const LinearAttnSplit& s, int dev, int sms,
                  int32_t* status, cudaStream_t stream) {
    auto* kernel = linear_attn_tc_kernel<kStatesOnly>;
    static const int regs = [&] {
        cudaFuncAttributes a{};
        return cudaFuncGetAttributes(&a, kernel) == cudaSuccess ? a.numRegs : 0;
    }();
    static std::atomic<bool> allowed[kMaxDevices];
    // the roles' registers come out of what the block is launched with: short of that they would wait for ever
    if (regs * kThreads < kRegsSum) return GDN_ERR_CUDA;
    if (allow_smem(kernel, (int)kSmem, allowed, dev) != cudaSuccess) return GDN_ERR_CUDA;
    const long long items = (long long)p.B * p.Hv * (kStatesOnly ? s.P - 1 : s.P);
    if (items > INT32_MAX - sms) return GDN_ERR_DIMS;  // (items are counted in 32 bits)
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(items < sms ? items : sms));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, m[0], m[1], m[2], m[3], p, s, status) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace

bool linear_attn_tc_supported(const LinearAttn& p) {
    const auto off = [](const void* a) { return (reinterpret_cast<uintptr_t>(a) & 15u) != 0; };
    return p.bf16 && p.Dk % 8 == 0 && p.Dv % 8 == 0 && !off(p.q) && !off(p.k) && !off(p.v) && !off(p.out);
}

gdn_status launch_linear_attn_tc(const LinearAttn& p, const LinearAttnSplit& s, int dev, int sms, int32_t* status,
                                 cudaStream_t stream) {
    CUtensorMap m[4];
    const long long hk = (long long)p.B * p.Hk, hv = (long long)p.B * p.Hv;
    if (!encode(&m[0], p.q, hk, p.S, p.Dk) || !encode(&m[1], p.k, hk, p.S, p.Dk) || !encode(&m[2], p.v, hv, p.S, p.Dv) ||
        !encode(&m[3], p.out, hv, p.S, p.Dv))
        return GDN_ERR_CUDA;
    if (s.P > 1) {
        const gdn_status e = launch<true>(m, p, s, dev, sms, status, stream);
        if (e != GDN_OK) return e;
    }
    return launch<false>(m, p, s, dev, sms, status, stream);
}

}  // namespace gdn
