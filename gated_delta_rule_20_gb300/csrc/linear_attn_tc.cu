// linear_attn_tc.cu -- prefill of linear attention with a decay for each head on the tensor cores (bf16).
//
// Chunks of 128 tokens, c_i the sum of the log-decays of a chunk up to token i, S the state in front of it:
//     o_i = scale ( e^{c_i} q_i S + sum_{j <= i} e^{c_i - c_j} (q_i . k_j) v_j )
//     S'  = e^{c_128} S + sum_j k_j (e^{c_128 - c_j} v_j)^T
//
// Products, 128 x 128 x 128 each (Dk = Dv = 128), all issued by one thread in this order a chunk:
//   QK   scores[i, j]        A = Q, B = K                  (shared memory)
//   KV   X[dv, dk] = (e^. V)^T K in three parts: A = part of (e^. V)^T (TMEM), B = K
//   QS   O = Q S             A = Q, B = S^T in bf16        (shared memory)
//   PV   O += P V            A = P (TMEM, over the scores), B = V
// so that while KV and QS run (two thirds of the products' time) the scores become P, and while QK and KV run the
// outputs before are written and the state is rounded.
// The state is fp32: X is added to it on the FMA units, and e^. v is cut into three bf16 parts that add up to its 24
// bits, so that the state is as exact as an fp32 recurrence's.  O sums both terms in one accumulator: a row is kept divided
// by e^{m_i}, m_i = max(c_i, -64), which is 1 in front of Q S, and its scores are e^{c_i - c_j - m_i}: at most
// e^64, inside bf16's range.  The output's last product is scale e^{m_i}.  (Rows past c_i = -64 so keep e^-64 of S instead of
// less: 1.6e-28.)
//
// Exponents.  c is summed within blocks of 32 tokens, forward for a row's factor and backward for a column's.  With block sums
// T_b, a score off the diagonal blocks takes e^{c_i - R} e^{R - c_j}, R the end of j's block, a factor of its row and one of its
// column, both of sums of what lies between the two alone; only the 32 x 32 diagonal blocks take an exponential an element, of
// c_i - c_j.  That is a difference of large sums for tokens behind several in the same 32 that start anew (of -100 each): it is off
// by a few 2^-24 of these, 1e-4 behind ten of them, where the score is rounded to 2^-8.
//
// Roles (896 threads): 4 warps turn scores into P, 8 hold the state (a thread: 64 rows of a column dv in fp32 registers), 8
// make the parts of e^. V, 4 write the outputs; one warp each for TMA, the products and the decays.  A CTA walks its
// sequences' chunks without a break: the pipeline runs through from one sequence to the next.  In the first pass of a split
// the scores' and the outputs' warps make parts of V as well.
//
// What bounds it.  A chunk brings in 96 KB and takes 32 KB away; where two value heads share a key head, 96 KB of these pass
// HBM, 1.85 us of the measured copy's rate among 128 CTAs.  Its products are 48 steps of 66 cycles, 1.6 us.  It takes 2.6 us, and
// 2.2 where 32 CTAs have HBM to themselves: the products wait for the parts and for P, which wait for products (tensor pipe
// active 64 % of the cycles, schedulers issuing 63 %).  One CTA an SM: two chunks of q, k and v and the state fill its shared
// memory; scores, O, X and the parts its tensor memory.
// Measured (bf16, 128 x 128 state), in a graph and, behind the commas, called from Python with inputs and outputs of its own each
// time: 4 x 32 heads (16 of keys) x 4096 tokens 84 to 85 us, 92; that is 5.0 TB/s, 73 % of the copy's rate, and 4.6; 16 x 32 heads (8
// of keys) x 2048 157 to 164, 174; 1 x 32 heads x 32768 in 9 segments 260 to 265, 276 (one pass: 562).
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
constexpr int kThreads = 896;
constexpr uint32_t kHalf = 16384, kTile = 2 * kHalf;  // 128 rows x 64 channels, and 128
constexpr uint32_t kOffQ = 0, kOffK = 2 * kTile, kOffV = 4 * kTile, kOffS = 6 * kTile, kOffSmall = 7 * kTile;
constexpr int kSub = 32, kSlots = 2;  // tokens a slot of the parts of e^. V, and slots
// TMEM columns: scores (P over their first 64), O, X, the parts' slots of 3 x 16
constexpr uint32_t kColP = 0, kColO = 128, kColX = 256, kColV = 384, kSlotCols = 48;
constexpr float kMinRow = -64.f * kLog2e;  // least m_i, in powers of two

// Registers a thread of each role; what the block is launched with covers their sum (launch checks it).
constexpr int kRegsP = 72, kRegsS = 112, kRegsV = 56, kRegsO = 56, kRegsCtl = 40;
constexpr int kRegsSum = (kRegsP + 2 * kRegsS + 2 * kRegsV + kRegsO + kRegsCtl) * 128;
// (the first role keeps what it is launched with: the others' rise and fall add up without it)
static_assert(kRegsP == 65536 / kThreads / 8 * 8, "registers a thread at launch");

struct Small {
    float c[2][kC];      // sums of log2-decays within blocks of 32
    float h[2][kC];      // e^(the log-decays behind the token in its block)
    float T[2][4];       // the blocks' log2-decays
    float w[2][4];       // e^(the log-decays behind the block)
    float total[2];      // e^(the chunk's)
    int bh[2], t[2], n[2];  // its head, its first token, and how many it has (0: there is no further chunk)
    uint64_t vtile[2], kqfull[2], tfree[2], decfull[2], decfree[2];
    uint64_t staged[2][2];  // a q tile's outputs, by halves of the channels
    uint64_t vfull[kSlots], vfree[kSlots];
    uint64_t sfull, sfree, xfull[2], xfree[2], qkfull, pfull, ofull, ofree, drain, stall;
    uint32_t tmem;
    int gave_up;
    int cta, items;  // with kHanded: this CTA's number, and how many items it has at most
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

// The same for 4 columns.
__device__ __forceinline__ void tmem_st16x128_x1(uint32_t taddr, uint32_t r0, uint32_t r1) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x1.b32 [%0], {%1,%2};" ::"r"(taddr), "r"(r0), "r"(r1) : "memory");
}
// 32 lanes x 16 consecutive columns.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
        : "r"(taddr));
}

// Waits, inline (a kernel that shares out its registers cannot call functions) and few instructions long (there are many
// of them): half a million tests, then false.  A test suspends the thread for 3.7 us (of the 2 that it asks for), so
// that it gives up after some 2 s.  (Shorter suspensions are more instructions for the others to wait behind: 4 % of the
// whole kernel.  A limit that a launch is given: 0.5 to 1 %.)
constexpr uint32_t kMostTests = 1u << 19, kTestNs = 2000;
__device__ __forceinline__ bool wait_one(uint64_t* bar, uint32_t parity) {
    uint32_t i = 0;
#pragma unroll 1
    while (!mbar_try_wait_sleep(bar, parity, kTestNs))
        if (++i == kMostTests) return false;
    return true;
}
// By a warp, with one answer for its lanes.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_one(bar, parity));
}

// Two fp32 values in one operation.
__device__ __forceinline__ unsigned long long pair(float lo, float hi) {
    return (unsigned long long)__float_as_uint(hi) << 32 | __float_as_uint(lo);
}
__device__ __forceinline__ float pair_lo(unsigned long long x) { return __uint_as_float((uint32_t)x); }
__device__ __forceinline__ float pair_hi(unsigned long long x) { return __uint_as_float((uint32_t)(x >> 32)); }
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint32_t pack2(unsigned long long x) { return pack_bf16x2(pair_lo(x), pair_hi(x)); }

// lo and hi less the two bf16 values in x (fma.rn.f32.bf16: on the FMA pipe, and no widening of x first).
__device__ __forceinline__ void less2(uint32_t x, float& lo, float& hi) {
    asm("{\n\t.reg .b16 l, h, minus;\n\tmov.b32 {l, h}, %2;\n\tmov.b16 minus, 0xBF80;\n\t"
        "fma.rn.f32.bf16 %0, l, minus, %0;\n\tfma.rn.f32.bf16 %1, h, minus, %1;\n\t}"
        : "+f"(lo), "+f"(hi)
        : "r"(x));
}
// The two bf16 values in m, times d, as the sum of three bf16 values each: an fp32 product's 24 bits, cut off 8 at a time
// (the differences are exact).  The work is spread over the pipes: widening and cutting on the ALU (a byte permutation cuts
// two values and packs them), products and differences on the FMA pipe; either pipe alone is 2 to 4 us slower of 87.
__device__ __forceinline__ void three_parts(uint32_t m, float d0, float d1, uint32_t& p0, uint32_t& p1, uint32_t& p2) {
    const auto cut = [](float a, float b) { return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632); };
    float a = bf16lo_to_f32(m) * d0, b = bf16hi_to_f32(m) * d1;
    p0 = cut(a, b);
    less2(p0, a, b);
    p1 = cut(a, b);
    less2(p1, a, b);
    p2 = cut(a, b);
}

__device__ __forceinline__ void tmem_st8u(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// What the kernel's walk over its items needs: (segment, head) pairs, heads fastest, every gridDim-th of them a CTA's.
// kHanded (one segment): every CTA has `whole` heads, and the heads that are left over are each cut into parts of `len` tokens,
// which `handed` CTAs run: part j of the r-th is CTA j rest + r's, after j of its whole heads, so that part j - 1 has left
// its state in state_out long before.  (152 SMs, us, whole heads alone and with parts: 16 x 32 heads x 2048 172, 162; 5 x 32
// x 4096 163, 133; 5 x 32 x 1024 50, 48; 40 x 16 x 800 104, 99.  Whole heads stay where they were, beside those that share their key
// head, whose q and k then come from L2.)
struct Items {
    int heads, segs, len;  // B Hv; segments that this launch runs; tokens of one (S where there is one)
    Divisor hv, group;     // by Hv: the batch; by Hv / Hk: the key head, counted over the batch
    int whole, rest, handed;
    uint32_t* flags;       // kHanded: how many CTAs have begun; 8 a CTA: whether its part's state has been written
};
struct Walk {  // a CTA's chunks one after another, over all of its items that have any
    int bh, seg, t, end;  // head (over the batch), segment (kHanded: items before), the chunk's first token, the item's end
    int part;             // of a head that is cut into parts: which (else -1)
};
__device__ __forceinline__ void place(Walk& k, const Items& it, const Small& sh) {  // (kHanded)
    const int j = sh.cta < it.handed ? sh.cta / it.rest : it.whole + 1, grid = gridDim.x;
    k.part = k.seg == j ? j : -1;
    k.bh = k.seg == j ? it.whole * grid + sh.cta - j * it.rest : sh.cta + (k.seg - (k.seg > j ? 1 : 0)) * grid;
}
template <bool kHanded>
__device__ __forceinline__ void next_item(Walk& k, const Items& it, const Small& sh) {
    if (kHanded) {
        ++k.seg;
        place(k, it, sh);
        return;
    }
    k.bh += gridDim.x;
    while (k.bh >= it.heads) {
        k.bh -= it.heads;
        ++k.seg;
    }
}
template <bool kHanded>
__device__ __forceinline__ int tokens_of(Walk& k, const LinearAttn& p, const Items& it) {  // the item's end without lengths
    int len = p.S;
    if (p.lengths) len = max(0, min(len, p.lengths[it.hv.of(k.bh)]));
    const int most = kHanded && k.part < 0 ? p.S : it.len;
    k.t = kHanded ? max(k.part, 0) * it.len : k.seg * it.len;
    k.end = len - k.t > most ? k.t + most : len;
    return p.S - k.t > most ? k.t + most : p.S;
}
template <bool kHanded>
__device__ __forceinline__ int items_of(const Items& it, const Small& sh) {
    return kHanded ? sh.items : it.segs;
}
template <bool kHanded>
__device__ __forceinline__ bool settle(Walk& k, const LinearAttn& p, const Items& it, const Small& sh) {
#pragma unroll 1
    for (; k.seg < items_of<kHanded>(it, sh); next_item<kHanded>(k, it, sh)) {
        (void)tokens_of<kHanded>(k, p, it);
        if (k.t < k.end) return true;
    }
    return false;
}
template <bool kHanded>
__device__ __forceinline__ Walk first_item(const Items& it, const Small& sh) {
    Walk k{(int)blockIdx.x, 0, 0, 0, -1};
    if (kHanded) {
        place(k, it, sh);
        return k;
    }
    while (k.bh >= it.heads) {
        k.bh -= it.heads;
        ++k.seg;
    }
    return k;
}
template <bool kHanded>
__device__ __forceinline__ bool next_chunk(Walk& k, const LinearAttn& p, const Items& it, const Small& sh) {
    k.t += kC;
    if (k.t < k.end) return true;
    next_item<kHanded>(k, it, sh);
    return settle<kHanded>(k, p, it, sh);
}
// The flag of a part that another CTA runs (bounded: a second at the least).
__device__ __forceinline__ bool wait_flag(const uint32_t* flag) {
    uint32_t v = 0;
#pragma unroll 1
    for (uint32_t i = 0; i < 2 * kMostTests; ++i) {
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(flag) : "memory");
        if (v) return true;
        asm volatile("nanosleep.u32 1000;");
    }
    return false;
}

// Descriptors in two words: an offset within shared memory is added to the low one (no carry leaves its address field).
struct Desc {
    uint32_t lo, hi;
};
__device__ __forceinline__ Desc desc_of(uint32_t saddr, uint32_t lbo) {
    const uint64_t d = make_sdesc(saddr, lbo, 1024);
    return Desc{(uint32_t)d, (uint32_t)(d >> 32)};
}
// One 128 x N x 16 step of D (+)= A B^T, A in shared memory or in tensor memory.
template <bool kAdd>
__device__ __forceinline__ void step_ss(uint32_t d, Desc a, uint32_t a_at, Desc b, uint32_t b_at, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tmov.b64 x, {%1, %2};\n\tmov.b64 y, {%3, %4};\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %5, p;\n\t}" ::"r"(d),
        "r"(a.lo + (a_at >> 4)), "r"(a.hi), "r"(b.lo + (b_at >> 4)), "r"(b.hi), "r"(idesc), "n"(kAdd ? 1 : 0)
        : "memory");
}
template <bool kAdd>
__device__ __forceinline__ void step_ts(uint32_t d, uint32_t a, Desc b, uint32_t b_at, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tmov.b64 y, {%2, %3};\n\tsetp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b.lo + (b_at >> 4)), "r"(b.hi), "r"(idesc), "n"(kAdd ? 1 : 0)
        : "memory");
}
// D = A B^T over `ksteps` steps of 16 along the rows of two tiles.  All eight steps of 128 channels run without a branch
// between them: products issued so follow one another every 66 cycles, their own time, and with a test or a
// descriptor made anew before each every 140.
__device__ __forceinline__ void product_rows(uint32_t d, Desc a, Desc b, uint32_t idesc, int ksteps) {
    step_ss<false>(d, a, 0, b, 0, idesc);
    if (ksteps == 8) {
#pragma unroll
        for (int k = 1; k < 8; ++k) {
            const uint32_t at = (k >> 2) * kHalf + (k & 3) * 32;
            step_ss<true>(d, a, at, b, at, idesc);
        }
    } else {
#pragma unroll 1
        for (int k = 1; k < ksteps; ++k) {
            const uint32_t at = (k >> 2) * kHalf + (k & 3) * 32;
            step_ss<true>(d, a, at, b, at, idesc);
        }
    }
}
// The six steps of one slot's 32 tokens: three parts, 16 tokens each.
__device__ __forceinline__ void product_parts(uint32_t d, uint32_t a, Desc b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tmov.b64 y, {%2, %3};\n\tsetp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"((int)add)
        : "memory");
    step_ts<true>(d, a + 16, b, 0, idesc);
    step_ts<true>(d, a + 32, b, 0, idesc);
    step_ts<true>(d, a + 8, b, 2048, idesc);
    step_ts<true>(d, a + 24, b, 2048, idesc);
    step_ts<true>(d, a + 40, b, 2048, idesc);
}

// 64 rows of a state column: rows `pitch` floats apart, `rows` of them there.  Of whole heads (128 x 128, the pitch known
// at compile time) a row is one instruction.
template <typename F>
__device__ __forceinline__ void column_rows(int pitch, int rows, F f) {
    if (pitch == kC && rows == 64) {
#pragma unroll
        for (int i = 0; i < 64; ++i) f(i, i * kC, true);
    } else {
#pragma unroll
        for (int i = 0; i < 64; ++i) {
            f(i, i * pitch, i < rows);
            if (i % 16 == 15) asm volatile("" ::: "memory");  // (no more addresses at once)
        }
    }
}

// kStatesOnly: the first pass of a split (end states and decays of segments 0 .. P - 2; only KV is formed).  kHanded: heads that
// are left over go in parts (see Items).
template <bool kStatesOnly, bool kHanded>
__global__ void __launch_bounds__(kThreads, 1)
    linear_attn_tc_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                          const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap to,
                          const __grid_constant__ LinearAttn p, const __grid_constant__ LinearAttnSplit split,
                          const __grid_constant__ Items it, int stall, int32_t* status) {
    extern __shared__ __align__(1024) uint8_t sm[];
    Small& sh = *reinterpret_cast<Small*>(sm + kOffSmall);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = warp & 3;
    const uint32_t sbase = smem_u32(sm);

    if (sbase & 1023u) {  // (the tiles' descriptors need it, and a launch without static shared memory has it)
        if (tid == 0 && status) atomicExch(status, (int32_t)GDN_ERR_CUDA);
        return;
    }
    if (tid == 0) {
        sh.gave_up = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.vtile[i], 1);
            mbar_init(&sh.kqfull[i], 1);
            mbar_init(&sh.tfree[i], 1);
            for (int h = 0; h < 2; ++h) mbar_init(&sh.staged[i][h], 128);
            mbar_init(&sh.decfull[i], 32);
            mbar_init(&sh.decfree[i], 769);  // 24 warps and the thread of the products
        }
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&sh.vfull[i], 128 * (kStatesOnly ? 4 : 2));
            mbar_init(&sh.vfree[i], 1);
        }
        mbar_init(&sh.sfull, 256);
        mbar_init(&sh.sfree, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.xfull[i], 1);
            mbar_init(&sh.xfree[i], 256);
        }
        mbar_init(&sh.qkfull, 1);
        mbar_init(&sh.pfull, 128);
        mbar_init(&sh.ofull, 1);
        mbar_init(&sh.ofree, 128);
        mbar_init(&sh.drain, 1);
        mbar_init(&sh.stall, 1);
        fence_mbar_init();
    }
    if (warp == 25) tmem_alloc(&sh.tmem, 512);
    if (warp == 24 && elect_one()) {
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
    if (kHanded) {
        // numbers in the order of beginning: a CTA that is waited for runs already
        if (tid == 0) {
            sh.cta = (int)atomicAdd(it.flags, 1u);
            sh.items = it.whole + (sh.cta < it.handed ? 1 : 0);
        }
        __syncthreads();
    }

    int cn = 0;      // chunks so far, over all items
    bool ok = true;  // no wait has run out
    // the first pass has no scores and no outputs: their warps make parts of V too
    constexpr int kGroups = kStatesOnly ? 4 : 2;
    const bool parts_role = kStatesOnly ? warp < 4 || (warp >= 12 && warp < 24) : warp >= 12 && warp < 20;
    if (!kStatesOnly && warp < 4) {
        // ------------------------------------------------------------ scores -> P
        const int a = quad;
        for (;; ++cn) {
            const int s = cn & 1;
            ok = wait_warp(&sh.decfull[s], (cn >> 1) & 1);
            if (!ok || sh.n[s] == 0) break;
            float R = 0.f;
#pragma unroll 1
            for (int m = 0; m < a; ++m) R += sh.T[s][m];
            const float ci = sh.c[s][32 * a + lane], shift = ci - fmaxf(R + ci, kMinRow);
            ok = wait_warp(&sh.qkfull, cn & 1);
            if (!ok) break;
            tc_fence_after();
            // 16 columns at a time, the next 16 on their way; loops that stay small: the roles share the
            // instruction caches.  What is written lies over score columns that this warp has read
            // c_i - m_i less the end of block b, for this block and the next one (sums of what lies between alone)
            float next = shift + (a > 2 ? sh.T[s][2] : 0.f), between = a > 2 ? next + sh.T[s][1] : a > 1 ? shift + sh.T[s][1] : shift;
            float x[16], y[16];
            tmem_ld16(tq4 + kColP, x);
            const auto off_diagonal = [&](const float (&v)[16], unsigned long long uu, int col) {
                uint32_t pk[8];
                const float4* h = reinterpret_cast<const float4*>(&sh.h[s][col]);
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const float4 hj = h[j / 4];
                    pk[j / 2] = pack2(mul2(pair(v[j], v[j + 1]), mul2(uu, pair(hj.x, hj.y))));
                    pk[j / 2 + 1] = pack2(mul2(pair(v[j + 2], v[j + 3]), mul2(uu, pair(hj.z, hj.w))));
                }
                tmem_st8u(tq4 + kColP + col / 2, pk);
            };
#pragma unroll 1
            for (int b = 0; b < a; ++b) {
                const float u = exp2_approx(between);
                const unsigned long long uu = pair(u, u);
                between = next;
                next = shift;
                tmem_wait_ld();
                tmem_ld16(tq4 + kColP + 32 * b + 16, y);
                off_diagonal(x, uu, 32 * b);
                tmem_wait_ld();
                tmem_ld16(tq4 + kColP + 32 * b + 32, x);
                off_diagonal(y, uu, 32 * b + 16);
            }
            tmem_wait_ld();
            tmem_ld16(tq4 + kColP + 32 * a + 16, y);
#pragma unroll 1
            for (int j0 = 0; j0 < 32; j0 += 16) {  // the diagonal block
                uint32_t pk[8];
                const float4* cc = reinterpret_cast<const float4*>(&sh.c[s][32 * a + j0]);
                const int last = lane - j0;
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const float4 cj = cc[j / 4];
                    const float y0 = j <= last ? x[j] * exp2_approx(shift - cj.x) : 0.f;
                    const float y1 = j + 1 <= last ? x[j + 1] * exp2_approx(shift - cj.y) : 0.f;
                    const float y2 = j + 2 <= last ? x[j + 2] * exp2_approx(shift - cj.z) : 0.f;
                    const float y3 = j + 3 <= last ? x[j + 3] * exp2_approx(shift - cj.w) : 0.f;
                    pk[j / 2] = pack_bf16x2(y0, y1);
                    pk[j / 2 + 1] = pack_bf16x2(y2, y3);
                }
                tmem_st8u(tq4 + kColP + 16 * a + j0 / 2, pk);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] = y[j];
            }
#pragma unroll 1
            for (int b = 2 * a + 2; b < 8; ++b) {  // columns behind the row's block
                const uint32_t zero[8] = {};
                tmem_st8u(tq4 + kColP + 8 * b, zero);
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&sh.pfull);
            mbar_arrive(&sh.decfree[s]);
        }
    } else if (warp >= 4 && warp < 12) {
        // ------------------------------------------------------------ the state: thread = 64 rows of column dv
        regs_inc<kRegsS>();
        const int dv = quad * 32 + lane, half = (warp - 4) >> 2;
        const int rows = dv < p.Dv ? min(64, p.Dk - 64 * half) : 0;  // of the 64 that are there (<= 0: none)
        const long long ns = (long long)p.Dk * p.Dv, heads = it.heads;
        const int first = 64 * half * p.Dv + dv;
        uint8_t* const sb = sm + kOffS + half * kHalf + dv * 128;
        float S[64];
        for (Walk k = first_item<kHanded>(it, sh); k.seg < items_of<kHanded>(it, sh) && ok; next_item<kHanded>(k, it, sh)) {
            (void)tokens_of<kHanded>(k, p, it);
            int pitch = p.Dv;
            asm volatile("" : "+r"(pitch));  // (64 rows' offsets are not kept in registers over the chunks)
            const float* src = p.state_in ? p.state_in + k.bh * ns : nullptr;
            if (!kStatesOnly && split.P > 1) src = split.start(k.seg, k.bh, heads, ns);
            if (kStatesOnly && k.seg) src = nullptr;
            if (kHanded && k.part > 0) {  // (each warp left what its namesake reads)
                ok = __all_sync(0xffffffffu, wait_flag(it.flags + 1 + 8 * (sh.cta - it.rest) + warp - 4));
                if (!ok) break;
                src = p.state_out + k.bh * ns;
            }
            if (src) {
                src += first;
                column_rows(pitch, rows, [&](int i, int at, bool in) { S[i] = !in ? 0.f : kHanded ? __ldcg(src + at) : src[at]; });
            } else {
#pragma unroll
                for (int i = 0; i < 64; ++i) S[i] = 0.f;
            }
            if (kStatesOnly && k.seg == 0) {  // the copy of state_in
                float* x = split.parts + ((split.P - 1) * heads + k.bh) * ns + first;
                column_rows(pitch, rows, [&](int i, int at, bool in) {
                    if (in) x[at] = S[i];
                });
            }
            float decay = 1.f;
            for (; k.t < k.end; k.t += kC, ++cn) {
                const int s = cn & 1;
                if (!kStatesOnly) {
                    // S^T in bf16, rows dv, when the product that reads the previous one is done
                    ok = cn == 0 || wait_warp(&sh.sfree, (cn - 1) & 1);
                    if (!ok) break;
#pragma unroll
                    for (int ch = 0; ch < 8; ++ch) {
                        const float* x = S + 8 * ch;
                        *reinterpret_cast<uint4*>(sb + ((ch ^ (dv & 7)) << 4)) =
                            make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                       pack_bf16x2(x[6], x[7]));
                    }
                    fence_proxy_async_smem();
                    mbar_arrive(&sh.sfull);
                }
                ok = wait_warp(&sh.decfull[s], (cn >> 1) & 1);
                if (!ok) break;
                const float e = sh.total[s];
                decay *= e;
                mbar_arrive(&sh.decfree[s]);
                const int xb = kStatesOnly ? cn & 1 : 0;  // (see the products)
                ok = wait_warp(&sh.xfull[xb], kStatesOnly ? (cn >> 1) & 1 : cn & 1);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    if (64 * half + 16 * b < p.Dk) {
                        float x[16];
                        tmem_ld16(tq4 + (xb ? kColO : kColX) + 64 * half + 16 * b, x);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            const unsigned long long y =
                                fma2(pair(e, e), pair(S[16 * b + i], S[16 * b + i + 1]), pair(x[i], x[i + 1]));
                            S[16 * b + i] = pair_lo(y);
                            S[16 * b + i + 1] = pair_hi(y);
                        }
                    }
                }
                tc_fence_before();
                mbar_arrive(&sh.xfree[xb]);
            }
            if (!ok) break;
            float* dst = nullptr;
            if (kStatesOnly) {
                dst = split.parts + (k.seg * heads + k.bh) * ns;
                if (tid == 128) split.decays[k.seg * heads + k.bh] = decay;
            } else if (kHanded || k.seg == split.P - 1) {
                dst = p.state_out + k.bh * ns;
            }
            if (dst) {
                dst += first;
                column_rows(pitch, rows, [&](int i, int at, bool in) {
                    if (in) dst[at] = S[i];
                });
                if (kHanded && k.part >= 0) {
                    __syncwarp();
                    if (lane == 0)
                        asm volatile("fence.acq_rel.gpu;\n\tst.release.gpu.global.u32 [%0], %1;" ::"l"(
                                         it.flags + 1 + 8 * sh.cta + warp - 4),
                                     "r"(1u)
                                     : "memory");
                }
            }
        }
    } else if (parts_role) {
        // ------------------------------------------------------------ parts of e^. V
        regs_dec<kRegsV>();
        constexpr int kOct = 4 / kGroups;  // of 8 tokens, of a slot's four, a warp
        const int group = warp < 4 ? 3 : (warp - 12) >> 2;
        const int tok = group * (kSub / kGroups) + (lane & 7);
        // the 16-byte piece of a row that this lane's address takes
        const uint32_t piece = (quad >> 1) * kHalf + sw128_offset(tok, (quad & 1) * 64 + (lane >> 3) * 16);
        const uint32_t at = tq4 + kColV + 4 * kOct * group;
        const bool there = quad * 32 < p.Dv;
        int vi = 0;  // slots so far
        for (;; ++cn) {
            const int s = cn & 1;
            ok = wait_warp(&sh.decfull[s], (cn >> 1) & 1);
            const int n = sh.n[s], subs = (n + kSub - 1) / kSub;
            if (!ok || n == 0) break;
            ok = wait_warp(&sh.vtile[s], (cn >> 1) & 1);
            if (!ok) break;
            uint8_t* vt = sm + kOffV + s * kTile;
            if (n < subs * kSub && p.lengths) {
                // rows behind the last token in the last 32: whatever they hold is not multiplied, not even by zero.
                // A warp clears the columns that it reads itself, of V and of K (some warps the same ones)
                const int rows = subs * kSub - n;
                ok = wait_warp(&sh.kqfull[s], (cn >> 1) & 1);
                if (!ok) break;
#pragma unroll 1
                for (int i = lane; i < rows * 8; i += 32) {
                    const uint32_t to = (quad >> 1) * kHalf + sw128_offset(n + (i >> 3), (quad & 1) * 64 + (i & 3) * 16);
                    *reinterpret_cast<uint4*>((i & 4 ? vt : sm + kOffK + s * kTile) + to) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                __syncwarp();
            }
            uint32_t from = smem_u32(vt) + piece;
            const float* h = &sh.h[s][group * (kSub / kGroups) + 2 * (lane & 3)];
            uint32_t m[kOct][4];
            float2 hh[kOct];
            const auto fetch = [&] {  // a slot's tokens of this warp
#pragma unroll
                for (int o = 0; o < kOct; ++o) {
                    ldmatrix_x4_trans(from + o * 1024, m[o]);
                    hh[o] = *reinterpret_cast<const float2*>(h + 8 * o);
                }
                from += kSub * 128;
                h += kSub;
            };
            fetch();
#pragma unroll 1
            for (int u = 0; u < subs; ++u, ++vi) {
                const int slot = vi & 1, turn = vi >> 1;
                uint32_t part[3][kOct][4];  // [part][8 tokens][8 columns dv], made before the slot is free
                const float wb = sh.w[s][u];
#pragma unroll
                for (int o = 0; o < kOct; ++o) {
                    const float d0 = hh[o].x * wb, d1 = hh[o].y * wb;
#pragma unroll
                    for (int i = 0; i < 4; ++i) three_parts(m[o][i], d0, d1, part[0][o][i], part[1][o][i], part[2][o][i]);
                }
                if (u + 1 < subs) fetch();
                if (turn > 0) {
                    ok = wait_warp(&sh.vfree[slot], (turn - 1) & 1);
                    if (!ok) break;
                }
                if (there) {
                    tc_fence_after();
                    const uint32_t to = at + slot * kSlotCols;
#pragma unroll
                    for (int q = 0; q < 3; ++q)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {  // 16 of the warp's columns dv each
                            const uint32_t dst = to + 16 * q + (r ? 16u << 16 : 0u);
                            const uint32_t *x = part[q][0] + 2 * r, *y = part[q][kOct - 1] + 2 * r;
                            if (kOct == 2)
                                tmem_st16x128_x2(dst, x[0], x[1], y[0], y[1]);
                            else
                                tmem_st16x128_x1(dst, x[0], x[1]);
                        }
                    tmem_wait_st();
                    tc_fence_before();
                }
                mbar_arrive(&sh.vfull[slot]);
            }
            if (!ok) break;
            mbar_arrive(&sh.decfree[s]);
        }
    } else if (!kStatesOnly && warp >= 20 && warp < 24) {
        // ------------------------------------------------------------ outputs
        regs_dec<kRegsO>();
        const int r = quad * 32 + lane;
        for (;; ++cn) {
            const int s = cn & 1;
            ok = wait_warp(&sh.decfull[s], (cn >> 1) & 1);
            const int n = sh.n[s];
            if (!ok || n == 0) break;
            float R = sh.c[s][r];
#pragma unroll 1
            for (int m = 0; m < quad; ++m) R += sh.T[s][m];
            const float f = p.scale * exp2_approx(fmaxf(R, kMinRow));
            uint8_t* row = static_cast<uint8_t*>(p.out) + ((long long)sh.bh[s] * p.S + sh.t[s] + r) * p.Pv * 2;
            // whole chunks and the tensor's end go out by TMA, from q's tile (its products are done); where a length
            // ends inside a chunk, a thread writes its row itself (rows behind the length: zeros, or nothing)
            const bool tma = n == kC || sh.t[s] + n == p.S;
            const int rows = p.zero_rest ? p.S - sh.t[s] : n;  // that are written so
            mbar_arrive(&sh.decfree[s]);
            ok = wait_warp(&sh.ofull, cn & 1);
            if (!ok) break;
            tc_fence_after();
            uint8_t* tile = sm + kOffQ + s * kTile + r * 128;
            const auto put = [&](const float (&x)[16], int col) {
                uint32_t o[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = pack2(mul2(pair(f, f), pair(x[2 * j], x[2 * j + 1])));
                const uint4 lo = make_uint4(o[0], o[1], o[2], o[3]), hi = make_uint4(o[4], o[5], o[6], o[7]);
                if (tma) {
                    uint8_t* half = tile + (col >> 6) * kHalf;
                    const int ch = (col & 63) >> 3;
                    *reinterpret_cast<uint4*>(half + ((ch ^ (r & 7)) << 4)) = lo;
                    *reinterpret_cast<uint4*>(half + (((ch + 1) ^ (r & 7)) << 4)) = hi;
                } else if (r < rows) {
                    const uint4 zero = make_uint4(0, 0, 0, 0);
                    if (col < p.Dv) *reinterpret_cast<uint4*>(row + 2 * col) = r < n ? lo : zero;
                    if (col + 8 < p.Dv) *reinterpret_cast<uint4*>(row + 2 * col + 16) = r < n ? hi : zero;
                }
            };
            // (columns past Dv come from whatever the tensor memory holds, and are not written)
#pragma unroll 1
            for (int col = 0; col < 128; col += 32) {
                if (col < p.Dv) {
                    float x[16], y[16];
                    tmem_ld16(tq4 + kColO + col, x);
                    tmem_ld16(tq4 + kColO + col + 16, y);
                    tmem_wait_ld();
                    put(x, col);
                    put(y, col + 16);
                }
                if (col & 32) {
                    fence_proxy_async_smem();
                    mbar_arrive(&sh.staged[s][col >> 6]);
                }
            }
            tc_fence_before();
            mbar_arrive(&sh.ofree);
        }
    } else {
        regs_dec<kRegsCtl>();
        if (warp == 24) {
            // -------------------------------------------------------- TMA, one thread
            if (elect_one()) {
                const uint32_t kb = p.Dk > 64 ? kTile : kHalf, vb = p.Dv > 64 ? kTile : kHalf;
                int v_issued = 0, kq_issued = 0;
                struct Tile {
                    int t, bh, n;
                } was[2] = {{0, 0, 0}, {0, 0, 0}};  // chunks cn - 2 and cn - 1 (n = 0: none)
                Walk k = first_item<kHanded>(it, sh);
                bool more = settle<kHanded>(k, p, it, sh);
                Walk far = k;  // a chunk two ahead, whose K and q are brought into L2 (V's load has the time)
                bool ahead = more && next_chunk<kHanded>(far, p, it, sh);
                // The engine works in order: what is needed first goes first.  V, out of which parts are made; the outputs of
                // chunk cn - 2, which leave the q tile that chunk cn takes; K and q; then the prefetch
                for (; more || was[0].n || was[1].n; ++cn) {
                    const int s = cn & 1, ph = (cn >> 1) & 1, bhk = it.group.of(k.bh);
                    if (more) {
                        ok = cn < 2 || wait_one(&sh.tfree[s], ph ^ 1);
                        if (!ok) break;
                        uint8_t* vt = sm + kOffV + s * kTile;
                        mbar_arrive_expect_tx(&sh.vtile[s], vb);
                        tma_load_3d(vt, &tv, &sh.vtile[s], 0, k.t, k.bh);
                        if (p.Dv > 64) tma_load_3d(vt + kHalf, &tv, &sh.vtile[s], 64, k.t, k.bh);
                        v_issued = cn + 1;
                    }
                    uint8_t* qt = sm + kOffQ + s * kTile;
                    if (was[0].n) {
                        const bool whole = was[0].n == kC || was[0].t + was[0].n == p.S;
#pragma unroll 1
                        for (int h = 0; h < 2 && ok; ++h) {
                            // (a barrier a tile: its next phase is that of chunk cn, whose q is loaded behind this wait.  This thread may
                            // come late, from a walk over many items without tokens, and the outputs of chunk cn - 1 be there too)
                            ok = wait_one(&sh.staged[s][h], ph ^ 1);
                            if (ok && whole && 64 * h < p.Dv)
                                tma_store_3d(&to, qt + h * kHalf, 64 * h, was[0].t, was[0].bh);
                        }
                        tma_store_commit();
                        if (!ok) break;
                    }
                    if (more) {
                        uint8_t* kt = sm + kOffK + s * kTile;
                        mbar_arrive_expect_tx(&sh.kqfull[s], kStatesOnly ? kb : 2 * kb);
                        tma_load_3d(kt, &tk, &sh.kqfull[s], 0, k.t, bhk);
                        if (p.Dk > 64) tma_load_3d(kt + kHalf, &tk, &sh.kqfull[s], 64, k.t, bhk);
                        kq_issued = cn + 1;
                    }
                    tma_store_wait_read0();
                    was[0] = was[1];
                    was[1].n = 0;
                    if (more) {
                        if (!kStatesOnly) {
                            tma_load_3d(qt, &tq, &sh.kqfull[s], 0, k.t, bhk);
                            if (p.Dk > 64) tma_load_3d(qt + kHalf, &tq, &sh.kqfull[s], 64, k.t, bhk);
                            was[1] = Tile{k.t, k.bh, min(kC, k.end - k.t)};
                        }
                        more = next_chunk<kHanded>(k, p, it, sh);
                        if (ahead) ahead = next_chunk<kHanded>(far, p, it, sh);
                        if (ahead) {
                            const int fhk = it.group.of(far.bh);
#pragma unroll 1
                            for (int x = 0; x < 128; x += 64) {
                                if (x < p.Dk) {
                                    tma_prefetch_l2_3d(&tk, x, far.t, fhk);
                                    if (!kStatesOnly) tma_prefetch_l2_3d(&tq, x, far.t, fhk);
                                }
                            }
                        }
                    }
                }
                tma_store_wait_all0();
                // every load has landed before the CTA ends (bounded)
#pragma unroll 1
                for (int i = max(0, v_issued - 2); i < v_issued; ++i) (void)wait_one(&sh.vtile[i & 1], (i >> 1) & 1);
#pragma unroll 1
                for (int i = max(0, kq_issued - 2); i < kq_issued; ++i) (void)wait_one(&sh.kqfull[i & 1], (i >> 1) & 1);
            }
            __syncwarp();
        } else if (warp == 25) {
            // -------------------------------------------------------- products, all by one thread
            if (elect_one()) {
                const int Nk = (p.Dk + 15) & ~15, Nv = (p.Dv + 15) & ~15, ksteps = Nk / 16;
                constexpr uint32_t kIdQK = make_idesc_bf16(128, 128, 0, 0);
                const uint32_t id_qs = make_idesc_bf16(128, Nv, 0, 0), id_pv = make_idesc_bf16(128, Nv, 0, 1),
                               id_kv = make_idesc_bf16(128, Nk, 0, 1);
                const Desc ds = desc_of(sbase + kOffS, 16);
                int vi = 0;
                // the tokens of chunk cn (0: there is none) once its tiles are loaded; -1 after a wait that ran out
                const auto next = [&] {
                    const int s = cn & 1, ph = (cn >> 1) & 1;
                    if (!wait_one(&sh.decfull[s], ph)) return -1;
                    const int n = sh.n[s];
                    mbar_arrive(&sh.decfree[s]);
                    if (n > 0 && !wait_one(&sh.kqfull[s], ph)) return -1;
                    return n;
                };
                int n = next();
                while (n > 0) {
                    const int s = cn & 1, subs = (n + kSub - 1) / kSub;
                    n = -1;
                    const Desc dq = desc_of(sbase + kOffQ + s * kTile, 16);
                    if (!kStatesOnly) {
                        tc_fence_after();
                        product_rows(tmem + kColP, dq, desc_of(sbase + kOffK + s * kTile, 16), kIdQK, ksteps);
                        mma_commit(&sh.qkfull);
                    }
                    // X of the chunk before has been read; in the first pass, which has no O, two X take turns
                    const int xb = kStatesOnly ? cn & 1 : 0;
                    const uint32_t col_x = tmem + (xb ? kColO : kColX);
                    if (kStatesOnly ? cn > 1 && !wait_one(&sh.xfree[xb], ((cn >> 1) - 1) & 1)
                                    : cn > 0 && !wait_one(&sh.xfree[xb], (cn - 1) & 1))
                        break;
                    Desc b = desc_of(sbase + kOffK + s * kTile, kHalf);
                    int u = 0;
#pragma unroll 1
                    for (; u < subs; ++u, ++vi) {
                        const int slot = vi & 1;
                        if (!wait_one(&sh.vfull[slot], (vi >> 1) & 1)) break;
                        tc_fence_after();
                        product_parts(col_x, tmem + kColV + slot * kSlotCols, b, id_kv, u > 0);
                        mma_commit(&sh.vfree[slot]);
                        b.lo += kSub * 128 / 16;
                    }
                    if (u < subs) break;
                    mma_commit(&sh.xfull[xb]);
                    if (kStatesOnly) {
                        mma_commit(&sh.tfree[s]);
                        ++cn;
                        n = next();
                        continue;
                    }
                    if (!wait_one(&sh.sfull, cn & 1) || (cn > 0 && !wait_one(&sh.ofree, (cn - 1) & 1))) break;
                    tc_fence_after();
                    product_rows(tmem + kColO, dq, ds, id_qs, ksteps);
                    mma_commit(&sh.sfree);
                    if (!wait_one(&sh.pfull, cn & 1) || !wait_one(&sh.vtile[s], (cn >> 1) & 1)) break;
                    tc_fence_after();
                    const Desc dvm = desc_of(sbase + kOffV + s * kTile, kHalf);
                    if (subs == kC / kSub) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            step_ts<true>(tmem + kColO, tmem + kColP + 8 * i, dvm, i * 2048, id_pv);
                    } else {
#pragma unroll 1
                        for (int i = 0; i < 2 * subs; ++i)
                            step_ts<true>(tmem + kColO, tmem + kColP + 8 * i, dvm, i * 2048, id_pv);
                    }
                    mma_commit(&sh.ofull);
                    mma_commit(&sh.tfree[s]);
                    ++cn;
                    n = next();
                }
                ok = n == 0;
                // every product has ended before the tensor memory is freed (bounded)
                mma_commit(&sh.drain);
                (void)wait_one(&sh.drain, 0);
            }
            __syncwarp();
        } else if (warp == 26) {
            // -------------------------------------------------------- decays, and the walk that most roles follow
            Walk k = first_item<kHanded>(it, sh);
            bool more = settle<kHanded>(k, p, it, sh);
            float g[4] = {};  // the log-decays of the walk's chunk, on their way while the chunk before is published
            const auto fetch = [&] {
                const float* from =
                    p.g_log + (p.head_decay ? k.bh - it.hv.of(k.bh) * p.Hv : (long long)k.bh * p.S + k.t + lane);
#pragma unroll
                for (int b = 0; b < 4; ++b) g[b] = 32 * b + lane < k.end - k.t ? from[p.head_decay ? 0 : 32 * b] : 0.f;
            };
            if (more) fetch();
            if (stall) ok = wait_warp(&sh.stall, 0);  // (on which nothing arrives: gdn_test_stall_prefill)
            for (; ok; ++cn) {
                const int s = cn & 1;
                float down[4];  // the log-decays from a token on to the end of its block
#pragma unroll
                for (int b = 0; b < 4; ++b) down[b] = least_decay(g[b]);
#pragma unroll
                for (int o = 1; o < 32; o <<= 1)
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const float z = __shfl_down_sync(0xffffffffu, down[b], o);
                        if (lane + o < 32) down[b] += z;
                    }
                // and from its block's beginning on to the token: a sum of its own, since the block's less what is behind the
                // token is a difference of two large ones where a block starts anew several times
                float up[4] = {};
                if (!kStatesOnly) {  // (which has no scores)
#pragma unroll
                    for (int b = 0; b < 4; ++b) up[b] = least_decay(g[b]);
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            const float z = __shfl_up_sync(0xffffffffu, up[b], o);
                            if (lane >= o) up[b] += z;
                        }
                }
                float T[4], after[4];
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    T[b] = __shfl_sync(0xffffffffu, down[b], 0);
                    after[b] = __shfl_down_sync(0xffffffffu, down[b], 1);
                    if (lane == 31) after[b] = 0.f;
                }
                // lane b: what block b's states are multiplied by behind it; lane 4: the whole chunk's
                const float t3 = T[3], t2 = T[2] + t3, t1 = T[1] + t2, t0 = T[0] + t1;
                const float behind = expf(lane == 3 ? 0.f : lane == 2 ? t3 : lane == 1 ? t2 : lane == 0 ? t1 : t0);
                ok = cn < 2 || wait_warp(&sh.decfree[s], ((cn >> 1) - 1) & 1);
                if (!ok) break;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    if (!kStatesOnly) sh.c[s][32 * b + lane] = kLog2e * up[b];
                    sh.h[s][32 * b + lane] = expf(after[b]);
                }
                if (lane < 4) {
                    sh.T[s][lane] = kLog2e * (lane == 3 ? T[3] : lane == 2 ? T[2] : lane == 1 ? T[1] : T[0]);
                    sh.w[s][lane] = behind;
                } else if (lane == 4) {
                    sh.total[s] = behind;
                    sh.bh[s] = k.bh;
                    sh.t[s] = k.t;
                    sh.n[s] = more ? min(kC, k.end - k.t) : 0;
                }
                mbar_arrive(&sh.decfull[s]);
                if (!more) break;
                more = next_chunk<kHanded>(k, p, it, sh);
                if (more) fetch();
            }
        } else if (!kStatesOnly && p.zero_rest) {
            // -------------------------------------------------------- zeros behind the lengths, from the next chunk on
#pragma unroll 1
            for (Walk k = first_item<kHanded>(it, sh); k.seg < items_of<kHanded>(it, sh); next_item<kHanded>(k, it, sh)) {
                const int end = tokens_of<kHanded>(k, p, it);
                const int from = k.end > k.t ? k.t + (k.end - k.t + kC - 1) / kC * kC : k.t;
                const int row = p.Pv / 8;  // in pieces of 16 bytes
                uint4* to = reinterpret_cast<uint4*>(p.out) + ((long long)k.bh * p.S + from) * row + lane;
                uint4* const stop = to + (long long)(end - from) * row - lane;  // (not past `to` where the tokens go to the end)
#pragma unroll 1
                for (; to < stop; to += 32) __stcs(to, make_uint4(0, 0, 0, 0));
            }
        }
    }
    if (!ok) sh.gave_up = 1;
    griddep_launch_dependents();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 25) {
        tmem_relinquish();
        tmem_dealloc(tmem, 512);
    }
    if (tid == 0 && sh.gave_up && status) atomicExch(status, (int32_t)GDN_ERR_TIMEOUT);
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

std::atomic<int> g_stall[kMaxDevices];  // gdn_test_stall_prefill

template <bool kStatesOnly, bool kHanded>
gdn_status launch(const CUtensorMap (&m)[4], const LinearAttn& p, const LinearAttnSplit& s, int dev, int sms,
                  int32_t* status, cudaStream_t stream) {
    auto* kernel = linear_attn_tc_kernel<kStatesOnly, kHanded>;
    static std::atomic<int> launched{0};  // registers a thread of the block at launch
    int regs = launched.load(std::memory_order_relaxed);
    if (regs == 0) {
        cudaFuncAttributes a{};
        if (cudaFuncGetAttributes(&a, kernel) != cudaSuccess) return GDN_ERR_CUDA;
        launched.store(regs = a.numRegs, std::memory_order_relaxed);
    }
    static std::atomic<bool> allowed[kMaxDevices];
    // the roles' registers come out of what the block is launched with: short of that they would wait for ever
    if (regs * kThreads < kRegsSum) return GDN_ERR_CUDA;
    if (allow_smem(kernel, (int)kSmem, allowed, dev) != cudaSuccess) return GDN_ERR_CUDA;
    const int items = p.B * p.Hv * (kStatesOnly ? s.P - 1 : s.P);  // (at most 2^24 heads, of 64 segments)
    Items it{p.B * p.Hv, kStatesOnly ? s.P - 1 : s.P, s.P > 1 || kHanded ? s.len : p.S, divisor(p.Hv), divisor(p.Hv / p.Hk),
             0, 0, 0, nullptr};
    if (kHanded) {
        it.whole = it.heads / sms;
        it.rest = it.heads % sms;
        it.handed = s.handed;
        it.flags = s.flags;
        if (cudaMemsetAsync(s.flags, 0, linear_attn_flag_bytes(s.handed), stream) != cudaSuccess) return GDN_ERR_CUDA;
    }
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
    const int stall = g_stall[dev].load(std::memory_order_relaxed);
    return cudaLaunchKernelEx(&cfg, kernel, m[0], m[1], m[2], m[3], p, s, it, stall, status) == cudaSuccess ? GDN_OK
                                                                                                            : GDN_ERR_CUDA;
}

}  // namespace

void set_linear_attn_test_stall(int dev, int on) { g_stall[dev].store(on, std::memory_order_relaxed); }

gdn_status launch_linear_attn_tc(const LinearAttn& p, const LinearAttnSplit& s, int dev, int sms, int32_t* status,
                                 cudaStream_t stream) {
    CUtensorMap m[4];
    const long long hk = (long long)p.B * p.Hk, hv = (long long)p.B * p.Hv;
    if (!encode(&m[0], p.q, hk, p.S, p.Pk) || !encode(&m[1], p.k, hk, p.S, p.Pk) || !encode(&m[2], p.v, hv, p.S, p.Pv) ||
        !encode(&m[3], p.out, hv, p.S, p.Pv))
        return GDN_ERR_CUDA;
    if (s.P > 1) {
        const gdn_status e = launch<true, false>(m, p, s, dev, sms, status, stream);
        if (e != GDN_OK) return e;
        if (launch_linear_attn_combine(p, s, stream) != cudaSuccess) return GDN_ERR_CUDA;
    }
    if (s.handed) return launch<false, true>(m, p, s, dev, sms, status, stream);
    return launch<false, false>(m, p, s, dev, sms, status, stream);
}

}  // namespace gdn
