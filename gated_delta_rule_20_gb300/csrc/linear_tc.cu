// linear_tc.cu -- gdn_linear on the tensor cores (bf16, and e4m3 with scales): tcgen05 with
// fp32 accumulators in TMEM, operands by TMA.
//
// Both kernels issue the product transposed, D^T[n][m] = sum_k W[n][k] x[m][k]: 128 weight
// columns n lie on the MMA's M axis (TMEM lanes), the tokens m on its N axis.  So one token
// costs 16 MMA columns instead of 128 rows, a thread of the epilogue has one n (its bias and
// weight scale are registers), and a warp's stores of a token are 32 neighbouring outputs in
// any N, with no staging.  Gated, a CTA's 128 rows are 64 of the gate and the 64 of the up
// half that belong to them (two TMA boxes), so both factors of an output meet in the CTA.
//
// A slab is 128 bytes of K (64 bf16, 128 e4m3): the widest 128-byte-swizzled tile row.  W comes
// K-major ([N, K]) or, bf16 only, MN-major ([K, N], boxes of 64 columns); x K-major.  Boxes read
// zero past the edges, so ragged M, N and K need no other care than not storing past M and N.
//
// linear_small_kernel (few tokens; bound by the weight's bytes): one CTA per 128 columns, K
// split over a cluster of up to 8 CTAs so that the weight streams through every SM; the partial
// sums meet in shared memory, are added in the ranks' order (the same result every time) and leave
// through the epilogue of the rank that owns the token.
//
// linear_large_kernel (many tokens; bound by the tensor cores): persistent CTA pairs
// (cta_group::2) on tiles of 256 columns x up to 256 tokens; every CTA loads its 128 columns and
// half of the tokens.  Two accumulators in TMEM: the epilogue of one tile runs beside the next
// tile's products.  (fp32 by bf16 parts, at the end of the file, takes all of TMEM for one tile; fp32 outputs of long
// sums add up blocks of K, see block_of.)
//
// linear_joint_kernel (a few tiles and a long K): two to four such pairs on a tile, each with its part of K.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstring>
#include <mutex>
#include <type_traits>

#include "gdn_internal.h"
#include "linear_epilogue.cuh"
#include "sm100_ptx.cuh"

namespace gdn {
namespace {

using namespace ptx;

constexpr int kSlabBytes = 128;                  // bytes of K a stage
constexpr uint32_t kWBytes = 128 * kSlabBytes;   // a CTA's 128 weight columns of a slab
constexpr uint32_t kHalfW = kWBytes / 2;         // one box of 64
constexpr int kMaxStages = 12;
constexpr int kMaxAccs = 5;

struct TcArgs {
    LinearArgs a;
    int slabs, stages, bn;          // bn: MMA N (tokens of a tile)
    uint32_t stage_bytes, tmem_cols, idesc;
    int up;                         // gated: the weight column where the up half starts (see Operands)
    int splits;                     // small kernel: K splits (cluster size)
    bool wide_out;                  // small kernel: 4 outputs a store
    int tiles_n, tiles_m, group;    // large kernel: the tile grid, n tiles walked together
    bool staged;                    // large kernel: bf16 output (and residual) by TMA
    int32_t* status;
    int accs, starts[kMaxAccs];     // fp32 by parts: accumulators of a tile, from 1 on each from its first slab (else one)
    int plane;                      // fp32 by parts: elements of K from one part to the next
    int block, blocks, ring;        // slabs of a block of K, blocks of a tile (small kernel: of a CTA), accumulators
    const uint8_t* tops;            // fp32 by parts: see LinearMarks (null otherwise)
    int marks;
};

constexpr int kEpiWarps = 8;                    // two a TMEM lane quadrant, half of the columns each
constexpr int kThreads = 64 + 32 * kEpiWarps;   // and a warp for the loads, one for the products

struct SmallBars {
    uint64_t full[kMaxStages], empty[kMaxStages], done;
    uint64_t acc_full[2], acc_empty[2];  // blocks of K before the last
    uint32_t tmem;
    int abort;
    uint32_t tops[kThreads / 32];  // fp32 by parts: see parts_fit_all
};

// A place in the ring of stages: the stage and the parity of the barrier phase that its next use waits
// for.  (Kept by counting: a division by the runtime number of stages costs more than the wait.)
struct Ring {
    int s = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int stages) {
        if (++s == stages) {
            s = 0;
            phase ^= 1;
        }
    }
};

// The tensor cores truncate a sum at every step of 16 terms, always towards zero, so that a sum of K bf16 products of
// both signs is off by about K 1e-9 of the sums' norm (2.1e-6 at K = 2048 and 1.9e-5 at 16384; fp32 sums 4e-7 and
// 1.5e-6), and sums of one sign by up to 4e-9 K.  bf16 outputs round that away; for fp32 outputs K is worked off in
// blocks of at most 8 slabs (512 in bf16: 5e-7) in a ring of accumulators, and the epilogue warps add every block to
// the tile's sums, in registers, with rounding, while the next ones' products run (kernels with BLOCKED).  A CTA pair's
// tile has 192 tokens at the most then (96 sums a thread), one of the small kernel 64: two accumulators of those are
// the 128 columns of TMEM that its widest tile takes without blocks, so that two CTAs always find room on an SM.
// M = 16384, K = 4096, N = 2048 184 us (152 in one accumulator): tiles of 224 tokens are best there, and the products wait
// for the epilogue at a tile's end.
constexpr int kBlockSlabs = 8;
__host__ __device__ inline int block_of(int slabs, bool blocked) {
    const int blocks = blocked ? (slabs + kBlockSlabs - 1) / kBlockSlabs : 1;
    return (slabs + blocks - 1) / blocks;
}

// Adds a block's accumulator to the sums, the first `cols` (32, 64 or 96) columns of it.
__device__ __forceinline__ void add_block(float (&sum)[3][32], uint32_t acc, int cols) {
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        if (j * 32 >= cols) break;
        float v[32];
        tmem_ld32(acc + j * 32, v);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) sum[j][i] += v[i];
    }
}
// The same for 16 columns.
__device__ __forceinline__ void add_columns(float (&sum)[2][8], uint32_t acc) {
    float v[2][8];
    tmem_ld8(acc, v[0]);
    tmem_ld8(acc + 8, v[1]);
    tmem_wait_ld();
#pragma unroll
    for (int j = 0; j < 16; ++j) sum[j / 8][j % 8] += v[j / 8][j % 8];
}

// The accumulator of a tile that slab k goes to (fp32 by parts: its x1 w1; the small products go to accumulator 0).
__device__ __forceinline__ int acc_at(const TcArgs& t, int k) {
    int q = 0;
    for (int i = 1; i < t.accs; ++i) q += k >= t.starts[i];
    return q;
}
// The same for slab after slab from k_lo: one comparison a slab.
template <bool PARTS>
struct AccWalk {
    int q = 0, next = INT32_MAX;
    __device__ __forceinline__ AccWalk(const TcArgs& t, int k_lo) {
        if constexpr (PARTS) {
            q = acc_at(t, k_lo);
            look(t);
        }
    }
    __device__ __forceinline__ void look(const TcArgs& t) { next = q + 1 < t.accs ? t.starts[q + 1] : INT32_MAX; }
    // Slab k: whether it is the first of its accumulator.
    __device__ __forceinline__ bool step(const TcArgs& t, int k) {
        if (!PARTS || k != next) return false;
        ++q;
        look(t);
        return true;
    }
};

// The four 32-byte steps of K of one slab, of the weight's stage and x's.  KN: W is MN-major (boxes of 64
// columns, 2048 bytes a step).
template <bool F8, bool KN, bool PAIR>
__device__ __forceinline__ void mma_slab(uint32_t tmem, uint32_t w, uint32_t x, uint32_t idesc, bool first) {
    const uint64_t dw = KN ? make_sdesc(w, kHalfW, 1024) : make_sdesc(w, 16, 1024);
    const uint64_t dx = make_sdesc(x + kWBytes, 16, 1024);
#pragma unroll
    for (int k = 0; k < 4; ++k)
        mma_step<F8, PAIR>(tmem, sdesc_add(dw, k * (KN ? 2048 : 32)), sdesc_add(dx, k * 32), idesc, !first || k > 0);
}

// Waits for the stages of a slab, s, from `at` on (left at the last of them); false: given up.
template <bool PARTS>
__device__ __forceinline__ bool wait_slab(uint64_t* full, Ring& at, int stages, int* s, volatile int* abort_flag) {
#pragma unroll
    for (int p = 0; p < (PARTS ? 3 : 1); ++p) {
        if (p > 0) at.next(stages);
        s[p] = at.s;
        if (!mbar_wait_warp(&full[at.s], at.phase, abort_flag)) return false;
    }
    return true;
}

template <bool PAIR>
__device__ __forceinline__ void commit(uint64_t* bar) {
    if constexpr (PAIR)
        mma_commit_pair(bar);
    else
        mma_commit(bar);
}

// The products of one slab and the hand-back of its stages.  first: of this tile, main: of its accumulator.  By
// parts a slab is three stages, the third parts in the first: each stage is loaded once for its two to three
// products and handed back as early as their order allows.
template <bool F8, bool KN, bool PARTS, bool PAIR>
__device__ __forceinline__ void mma_stages(const TcArgs& t, uint32_t tmem, uint32_t sm, const int* at, uint64_t* empty,
                                           int acc, bool first, bool main) {
    const uint32_t s0 = sm + at[0] * t.stage_bytes;
    if constexpr (!PARTS) {
        mma_slab<F8, KN, PAIR>(tmem, s0, s0, t.idesc, main);
        commit<PAIR>(&empty[at[0]]);
    } else {
        const uint32_t s1 = sm + at[1] * t.stage_bytes, s2 = sm + at[2] * t.stage_bytes;
        mma_slab<F8, KN, PAIR>(tmem, s0, s2, t.idesc, first);  // w3 x1
        mma_slab<F8, KN, PAIR>(tmem, s2, s0, t.idesc, false);  // w1 x3
        commit<PAIR>(&empty[at[0]]);
        mma_slab<F8, KN, PAIR>(tmem, s1, s1, t.idesc, false);  // w2 x2
        mma_slab<F8, KN, PAIR>(tmem, s1, s2, t.idesc, false);  // w2 x1
        mma_slab<F8, KN, PAIR>(tmem, s2, s1, t.idesc, false);  // w1 x2
        commit<PAIR>(&empty[at[1]]);
        mma_slab<F8, KN, PAIR>(tmem + acc * t.bn, s2, s2, t.idesc, main);  // w1 x1
        commit<PAIR>(&empty[at[2]]);
    }
}

// The sum over the S ranks' partial sums (in the ranks' order) of 4 neighbouring columns a thread, and
// the epilogue, for the tokens rank, rank + S, ... of the tile.  e: epilogue thread; part: [token][128].
template <int S>
__device__ __forceinline__ void join_splits(const TcArgs& t, uint32_t part, int e, int rank, int n0, int m0, int cols) {
    const LinearArgs& a = t.a;
    const int width = a.gated ? 16 : 32;  // threads of a token
    const int n = n0 + e % width * 4;
    if (n >= a.N) return;
    const uint32_t at = part + e % width * 16;
    uint32_t peer[S];
#pragma unroll
    for (int q = 0; q < S; ++q) peer[q] = S > 1 ? map_to_rank(at, q) : at;
    for (int c = rank + S * (e / width); c < cols; c += S * (32 * kEpiWarps / width)) {
        float4 g[S], u[S];
#pragma unroll
        for (int q = 0; q < S; ++q) {
            g[q] = ld_cluster_f32x4(peer[q] + c * 512);
            if (a.gated) u[q] = ld_cluster_f32x4(peer[q] + c * 512 + 256);
        }
        const int m = m0 + c;
        const long long i = (long long)m * a.N + n;
        float v[4], w[4], r[4];
        if (a.res) {
#pragma unroll
            for (int j = 0; j < 4; ++j) r[j] = load_out(a, i + min(j, a.N - 1 - n));
        }
#pragma unroll
        for (int q = 1; q < S; ++q) {
            g[0].x += g[q].x, g[0].y += g[q].y, g[0].z += g[q].z, g[0].w += g[q].w;
            if (a.gated) u[0].x += u[q].x, u[0].y += u[q].y, u[0].z += u[q].z, u[0].w += u[q].w;
        }
        v[0] = g[0].x, v[1] = g[0].y, v[2] = g[0].z, v[3] = g[0].w;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = activate(a.act, affine(a, v[j], m, n + min(j, a.N - 1 - n)));
        if (a.gated) {
            w[0] = u[0].x, w[1] = u[0].y, w[2] = u[0].z, w[3] = u[0].w;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] *= affine(a, w[j], m, a.N + n + min(j, a.N - 1 - n));
        }
        if (a.res) {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] += r[j];
        }
        if (t.wide_out) {  // N a multiple of 4, the output aligned to 4 elements
            if (a.out_f32)
                *reinterpret_cast<float4*>(static_cast<float*>(a.out) + i) = make_float4(v[0], v[1], v[2], v[3]);
            else
                *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + i) =
                    make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n + j < a.N) store_out(a, i + j, v[j]);
        }
    }
}

// PARTS: an fp32 product by bf16 parts (several accumulators a tile, operands that parts may not fit).
// BLOCKED: several blocks of K (see block_of).
template <bool F8, bool KN, bool PARTS, bool BLOCKED>
__global__ void __launch_bounds__(kThreads, 2) linear_small_kernel(const __grid_constant__ CUtensorMap tm_w,
                                                           const __grid_constant__ CUtensorMap tm_x,
                                                           const __grid_constant__ TcArgs t) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const LinearArgs& a = t.a;
    constexpr int kSlabElems = F8 ? 128 : 64, kSlabStages = PARTS ? 3 : 1;
    const int stages = t.stages;
    SmallBars* bars = reinterpret_cast<SmallBars*>(sm + stages * t.stage_bytes);
    volatile int* abort_flag = &bars->abort;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = t.splits > 1 ? (int)cluster_rank() : 0;
    const int n0 = ((int)blockIdx.x / t.splits) * (a.gated ? 64 : 128);  // outputs of this tile
    const int n1 = a.gated ? t.up + n0 : n0 + 64;                        // weight column of the second box
    const int m0 = (int)blockIdx.y * t.bn;
    griddep_launch_dependents();  // the next kernel's CTAs may be set up beside this one (they wait as below)
    const int k_lo = (int)((long long)t.slabs * rank / t.splits), k_hi = (int)((long long)t.slabs * (rank + 1) / t.splits);

    if (warp == 0) {  // a barrier a lane
        if (lane < stages) {
            mbar_init(&bars->full[lane], 1);
            mbar_init(&bars->empty[lane], 1);
        } else if (BLOCKED && lane >= 16 && lane < 18) {
            mbar_init(&bars->acc_full[lane - 16], 1);
            mbar_init(&bars->acc_empty[lane - 16], kEpiWarps);
        } else if (lane == 30) {
            mbar_init(&bars->done, 1);
            bars->abort = 0;
        }
        fence_mbar_init();
        if (lane == 31) {
            tma_prefetch_desc(&tm_w);
            tma_prefetch_desc(&tm_x);
        }
        __syncwarp();
    }
    if (warp == 1) {
        tmem_alloc(&bars->tmem, t.tmem_cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem;
    griddep_wait();  // the preceding kernel's results; nothing of the caller's is read before
    const bool run = !PARTS || parts_fit_all<kThreads>(t.tops, t.marks, a.K, bars->tops);  // one answer for the whole grid

    if (warp == 0 && run) {  // TMA producer
        int loaded = 0, part = kSlabStages - 1, slab = k_lo * kSlabElems;
        Ring at;
        for (int i = 0; i < (k_hi - k_lo) * kSlabStages; ++i, at.next(stages)) {
            const int s = at.s, k = PARTS ? slab + part * t.plane : slab;
            if (i >= stages && !mbar_wait_warp(&bars->empty[s], at.phase ^ 1, abort_flag)) break;
            if (!PARTS || --part < 0) {
                part = kSlabStages - 1;
                slab += kSlabElems;
            }
            uint8_t* st = sm + s * t.stage_bytes;
            if (elect_one()) {
                mbar_arrive_expect_tx(&bars->full[s], t.stage_bytes);
                tma_load_3d(st, &tm_w, &bars->full[s], KN ? n0 : k, KN ? k : n0, 0);
                tma_load_3d(st + kHalfW, &tm_w, &bars->full[s], KN ? n1 : k, KN ? k : n1, 0);
                tma_load_3d(st + kWBytes, &tm_x, &bars->full[s], k, m0, 0);
            }
            __syncwarp();
            loaded = i + 1;
        }
        // every issued load has landed before the CTA can exit (bounded)
        for (int i = (loaded > stages ? loaded - stages : 0); i < loaded; ++i)
            (void)mbar_wait(&bars->full[i % stages], (i / stages) & 1);
    } else if (warp == 1 && run) {  // MMA issuer
        int issued = 0, block = 0, in = 0;  // the block of K, and the slab in it
        Ring at;
        AccWalk<PARTS> acc(t, k_lo);
        for (int i = 0; i < k_hi - k_lo; ++i, at.next(stages)) {
            int s[kSlabStages];
            if (BLOCKED && in == t.block) {
                if (++block >= 2 && !mbar_wait_warp(&bars->acc_empty[block & 1], ((block - 2) >> 1) & 1, abort_flag)) break;
                in = 0;
            }
            if (!wait_slab<PARTS>(bars->full, at, stages, s, abort_flag)) break;
            tc_fence_after();
            const bool main = acc.step(t, k_lo + i) || (BLOCKED ? in : i) == 0;
            if (elect_one()) {
                mma_stages<F8, KN, PARTS, false>(t, BLOCKED ? tmem + (block & 1) * t.bn : tmem, smem_u32(sm), s, bars->empty,
                                                 acc.q, i == 0, main);
                if (i + 1 == k_hi - k_lo)
                    mma_commit(&bars->done);
                else if (BLOCKED && in + 1 == t.block)
                    mma_commit(&bars->acc_full[block & 1]);
            }
            __syncwarp();
            ++in;
            issued = (i + 1) * kSlabStages;
        }
        if (issued < (k_hi - k_lo) * kSlabStages && issued > 0)  // gave up: what was issued ends first (bounded)
            (void)mbar_wait(&bars->empty[(issued - 1) % stages], ((issued - 1) / stages) & 1);
    }
    __syncwarp();
    // The partial sums of this CTA's K range, [token][128 columns] over the stages (all of them read).
    float* part = reinterpret_cast<float*>(sm);
    const int cols = min(t.bn, a.M - m0);
    const int e = tid - 64;  // epilogue thread
    bool ok = false;
    if (warp >= 2 && run) {
        const int row = (warp & 3) * 32 + lane, blocks = BLOCKED ? (k_hi - k_lo + t.block - 1) / t.block : 1;
        const uint32_t base = tmem + ((uint32_t)(row & ~31) << 16);
        const int first = (warp - 2) / 4 * 16;  // this warp's columns: first, first + 32, ... and the 15 behind each
        ok = true;
        float sum[2][2][8];  // BLOCKED: of the blocks of K (at most 64 columns)
        if constexpr (BLOCKED) {
#pragma unroll
            for (int j = 0; j < 32; ++j) sum[j / 16][j / 8 % 2][j % 8] = 0.f;
            for (int q = 0; q + 1 < blocks; ++q) {
                ok = mbar_wait_warp(&bars->acc_full[q & 1], (q >> 1) & 1, abort_flag);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (first + 32 * h < cols) add_columns(sum[h], base + (q & 1) * t.bn + first + 32 * h);
                tc_fence_before();
                __syncwarp();
                if (lane == 0 && q + 2 < blocks) mbar_arrive(&bars->acc_empty[q & 1]);
            }
        }
        ok = __all_sync(0xffffffffu, mbar_wait_or_abort(&bars->done, 0, abort_flag)) && ok;  // one answer a warp
        tc_fence_after();
        if (ok) {
            if constexpr (BLOCKED) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int c0 = first + 32 * h;
                    if (c0 >= cols) break;
                    add_columns(sum[h], base + ((blocks - 1) & 1) * t.bn + c0);
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (c0 + j < cols) part[(c0 + j) * 128 + row] = sum[h][j / 8][j % 8];
                }
            }
            const uint32_t lanes = base;
            for (int c0 = first; !BLOCKED && c0 < cols; c0 += 32) {  // (columns come in 16s: t.bn)
                float v[2][8];
                tmem_ld8(lanes + c0, v[0]);
                tmem_ld8(lanes + c0 + 8, v[1]);
                tmem_wait_ld();
                if constexpr (PARTS) {  // and of the accumulators that this rank's slabs went to
                    float sum[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) sum[j] = v[j / 8][j % 8];
                    for (int q = acc_at(t, k_lo); q <= acc_at(t, k_hi - 1); ++q) {
                        tmem_ld8(lanes + q * t.bn + c0, v[0]);
                        tmem_ld8(lanes + q * t.bn + c0 + 8, v[1]);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j) sum[j] += v[j / 8][j % 8];
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j / 8][j % 8] = sum[j];
                }
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (c0 + j < cols) part[(c0 + j) * 128 + row] = v[j / 8][j % 8];
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    if (t.splits > 1)
        cluster_sync();
    else
        __syncthreads();
    if (ok) {
        switch (t.splits) {
            case 1: join_splits<1>(t, smem_u32(part), e, rank, n0, m0, cols); break;
            case 2: join_splits<2>(t, smem_u32(part), e, rank, n0, m0, cols); break;
            case 4: join_splits<4>(t, smem_u32(part), e, rank, n0, m0, cols); break;
            default: join_splits<8>(t, smem_u32(part), e, rank, n0, m0, cols); break;
        }
    }
    __syncwarp();
    // a CTA's shared memory stays until every rank has read it
    if (t.splits > 1)
        cluster_sync_relaxed();
    else
        __syncthreads();
    if (tid == 0 && bars->abort) atomicExch(t.status, (int32_t)GDN_ERR_TIMEOUT);
    if (warp == 1) tmem_dealloc(tmem, t.tmem_cols);
}

// ------------------------------------------------------------------ many tokens
constexpr int kLargeStages = 10;
constexpr int kMaxRing = 4;                        // accumulators of a CTA pair (two, unless BLOCKED)
constexpr uint32_t kSwapBytes = 4 * 2 * 2 * 16 * 32 * 4;  // gated: 4 warp pairs x 2 turns x 2 ways x 16 values x 32 lanes
constexpr uint32_t kBoxRow = 128;                  // a staged output row: 64 bf16 columns

struct LargeBars {
    uint64_t full[kLargeStages], empty[kLargeStages];  // full: the leader's are used
    uint64_t acc_full[kMaxRing], acc_empty[kMaxRing];  // acc_empty: the leader's are used
    uint64_t res_full[kEpiWarps / 2];                  // staged residual boxes
    uint32_t tmem;
    int abort;
    uint32_t tops[kThreads / 32];                      // fp32 by parts: see parts_fit_all
};

// A tile's tokens are worked off in chunks of 32, the first half of them (rounded up) by the first four
// epilogue warps, the rest by the others: this warp's first chunk and their number.
__device__ __forceinline__ int first_chunk(const TcArgs& t, int half) { return half ? (t.bn / 32 + 1) / 2 : 0; }
__device__ __forceinline__ int chunks_of(const TcArgs& t, int half) { return (t.bn / 32 + 1 - half) / 2; }

// Shared memory of the staged output boxes: one a chunk, of 32 tokens (gated 16) x 64 columns, for two warps.
__host__ __device__ inline uint32_t box_bytes(const TcArgs& t) {
    return t.staged ? kEpiWarps / 2 * ((t.bn / 32 + 1) / 2) * (t.a.gated ? 16 : 32) * kBoxRow : 0;
}

// The tile of a pair's turn: n tiles walk in groups of t.group, tokens inside a group, so that the
// tiles that run at once share weights and tokens in L2.
__device__ __forceinline__ void tile_at(const TcArgs& t, int i, int* n, int* m) {
    const int g = i / (t.group * t.tiles_m), in = i - g * t.group * t.tiles_m;
    const int width = min(t.group, t.tiles_n - g * t.group);
    *m = in / width;
    *n = g * t.group + in - *m * width;
}

// A pair's turns: its tiles, or their blocks of K.  They take the two accumulators alternately; fp32 by parts takes all of
// TMEM for every tile.  The (first) accumulator of a turn, and how many turns have had it before.
template <bool PARTS>
__device__ __forceinline__ int acc_of(int turn) { return PARTS ? 0 : turn & 1; }
template <bool PARTS>
__device__ __forceinline__ int acc_use(int turn) { return PARTS ? turn : turn >> 1; }

// The tiles of a pair in turn, for a converged warp: every lane works out one of the next 32 (the
// divisions take a few hundred cycles, which would stall the loads at every tile), and hands it out.
struct Tiles {
    int n, m;
    __device__ __forceinline__ void get(const TcArgs& t, int turn, int pair, int pairs, int tiles, int* tn, int* tm) {
        if ((turn & 31) == 0) {
            const int mine = pair + (turn + (int)(threadIdx.x & 31)) * pairs;
            tile_at(t, mine < tiles ? mine : 0, &n, &m);
        }
        *tn = __shfl_sync(0xffffffffu, n, turn & 31);
        *tm = __shfl_sync(0xffffffffu, m, turn & 31);
    }
};

// The residual of tokens m0 .. m0 + C - 1 at column n < N, raw (the last row again past M, which is
// not stored): independent loads, issued well before they are used.
template <int C>
__device__ __forceinline__ void load_residual(const LinearArgs& a, uint32_t (&r)[C], int m0, int n) {
    const int last = a.M - 1 - m0;
    if (last < 0) return;
    const long long at = (long long)m0 * a.N + n;
    if (a.out_f32) {
        const uint32_t* p = static_cast<const uint32_t*>(a.res) + at;
#pragma unroll
        for (int j = 0; j < C; ++j) r[j] = p[(long long)min(j, last) * a.N];
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(a.res) + at;
#pragma unroll
        for (int j = 0; j < C; ++j) r[j] = (uint32_t)p[(long long)min(j, last) * a.N] << 16;  // bf16 -> fp32 bits
    }
}

// C tokens of one output column n: activation, gate (u, or null), residual (raw), rounding, store.
template <int C>
__device__ __forceinline__ void finish(const LinearArgs& a, float (&v)[C], const float* u, const uint32_t (&r)[C], int m0,
                                       int n) {
    activate_all<C>(a.act, v);
    if (u) {
#pragma unroll
        for (int j = 0; j < C; ++j) v[j] *= u[j];
    }
    if (a.res) {
#pragma unroll
        for (int j = 0; j < C; ++j) v[j] += __uint_as_float(r[j]);
    }
    const long long at = (long long)m0 * a.N + n;
    const int rows = a.M - m0;
    if (a.out_f32) {
        float* o = static_cast<float*>(a.out) + at;
        if (rows >= C) {
#pragma unroll
            for (int j = 0; j < C; ++j) o[(long long)j * a.N] = v[j];
        } else {
#pragma unroll
            for (int j = 0; j < C; ++j)
                if (j < rows) o[(long long)j * a.N] = v[j];
        }
    } else {
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out) + at;
        if (rows >= C) {
#pragma unroll
            for (int j = 0; j < C; ++j) o[(long long)j * a.N] = __float2bfloat16_rn(v[j]);
        } else {
#pragma unroll
            for (int j = 0; j < C; ++j)
                if (j < rows) o[(long long)j * a.N] = __float2bfloat16_rn(v[j]);
        }
    }
}

// The epilogue warps of linear_large_kernel, for any output: every tile of the pair, 32 tokens at a time.  The first
// residual values of a tile are loaded before its products are done, the next chunk's before this
// one's are used.
// A tile's blocks of K added up, from the accumulator `at` of the ring on; the sums are left in the last block's, from
// where they are finished as those of other tiles.  left: blocks of this and later tiles of the pair.  (Not inlined: the
// 96 sums leave no registers for what the epilogue has there, which went to local memory at every block.)
__device__ __noinline__ bool add_blocks(LargeBars* bars, uint32_t base, int bn, int ring, int cols, Ring at, int blocks,
                                        int left) {
    float sum[3][32];
#pragma unroll
    for (int j = 0; j < 96; ++j) sum[j / 32][j % 32] = 0.f;
    for (int q = 0;; ++q) {
        if (!mbar_wait_warp(&bars->acc_full[at.s], at.phase, &bars->abort)) return false;
        tc_fence_after();
        add_block(sum, base + at.s * bn, cols);
        if (q + 1 == blocks) break;
        tc_fence_before();
        __syncwarp();
        if ((threadIdx.x & 31) == 0 && q + ring < left)
            mbar_arrive_cluster_relaxed(map_to_rank(smem_u32(&bars->acc_empty[at.s]), 0));
        at.next(ring);
    }
#pragma unroll
    for (int j = 0; j < 3; ++j)
        if (j * 32 < cols) tmem_st32(base + at.s * bn + j * 32, sum[j]);
    tmem_wait_st();
    return true;
}

// BLOCKED: tiles of several blocks of K (see block_of).
template <bool GATED, bool PARTS, bool BLOCKED>
__device__ __forceinline__ void epilogue(const TcArgs& t, LargeBars* bars, float* swap, uint32_t tmem, int rank, int pair,
                                         int pairs, int tiles) {
    constexpr int C = GATED ? 16 : 32;  // tokens of a chunk that this warp finishes
    const LinearArgs& a = t.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quad = warp & 3, half = (warp - 2) >> 2;
    const int c_lo = first_chunk(t, half) * 32, hc = chunks_of(t, half) * 32;  // this warp's columns of the tile
    const int row = quad * 32 + lane;
    // gated: rows 0 .. 63 (quadrants 0, 1) are the gate's, the others the up half's; a warp of each
    // exchange their factors, gate rows finish a chunk's first 16 tokens and up rows its last 16
    const bool up = GATED && quad >= 2;
    const int own = up ? 16 : 0;
    const uint32_t pair_bar = 1 + (quad & 1) + 2 * half;
    float* ex = swap + ((quad & 1) + 2 * half) * (2 * 2 * 16 * 32) + lane;
    volatile int* abort_flag = &bars->abort;
    const uint32_t done0 = map_to_rank(smem_u32(&bars->acc_empty[0]), 0);
    const uint32_t done1 = map_to_rank(smem_u32(&bars->acc_empty[1]), 0);
    int turn = 0, flip = 0;
    const int turns = (tiles - pair + pairs - 1) / pairs;
    Ring acc_at;  // BLOCKED: of the accumulators
    Tiles walk;
    for (int tile = pair; tile < tiles; tile += pairs, ++turn) {
        int tn, tm;
        walk.get(t, turn, pair, pairs, tiles, &tn, &tm);
        // this thread's weight column and the output that it belongs to
        const int n = (tn * 2 + rank) * (GATED ? 64 : 128) + (GATED ? row & 63 : row);
        const int col = up ? a.N + n : n;
        const bool live = n < a.N;
        const float ws = a.w_scale && live ? a.w_scale[col] : 1.f;
        const float bias = a.bias && live ? a.bias[col] : 0.f;
        const int m_lo = tm * t.bn + c_lo;
        uint32_t res[C];
        const uint32_t base = tmem + c_lo + ((uint32_t)(quad * 32) << 16);
        bool ok = true;
        const int left = (turns - turn) * t.blocks;
        if constexpr (BLOCKED) {
            ok = add_blocks(bars, base, t.bn, t.ring, hc, acc_at, t.blocks, left);
            for (int q = 0; q + 1 < t.blocks; ++q) acc_at.next(t.ring);
        }
        const int b = BLOCKED ? acc_at.s : acc_of<PARTS>(turn);
        if (a.res && live) load_residual<C>(a, res, m_lo + own, n);
        if (!BLOCKED) ok = mbar_wait_warp(&bars->acc_full[b], acc_use<PARTS>(turn) & 1, abort_flag);
        // one answer for both warps of a gated pair, which meet at a barrier below
        if (GATED ? named_bar_any(pair_bar, 64, !ok) : !ok) break;
        tc_fence_after();
        const uint32_t src = base + b * t.bn;
#pragma unroll 1
        for (int c = 0; c < hc; c += 32) {
            const int m0 = m_lo + c;
            float v[32];
            tmem_ld32(src + c, v);
            uint32_t r[C];
#pragma unroll
            for (int j = 0; j < C; ++j) r[j] = res[j];
            if (a.res && live && c + 32 < hc) load_residual<C>(a, res, m0 + 32 + own, n);
            tmem_wait_ld();
            for (int q = 1; PARTS && q < t.accs; ++q) {
#pragma unroll
                for (int i = 0; i < 32; i += 8) {
                    float w[8];
                    tmem_ld8(src + q * t.bn + c + i, w);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[i + j] += w[j];
                }
            }
            // read: a later product may overwrite it
            if (c + 32 >= hc && (BLOCKED ? t.blocks - 1 + t.ring < left : turn + (PARTS ? 1 : 2) < turns)) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (BLOCKED)
                        mbar_arrive_cluster_relaxed(map_to_rank(smem_u32(&bars->acc_empty[b]), 0));
                    else
                        mbar_arrive_cluster(b ? done1 : done0);
                }
            }
            if (a.x_scale) {
                const float mine = m0 + lane < a.M ? a.x_scale[m0 + lane] : 0.f;
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] *= __shfl_sync(0xffffffffu, mine, j) * ws;
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] += bias;
            if constexpr (!GATED) {
                if (live) finish<32>(a, v, nullptr, r, m0, n);
            } else {
                float* box = ex + flip * (2 * 16 * 32);  // used in turns, so that one barrier a chunk is enough
                flip ^= 1;
#pragma unroll
                for (int j = 0; j < 16; ++j) box[(own + j) * 32] = up ? v[j] : v[16 + j];
                named_bar_sync(pair_bar, 64);
                float g[16], w[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float other = box[((16 - own) + j) * 32];
                    g[j] = up ? other : v[j];
                    w[j] = up ? v[16 + j] : other;
                }
                if (live) finish<16>(a, g, w, r, m0 + own, n);
            }
        }
        if (BLOCKED) acc_at.next(t.ring);
    }
}

// The same for bf16 outputs that TMA can store (N a multiple of 8, 16-byte aligned).  Two warps (64 TMEM
// lanes) fill boxes of a chunk's 32 tokens.  They read TMEM in the layout of 8x8 fragments, in which a
// thread has pairs of neighbouring tokens: packed to bf16, four fragments a stmatrix land transposed, as a
// row of 64 columns (128 bytes, a whole line) a token, with an eighth of the shared-memory stores that
// single elements take and no address arithmetic; a TMA store takes the box away (and clips it to the
// matrix).  The residual comes the same way back: a TMA load into the box while the tile's products run,
// and ldmatrix.  The two warps meet twice a tile (boxes free, boxes full).
template <bool GATED>
__device__ __forceinline__ void epilogue_staged(const TcArgs& t, const CUtensorMap* tm_out, const CUtensorMap* tm_res,
                                                LargeBars* bars, uint8_t* boxes, float* swap, uint32_t tmem, int rank,
                                                int pair, int pairs, int tiles) {
    constexpr int kTokens = GATED ? 16 : 32;  // of a chunk's 32 tokens, those that this warp finishes
    constexpr int kPieces = kTokens / 8;      // fragments of 8 tokens among them
    constexpr uint32_t kBoxBytes = kTokens * kBoxRow;
    const LinearArgs& a = t.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quad = warp & 3, half = (warp - 2) >> 2, duo = quad >> 1;
    const bool issuer = (quad & 1) == 0;  // of the two warps of a box
    const bool up = GATED && duo == 1;
    const int own = up ? 16 : 0;  // gated: gate rows finish a chunk's first 16 tokens, up rows the others
    // the warps that share boxes (gated: all four of a half of the chunks); the warps of a gate and its up rows
    const uint32_t box_bar = GATED ? 1 + half : 1 + half * 2 + duo, box_threads = GATED ? 128 : 64;
    const uint32_t swap_bar = 5 + half * 2 + (quad & 1);
    float* sw = swap + (half * 2 + (quad & 1)) * (2 * 2 * 16 * 32) + lane;  // gated: [turn][up][16 values][lane]
    const int c_lo = first_chunk(t, half) * 32, chunks = chunks_of(t, half);
    uint8_t* box = boxes + (half * 2 + duo) * ((t.bn / 32 + 1) / 2) * kBoxBytes;
    uint64_t* res_full = &bars->res_full[half * 2 + duo];
    volatile int* abort_flag = &bars->abort;
    const uint32_t done0 = map_to_rank(smem_u32(&bars->acc_empty[0]), 0);
    const uint32_t done1 = map_to_rank(smem_u32(&bars->acc_empty[1]), 0);
    const bool has_res = a.res != nullptr;
    Tiles walk;
    // first column of the boxes and first token of these chunks of a tile
    auto place = [&](int turn, int* n, int* m) {
        int tn, tm;
        walk.get(t, turn, pair, pairs, tiles, &tn, &tm);
        *n = (tn * 2 + rank) * (GATED ? 64 : 128) + (GATED ? 0 : duo * 64);
        *m = tm * t.bn + c_lo;
    };
    // a tile's boxes here that hold something of the matrix
    auto boxes_in = [&](int n, int m) { return n < a.N ? max(0, min(chunks, (a.M - m - own + 31) / 32)) : 0; };
    auto fetch_residual = [&](int n, int m) {  // one lane
        const int count = has_res ? boxes_in(n, m) : 0;
        if (count == 0) return;
        mbar_arrive_expect_tx(res_full, count * kBoxBytes);
        for (int i = 0; i < count; ++i) tma_load_3d(box + i * kBoxBytes, tm_res, res_full, n, m + i * 32 + own, 0);
    };
    auto load_scales = [&](float (&xs)[8], int m) {  // of tokens m + 8 k + 2 (lane % 4) + {0, 1}
#pragma unroll
        for (int k = 0; k < 8; ++k) xs[k] = a.x_scale[min(m + 8 * (k >> 1) + 2 * (lane & 3) + (k & 1), a.M - 1)];
    };
    int n_box = a.N, m_tile = a.M, turn = 0, flip = 0;
    uint32_t phase = 0;  // parity of the next residual
    bool ok = true;
    if (pair < tiles) place(0, &n_box, &m_tile);
    if (issuer && elect_one()) fetch_residual(n_box, m_tile);
    __syncwarp();
    bool in_flight = has_res && boxes_in(n_box, m_tile) > 0;  // the tile's residual has been asked for, not waited for
    for (int tile = pair; tile < tiles; tile += pairs, ++turn) {
        const int b = turn & 1, live = boxes_in(n_box, m_tile);
        int n_next = a.N, m_next = a.M;
        if (tile + pairs < tiles) place(turn + 1, &n_next, &m_next);
        float ws[2][2], bias[2][2], xs[8];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const int n = n_box + (quad & 1) * 32 + 16 * h + 8 * g + (lane >> 2);
                const int col = up ? a.N + n : n;
                ws[h][g] = a.w_scale && n < a.N ? a.w_scale[col] : 1.f;
                bias[h][g] = a.bias && n < a.N ? a.bias[col] : 0.f;
            }
        if (a.x_scale) load_scales(xs, m_tile);
        if (issuer && !has_res) {  // the last tile's stores have read the boxes (with a residual: waited for below)
            if (elect_one()) tma_store_wait_read0();
            __syncwarp();
        }
        ok = __all_sync(0xffffffffu, mbar_wait_or_abort(&bars->acc_full[b], (turn >> 1) & 1, abort_flag)) && ok;
        if (in_flight) {
            ok = mbar_wait_warp(res_full, phase, abort_flag) && ok;
            if (ok) {
                phase ^= 1;
                in_flight = false;
            }
        }
        if (named_bar_any(box_bar, box_threads, !ok)) break;  // the boxes are free; and one answer for all who meet here
        tc_fence_after();
        // (Two chunks at a time, or the next one read ahead, gain nothing: the code of an activation over 64 values
        // is fetched anew at every tile.  M = 16384, K = 512, N = 4096 with GELU: 96 us so, 152 with two.)
#pragma unroll 1
        for (int chunk = 0; chunk < chunks; ++chunk) {
            float v[2][16];  // 16 columns (TMEM lanes) each
#pragma unroll
            for (int h = 0; h < 2; ++h)
                tmem_ld16x256_x4(tmem + b * t.bn + c_lo + chunk * 32 + ((uint32_t)(quad * 32 + 16 * h) << 16), v[h]);
            tmem_wait_ld();
            // the accumulator is read (told only where it is used again: the arrival waits for earlier writes, 0.5 us)
            if (chunk == chunks - 1 && tile + 2 * pairs < tiles) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(b ? done1 : done0);
            }
            if (a.x_scale) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[h][j] *= xs[2 * (j >> 2) + (j & 1)] * ws[h][(j >> 1) & 1];
                if (chunk + 1 < chunks) load_scales(xs, m_tile + (chunk + 1) * 32);
            }
            if (a.bias) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[h][j] += bias[h][(j >> 1) & 1];
            }
            if constexpr (!GATED) {
                activate_all<16, true>(a.act, v[0]);
                activate_all<16, true>(a.act, v[1]);
            } else {
                // gate rows hand over their last 16 tokens and up rows their first 16, through two buffers in turn
                // (the barrier of the exchange in between tells that a buffer has been read)
                float* ex = sw + flip * (2 * 16 * 32);
                flip ^= 1;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < 8; ++j) ex[(own + 8 * h + j) * 32] = up ? v[h][j] : v[h][8 + j];
                named_bar_sync(swap_bar, 64);
                float g[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) g[j] = up ? ex[j * 32] : v[j >> 3][j & 7];
                activate_all<16, true>(a.act, g);
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j >> 3][j & 7] = g[j] * (up ? v[j >> 3][8 + (j & 7)] : ex[(16 + j) * 32]);
            }
            if (chunk < live) {
                const uint32_t at = smem_u32(box + chunk * kBoxBytes);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int k = 0; k < kPieces; k += 2) {
                        // matrix lane / 8 of the four: tokens 8 (k + its high bit), columns 16 h + 8 (its low bit)
                        const uint32_t token = 8 * (k + (lane >> 4)) + (lane & 7);
                        const uint32_t column = 4 * (quad & 1) + 2 * h + ((lane >> 3) & 1);  // in pieces of 8
                        const uint32_t addr = at + token * kBoxRow + ((column ^ (token & 7)) << 4);
                        float* f = &v[h][4 * k];
                        if (has_res) {
                            uint32_t r[4];
                            ldmatrix_x4_trans(addr, r);
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                f[2 * q] += bf16lo_to_f32(r[q]);
                                f[2 * q + 1] += bf16hi_to_f32(r[q]);
                            }
                        }
                        stmatrix_x4_trans(addr, pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                                          pack_bf16x2(f[6], f[7]));
                    }
                fence_proxy_async_smem();
            }
        }
        named_bar_sync(box_bar, box_threads);  // the boxes are full
        if (issuer && elect_one()) {
            for (int i = 0; i < live; ++i) tma_store_3d(tm_out, box + i * kBoxBytes, n_box, m_tile + i * 32 + own, 0);
            tma_store_commit();
            if (has_res) {  // the next tile's residual takes the boxes as soon as they are read
                tma_store_wait_read0();
                fetch_residual(n_next, m_next);
            }
        }
        __syncwarp();
        n_box = n_next;
        m_tile = m_next;
        in_flight = has_res && boxes_in(n_box, m_tile) > 0;
    }
    if (in_flight) (void)mbar_wait(res_full, phase);  // gave up: the load lands first (bounded)
    __syncwarp();
    if (issuer && elect_one()) tma_store_wait_read0();
    __syncwarp();
}

template <bool F8, bool KN, bool PARTS, bool BLOCKED>
__global__ void __launch_bounds__(kThreads, 1)
    linear_large_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                        const __grid_constant__ CUtensorMap tm_out, const __grid_constant__ CUtensorMap tm_res,
                        const __grid_constant__ TcArgs t) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const LinearArgs& a = t.a;
    constexpr int kSlabElems = F8 ? 128 : 64, kSlabStages = PARTS ? 3 : 1;
    const int stages = t.stages;
    uint8_t* boxes = sm + stages * t.stage_bytes;
    float* swap = reinterpret_cast<float*>(boxes + box_bytes(t));
    LargeBars* bars = reinterpret_cast<LargeBars*>(boxes + box_bytes(t) + (a.gated ? kSwapBytes : 0));
    volatile int* abort_flag = &bars->abort;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)cluster_rank();
    const int tiles = t.tiles_n * t.tiles_m, pairs = (int)gridDim.x / 2, pair = (int)blockIdx.x / 2;
    const int per = a.gated ? 64 : 128;  // outputs of a CTA
    griddep_launch_dependents();  // as in the small kernel

    if (warp == 0) {  // (a barrier a lane: one after another they were 0.1 us)
        if (lane < stages) {
            mbar_init(&bars->full[lane], 1);
            mbar_init(&bars->empty[lane], 1);
        } else if (lane >= 16 && lane < (BLOCKED ? 16 + kMaxRing : 18)) {
            mbar_init(&bars->acc_full[lane - 16], 1);
            mbar_init(&bars->acc_empty[lane - 16], 2 * kEpiWarps);
        } else if (lane >= 20 && lane < 20 + kEpiWarps / 2) {
            mbar_init(&bars->res_full[lane - 20], 1);
        } else if (lane == 30) {
            bars->abort = 0;
        }
        fence_mbar_init();
        if (lane == 31) {
            tma_prefetch_desc(&tm_w);
            tma_prefetch_desc(&tm_x);
        }
        __syncwarp();
    }
    if (warp == 1) tmem_alloc_pair(&bars->tmem, t.tmem_cols);
    tc_fence_before();
    __syncthreads();
    cluster_sync_relaxed();  // the peer's barriers are initialised (fence_mbar_init)
    tc_fence_after();
    const uint32_t tmem = bars->tmem;
    griddep_wait();
    const bool run = !PARTS || parts_fit_all<kThreads>(t.tops, t.marks, a.K, bars->tops);  // one answer for the whole grid

    if (!run) {
    } else if (warp == 0) {  // TMA producer: this CTA's columns and its half of the tokens
        int i = 0;    // slabs loaded
        bool live = true;
        Tiles walk;
        Ring at;
        int turn = 0;
        for (int tile = pair; tile < tiles && live; tile += pairs, ++turn) {
            int tn, tm;
            walk.get(t, turn, pair, pairs, tiles, &tn, &tm);
            const int n0 = (tn * 2 + rank) * per, n1 = a.gated ? t.up + n0 : n0 + 64;
            const int m0 = tm * t.bn + rank * (t.bn / 2);
            int part = kSlabStages - 1, slab = 0;
            for (int j = 0; j < t.slabs * kSlabStages; ++j, ++i, at.next(stages)) {
                const int s = at.s, k = PARTS ? slab + part * t.plane : slab;
                if (i >= stages && !mbar_wait_warp(&bars->empty[s], at.phase ^ 1, abort_flag)) {
                    live = false;
                    break;
                }
                if (!PARTS || --part < 0) {
                    part = kSlabStages - 1;
                    slab += kSlabElems;
                }
                uint8_t* st = sm + s * t.stage_bytes;
                if (elect_one()) {
                    if (rank == 0) mbar_arrive_expect_tx(&bars->full[s], 2 * t.stage_bytes);
                    const uint32_t bar = map_to_rank(smem_u32(&bars->full[s]), 0);
                    tma_load_3d_pair(st, &tm_w, bar, KN ? n0 : k, KN ? k : n0, 0);
                    tma_load_3d_pair(st + kHalfW, &tm_w, bar, KN ? n1 : k, KN ? k : n1, 0);
                    tma_load_3d_pair(st + kWBytes, &tm_x, bar, k, m0, 0);
                }
                __syncwarp();
            }
        }
        // the leader sees both CTAs' loads land before the pair can exit (bounded)
        if (rank == 0)
            for (int j = (i > stages ? i - stages : 0); j < i; ++j)
                (void)mbar_wait(&bars->full[j % stages], (j / stages) & 1);
    } else if (warp == 1) {
        if (rank == 0) {  // MMA issuer of the pair
            int i = 0, turn = 0;
            Ring at, acc_at;  // acc_at: of the accumulators, BLOCKED
            bool live = true;
            for (int tile = pair; tile < tiles && live; tile += pairs) {
                AccWalk<PARTS> acc(t, 0);
                int b = 0, end = 0;  // the turn's accumulator and the end of its slabs
                for (int k = 0; k < t.slabs; ++k, i += kSlabStages, at.next(stages)) {
                    const bool first = BLOCKED ? k == end : k == 0;
                    if (first) {
                        const bool used = BLOCKED ? turn >= t.ring : acc_use<PARTS>(turn) >= 1;
                        const uint32_t phase = BLOCKED ? acc_at.phase : acc_use<PARTS>(turn) & 1;
                        b = BLOCKED ? acc_at.s : acc_of<PARTS>(turn);
                        end = BLOCKED ? min(k + t.block, t.slabs) : t.slabs;
                        ++turn;
                        if (BLOCKED) acc_at.next(t.ring);
                        if (used && !mbar_wait_warp(&bars->acc_empty[b], phase ^ 1, abort_flag)) {
                            live = false;
                            break;
                        }
                        tc_fence_after();
                    }
                    int s[kSlabStages];
                    if (!wait_slab<PARTS>(bars->full, at, stages, s, abort_flag)) {
                        live = false;
                        break;
                    }
                    tc_fence_after();
                    const bool main = acc.step(t, k) || first;
                    if (elect_one()) {
                        mma_stages<F8, KN, PARTS, true>(t, tmem + b * t.bn, smem_u32(sm), s, bars->empty, acc.q, k == 0,
                                                        main);
                        if (k + 1 == end) mma_commit_pair(&bars->acc_full[b]);
                    }
                    __syncwarp();
                }
            }
            if (i > 0) (void)mbar_wait(&bars->empty[(i - 1) % stages], ((i - 1) / stages) & 1);  // all products are done
        }
    } else if (!PARTS && !BLOCKED && t.staged) {
        if (a.gated)
            epilogue_staged<true>(t, &tm_out, &tm_res, bars, boxes, swap, tmem, rank, pair, pairs, tiles);
        else
            epilogue_staged<false>(t, &tm_out, &tm_res, bars, boxes, swap, tmem, rank, pair, pairs, tiles);
    } else if (a.gated) {
        epilogue<true, PARTS, BLOCKED>(t, bars, swap, tmem, rank, pair, pairs, tiles);
    } else {
        epilogue<false, PARTS, BLOCKED>(t, bars, swap, tmem, rank, pair, pairs, tiles);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync_relaxed();
    if (tid == 0 && bars->abort) atomicExch(t.status, (int32_t)GDN_ERR_TIMEOUT);
    __syncwarp();
    if (warp == 1) tmem_dealloc_pair(tmem, t.tmem_cols);
    cluster_sync_relaxed();  // neither CTA exits while the pair's TMEM is being freed
}

// ------------------------------------------------------------------ a few tiles, K split over pairs
// One tile a cluster of `splits` CTA pairs, each with its part of K; then pair q finishes the 32-token chunks
// q, q + splits, ... of the tile: every pair sends its sums of the others' chunks into their shared memory (the
// stages, which are free by then), and adds what it gets in the pairs' order.
//
// Bound as linear_large_kernel, by the weight's and the tokens' way from L2; with fewer tiles than pairs of SMs the
// parts of K fill the others, or allow larger tiles.
constexpr uint32_t kChunkBytes = 128 * 32 * 4;  // a chunk's partial sums in a CTA: [token / 4][row][4]

// Where the sums of chunk c from pair `from` lie in the CTA that finishes it.
__device__ __forceinline__ uint32_t chunk_slot(int c, int from, int splits) {
    const int owner = c % splits;
    return (uint32_t)(c / splits * (splits - 1) + (from < owner ? from : from - 1)) * kChunkBytes;
}

// The chunks that this warp finishes of the tile at (tn, tm); `part`: the shared memory that the others have filled.
template <bool GATED>
__device__ __forceinline__ void finish_chunks(const TcArgs& t, float* swap, uint32_t part, uint32_t tmem, int rank, int q,
                                              int tn, int tm) {
    constexpr int C = GATED ? 16 : 32;
    const LinearArgs& a = t.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quad = warp & 3, half = (warp - 2) >> 2, row = quad * 32 + lane, S = t.splits;
    const bool up = GATED && quad >= 2;  // as in `epilogue`
    const int own = up ? 16 : 0;
    const uint32_t pair_bar = 1 + (quad & 1) + 2 * half;
    float* ex = swap + ((quad & 1) + 2 * half) * (2 * 2 * 16 * 32) + lane;
    const int n = (tn * 2 + rank) * (GATED ? 64 : 128) + (GATED ? row & 63 : row), col = up ? a.N + n : n;
    const bool live = n < a.N;
    const float ws = a.w_scale && live ? a.w_scale[col] : 1.f;
    const float bias = a.bias && live ? a.bias[col] : 0.f;
    int flip = 0;
#pragma unroll 1
    for (int c = q + half * S; c < t.bn / 32; c += 2 * S) {
        const int m0 = tm * t.bn + c * 32;
        uint32_t r[C];
        if (a.res && live) load_residual<C>(a, r, m0 + own, n);
        float v[32], sum[32];
        tmem_ld32(tmem + c * 32 + ((uint32_t)(quad * 32) << 16), v);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; ++j) sum[j] = 0.f;
#pragma unroll 1
        for (int p = 0; p < S; ++p) {
            if (p == q) {
#pragma unroll
                for (int j = 0; j < 32; ++j) sum[j] += v[j];
                continue;
            }
            const uint32_t at = part + chunk_slot(c, p, S) + row * 16;
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
                const float4 w = ld_cluster_f32x4(at + j / 4 * 2048);
                sum[j] += w.x, sum[j + 1] += w.y, sum[j + 2] += w.z, sum[j + 3] += w.w;
            }
        }
        if (a.x_scale) {
            const float mine = m0 + lane < a.M ? a.x_scale[m0 + lane] : 0.f;
#pragma unroll
            for (int j = 0; j < 32; ++j) sum[j] *= __shfl_sync(0xffffffffu, mine, j) * ws;
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) sum[j] += bias;
        if constexpr (!GATED) {
            if (live) finish<32>(a, sum, nullptr, r, m0, n);
        } else {
            float* box = ex + flip * (2 * 16 * 32);
            flip ^= 1;
#pragma unroll
            for (int j = 0; j < 16; ++j) box[(own + j) * 32] = up ? sum[j] : sum[16 + j];
            named_bar_sync(pair_bar, 64);
            float g[16], w[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float other = box[((16 - own) + j) * 32];
                g[j] = up ? other : sum[j];
                w[j] = up ? sum[16 + j] : other;
            }
            if (live) finish<16>(a, g, w, r, m0 + own, n);
        }
    }
}

template <bool F8, bool KN, bool BLOCKED>
__global__ void __launch_bounds__(kThreads, 1) linear_joint_kernel(const __grid_constant__ CUtensorMap tm_w,
                                                                   const __grid_constant__ CUtensorMap tm_x,
                                                                   const __grid_constant__ TcArgs t) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const LinearArgs& a = t.a;
    constexpr int kSlabElems = F8 ? 128 : 64;
    const int stages = t.stages, S = t.splits;
    float* swap = reinterpret_cast<float*>(sm + stages * t.stage_bytes);
    LargeBars* bars = reinterpret_cast<LargeBars*>(sm + stages * t.stage_bytes + (a.gated ? kSwapBytes : 0));
    volatile int* abort_flag = &bars->abort;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int place = (int)cluster_rank(), q = place >> 1, rank = place & 1, leader = place & ~1;
    const int tile = (int)blockIdx.x / (2 * S), tm = tile / t.tiles_n, tn = tile - tm * t.tiles_n;
    const int k_lo = (int)((long long)t.slabs * q / S), k_hi = (int)((long long)t.slabs * (q + 1) / S);
    griddep_launch_dependents();

    if (warp == 0) {
        if (lane < stages) {
            mbar_init(&bars->full[lane], 1);
            mbar_init(&bars->empty[lane], 1);
        } else if (lane >= 16 && lane < (BLOCKED ? 18 : 17)) {
            mbar_init(&bars->acc_full[lane - 16], 1);
            if (BLOCKED) mbar_init(&bars->acc_empty[lane - 16], 2 * kEpiWarps);
        } else if (lane == 30) {
            bars->abort = 0;
        }
        fence_mbar_init();
        if (lane == 31) {
            tma_prefetch_desc(&tm_w);
            tma_prefetch_desc(&tm_x);
        }
        __syncwarp();
    }
    if (warp == 1) tmem_alloc_pair(&bars->tmem, t.tmem_cols);
    tc_fence_before();
    __syncthreads();
    cluster_sync_relaxed();  // the peers' barriers are initialised (fence_mbar_init)
    tc_fence_after();
    const uint32_t tmem = bars->tmem;
    griddep_wait();

    bool ok = false;
    float sum[3][32];  // BLOCKED: of the chunks whose blocks this warp adds
    if (warp == 0) {  // TMA producer: this CTA's columns and its half of the tokens
        const int per = a.gated ? 64 : 128, n0 = (tn * 2 + rank) * per, n1 = a.gated ? t.up + n0 : n0 + 64;
        const int m0 = tm * t.bn + rank * (t.bn / 2);
        int i = 0;
        Ring at;
        for (; i < k_hi - k_lo; ++i, at.next(stages)) {
            const int s = at.s, k = (k_lo + i) * kSlabElems;
            if (i >= stages && !mbar_wait_warp(&bars->empty[s], at.phase ^ 1, abort_flag)) break;
            uint8_t* st = sm + s * t.stage_bytes;
            if (elect_one()) {
                if (rank == 0) mbar_arrive_expect_tx(&bars->full[s], 2 * t.stage_bytes);
                const uint32_t bar = map_to_rank(smem_u32(&bars->full[s]), leader);
                tma_load_3d_pair(st, &tm_w, bar, KN ? n0 : k, KN ? k : n0, 0);
                tma_load_3d_pair(st + kHalfW, &tm_w, bar, KN ? n1 : k, KN ? k : n1, 0);
                tma_load_3d_pair(st + kWBytes, &tm_x, bar, k, m0, 0);
            }
            __syncwarp();
        }
        if (rank == 0)  // the leader sees both CTAs' loads land (bounded)
            for (int j = (i > stages ? i - stages : 0); j < i; ++j)
                (void)mbar_wait(&bars->full[j % stages], (j / stages) & 1);
    } else if (warp == 1) {
        if (rank == 0) {  // MMA issuer of the pair
            const uint32_t both = 3u << leader;
            int i = 0, block = 0, in = 0;  // the block of K, and the slab in it
            Ring at;
            for (; i < k_hi - k_lo; ++i, at.next(stages)) {
                if (BLOCKED && in == t.block) {
                    if (++block >= 2 && !mbar_wait_warp(&bars->acc_empty[block & 1], ((block - 2) >> 1) & 1, abort_flag))
                        break;
                    in = 0;
                }
                if (!mbar_wait_warp(&bars->full[at.s], at.phase, abort_flag)) break;
                tc_fence_after();
                const int b = BLOCKED ? block & 1 : 0;
                if (elect_one()) {
                    const uint32_t st = smem_u32(sm) + at.s * t.stage_bytes;
                    mma_slab<F8, KN, true>(tmem + b * t.bn, st, st, t.idesc, (BLOCKED ? in : i) == 0);
                    mma_commit_pair(&bars->empty[at.s], both);
                    if (i + 1 == k_hi - k_lo || (BLOCKED && in + 1 == t.block)) mma_commit_pair(&bars->acc_full[b], both);
                }
                __syncwarp();
                ++in;
            }
            if (i > 0) (void)mbar_wait(&bars->empty[(i - 1) % stages], ((i - 1) / stages) & 1);  // all products are done
        }
    } else if constexpr (BLOCKED) {
        const int blocks = (k_hi - k_lo + t.block - 1) / t.block;
        const uint32_t done0 = map_to_rank(smem_u32(&bars->acc_empty[0]), leader);
        const uint32_t done1 = map_to_rank(smem_u32(&bars->acc_empty[1]), leader);
        // this warp's chunks `half`, half + 2, half + 4
        const uint32_t at = tmem + ((warp - 2) >> 2) * 32 + ((uint32_t)((warp & 3) * 32) << 16);
#pragma unroll
        for (int i = 0; i < 96; ++i) sum[i / 32][i % 32] = 0.f;
        for (int b = 0; b < blocks; ++b) {
            ok = mbar_wait_warp(&bars->acc_full[b & 1], (b >> 1) & 1, abort_flag);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int j = 0; j < 3; ++j) {
                if (((warp - 2) >> 2) + 2 * j >= t.bn / 32) break;
                float v[32];
                tmem_ld32(at + (b & 1) * t.bn + j * 64, v);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) sum[j][i] += v[i];
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0 && b + 2 < blocks) mbar_arrive_cluster_relaxed(b & 1 ? done1 : done0);
        }
    } else {
        ok = __all_sync(0xffffffffu, mbar_wait_or_abort(&bars->acc_full[0], 0, abort_flag));
    }
    __syncwarp();
    cluster_sync();  // every pair's products are done: the stages are free
    if (ok) {
        tc_fence_after();
        const int quad = warp & 3, half = (warp - 2) >> 2;
#pragma unroll
        for (int j = 0; j < (BLOCKED ? 3 : 4); ++j) {
            const int c = half + 2 * j;
            if (c >= t.bn / 32) break;
            const uint32_t mine = tmem + c * 32 + ((uint32_t)(quad * 32) << 16);
            float v[32];
            if constexpr (BLOCKED) {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = sum[j][i];
                if (c % S == q) {  // finished below, by another warp
                    tmem_st32(mine, v);
                    tmem_wait_st();
                    tc_fence_before();
                }
            }
            if (c % S == q) continue;
            if constexpr (!BLOCKED) {
                tmem_ld32(mine, v);
                tmem_wait_ld();
            }
            const uint32_t slot = smem_u32(sm) + chunk_slot(c, q, S) + (quad * 32 + lane) * 16;
            const uint32_t to = map_to_rank(slot, 2 * (c % S) + rank);
#pragma unroll
            for (int i = 0; i < 32; i += 4) st_cluster_f32x4(to + i / 4 * 2048, v[i], v[i + 1], v[i + 2], v[i + 3]);
        }
    }
    __syncwarp();
    cluster_sync();  // the partial sums are there
    if (warp >= 2) {
        if (BLOCKED) tc_fence_after();
        const uint32_t pair_bar = 1 + (warp & 1) + 2 * ((warp - 2) >> 2);
        if (a.gated) ok = !named_bar_any(pair_bar, 64, !ok);  // one answer for the warps that meet at a barrier
        if (ok && a.gated)
            finish_chunks<true>(t, swap, smem_u32(sm), tmem, rank, q, tn, tm);
        else if (ok)
            finish_chunks<false>(t, swap, smem_u32(sm), tmem, rank, q, tn, tm);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync_relaxed();
    if (tid == 0 && bars->abort) atomicExch(t.status, (int32_t)GDN_ERR_TIMEOUT);
    __syncwarp();
    if (warp == 1) tmem_dealloc_pair(tmem, t.tmem_cols);
    cluster_sync_relaxed();  // neither CTA exits while the pair's TMEM is being freed
}

// ------------------------------------------------------------------ host side
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encoder() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// A [rows][cols] matrix (cols contiguous, rows `pitch` elements apart) in boxes of 128 bytes x box_rows
// with the 128-byte swizzle; what lies outside reads as zero and is not written.
bool encode(CUtensorMap* map, bool f8, const void* ptr, long long rows, long long cols, long long pitch, int box_rows) {
    EncodeTiledFn enc = encoder();
    if (!enc) return false;
    const cuuint64_t size = f8 ? 1 : 2;
    cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, 1};
    cuuint64_t strides[2] = {(cuuint64_t)pitch * size, (cuuint64_t)rows * pitch * size};
    cuuint32_t box[3] = {(cuuint32_t)(kSlabBytes / size), (cuuint32_t)box_rows, 1}, estr[3] = {1, 1, 1};
    return enc(map, f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr),
               dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kSmemLimit = 227 * 1024;

// A launch in clusters of `cluster` CTAs that may be set up while the stream's preceding kernel ends
// (programmatic stream serialization; the kernels wait for that kernel before they read anything).
template <typename... P, typename... Q>
cudaError_t launch(void (*kernel)(P...), std::atomic<bool> (&done)[kMaxDevices], int dev, dim3 grid, int threads,
                   size_t smem, int cluster, cudaStream_t s, const Q&... args) {
    const cudaError_t e = allow_smem(kernel, kSmemLimit, done, dev);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// A launch of 256 threads a CTA behind everything before it.  (Its own result: cudaGetLastError would also report an
// earlier error of the calling thread.)
template <typename... P, typename... Q>
cudaError_t launch_plain(void (*kernel)(P...), unsigned grid, cudaStream_t s, const Q&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Where TMA finds x and the weight: the caller's arrays, or copies of them with rows of whole 16-byte
// pieces.  Pitches in elements; up: the weight column where a gated weight's up half starts.
struct Operands {
    const void *x, *w;
    long long x_pitch, w_pitch, w_cols;
    int up;
    const uint8_t* tops = nullptr;  // see TcArgs
    int marks = 0;
    int accs = 1, starts[kMaxAccs] = {};
    int plane = 0;  // of parts: see TcArgs (depth: the rows or columns of K that there are)
    long long depth(const LinearArgs& a) const { return plane ? 3LL * plane : a.K; }
};

template <bool F8, bool KN, bool PARTS, bool BLOCKED>
cudaError_t launch_small_as(const TcArgs& t, const CUtensorMap& tw, const CUtensorMap& tx, int tiles, int tiles_m,
                            size_t smem, int dev, cudaStream_t s) {
    static std::atomic<bool> done[kMaxDevices];
    const dim3 grid((unsigned)(tiles * t.splits), (unsigned)tiles_m);
    return launch(linear_small_kernel<F8, KN, PARTS, BLOCKED>, done, dev, grid, kThreads, smem, t.splits, s, tw, tx, t);
}
template <bool F8, bool KN, bool PARTS>
cudaError_t launch_small(const TcArgs& t, const CUtensorMap& tw, const CUtensorMap& tx, int tiles, int tiles_m, size_t smem,
                         int dev, cudaStream_t s) {
    if constexpr (!PARTS) {
        if (t.blocks > 1) return launch_small_as<F8, KN, false, true>(t, tw, tx, tiles, tiles_m, smem, dev, s);
    }
    return launch_small_as<F8, KN, PARTS, false>(t, tw, tx, tiles, tiles_m, smem, dev, s);
}

// What runs, on tiles of bn tokens: pairs (large), with K over `splits` of them where that is more than one, or
// the small kernel with K over `splits` CTAs.
struct Plan {
    bool large;
    int bn, splits;
};

// The estimated time of every choice, in us, and the least of them.  A slab is 16 KB of weight and 128
// bytes of every token of the tile.  Fitted to sweeps of M = 1 .. 512, K and N = 512 .. 8192 (bf16, us in a
// graph over weights larger than L2):
//   - small: one CTA takes in about 85 KB/us and two on an SM 115, all together at most 6.3 MB/us; the
//     partial sums' way through TMEM and shared memory costs 0.3 + bn / 60, a third more over 8 CTAs.  M = 64,
//     K = N = 2048: 12.4 (32 tokens, no split), 8.3 (2), 6.8 (4), 6.9 (8);
//   - pairs: 0.28 us a slab at 256 tokens (the tensor cores' time), in proportion down to 0.19 (the weight's way
//     from L2), and bn / 300 for the last tile's outputs.  M = 512, K = N = 4096: 20.6 the best small plan, 16.9 pairs
//     at 128, 22.4 at 256; K = 16384, N = 512: 17.1 small, 55 pairs.
//   - pairs that split K: the same for their share of K, and 0.6 us a pair and bn 0.012 for the sums' way.  Where not
//     all clusters fit at once this is no choice (of 4, 6 and 8 CTAs 36, 23 and 15 do on 152 SMs).  M = 768, K = 8192,
//     N = 2048: 28.7 pairs, 20.5 two a tile of 192; M = 384, K = 4096, N = 2048: 13.7 small, 15.8 pairs, 11.6 two a tile
//     of 128; M = 1024, K = N = 2048: 10.3 pairs, 12.5 two a tile of 256.
// On the 48 shapes (M = 64 .. 1024) that it was fitted to the choice is 0.3 % behind the best of all on average, by parts
// on 17 shapes it is it; on others it may be further off (M = 32, K = N = 8192 with fp32 output: 33 us, 25 the best).
//   - blocks of K (see block_of): tiles of at most 192 tokens, in the small kernel 64; pairs
//     lose about 2 us and 0.2 a block, where they split K half of that.  M = 64, K = 2048, N = 8192: 13.4 pairs of 64 tokens
//     (10.1 without blocks), 10.9 small; M = 1024, K = 8192, N = 2048: 36.8 pairs, 47 small.
Plan plan(const LinearArgs& a, int slabs, int accs, int sms) {
    const bool blocked = a.out_f32 && accs == 1;
    const long long wn = a.gated ? 2LL * a.N : a.N, tiles1 = (wn + 127) / 128, tiles2 = (wn + 255) / 256;
    const int parts = accs > 1 ? 3 : 1, products = accs > 1 ? 6 : 1;  // stages and products of a slab
    const double weight_mb = tiles1 * slabs * parts * (16.0 / 1024);
    const int pairs = sms > 1 ? sms / 2 : 1;
    Plan best{true, 64, 1};
    double least = 1e30;
    for (int bn = accs > 1 ? 512 / accs / 32 * 32 : 256; bn >= 64; bn -= 32) {  // (TMEM: 512 columns)
        const long long tiles = tiles2 * ((a.M + bn - 1) / bn), turns = (tiles + pairs - 1) / pairs;
        const double mma = products * bn * (0.28 / 256), in = parts * (accs > 1 ? (16 + bn / 16) / 105.0 : 0.19);
        double t = bn / 300.0 + (double)turns * slabs * (mma > in ? mma : in);
        if (accs > 1) t += (turns - 1) * accs * bn / 200.0;  // epilogues that nothing runs beside
        if (t < 1.0 + weight_mb / 6.3) t = 1.0 + weight_mb / 6.3;
        if (blocked && slabs > kBlockSlabs) t += 2.0 + 0.2 * (slabs / kBlockSlabs);
        if (t < least && !(bn > 192 && blocked && slabs > kBlockSlabs)) least = t, best = Plan{true, bn, 1};
        for (int S = 2; S <= 4 && accs == 1 && 2 * S <= slabs; ++S) {
            if (bn > 192 && blocked && (slabs + S - 1) / S > kBlockSlabs) continue;
            if (tiles > sms / (2 * S) - 2 * (S - 1)) break;
            t = (slabs + S - 1) / S * (mma > in ? mma : in);
            if (t < weight_mb / 6.3) t = weight_mb / 6.3;
            t += 0.012 * bn + 0.6 * S;
            if (blocked && (slabs + S - 1) / S > kBlockSlabs) t += 1.0 + 0.1 * (slabs / S / kBlockSlabs);
            if (t < least) least = t, best = Plan{true, bn, S};
        }
    }
    // (TMEM: 256 columns where two CTAs share an SM's, by parts all of it)
    for (int bn = 16; bn <= (accs > 4 ? 64 : accs > 1 ? 256 / accs : 128); bn *= 2) {
        if (bn > 16 && bn / 2 >= a.M) break;
        const long long tiles_m = (a.M + bn - 1) / bn;
        if (tiles_m > 65535) continue;  // the grid's limit
        for (int S = 1; S <= 8 && S * 2 <= (slabs > 2 ? slabs : 2); S *= 2) {
            const long long ctas = tiles1 * tiles_m * S;
            if (blocked && bn > 64 && (slabs + S - 1) / S > kBlockSlabs) continue;
            const int beside = accs > 1 ? 1 : 2;
            // CTAs at once: clusters stay inside one of 8 groups of SMs (of 16 to 20: two clusters of 8 do not fit).
            // (Fewer than 48 SMs have no room for clusters of 8 CTAs, and by parts fewer than 96.)
            const long long room = 8LL * ((sms / 8 * beside - (S == 8 ? 4 : 0)) / S) * S;
            if (room <= 0) continue;
            const long long waves = (ctas + room - 1) / room;
            const long long an_sm = ctas <= sms ? 1 : waves * beside;  // CTAs one after another, or beside one another
            const double kb = (double)an_sm * ((slabs + S - 1) / S) * parts * (16 + bn / 8.0);
            double t = kb / (an_sm == 1 || beside == 1 ? 85 : 115);
            if (t < weight_mb / 6.3) t = weight_mb / 6.3;
            double join = 0.3 + bn / 60.0;
            if (S == 8) join = join * 1.3 + 0.2;
            t += join * waves + 3.0 * (waves - 1);
            if (t < least) least = t, best = Plan{false, bn, S};
        }
    }
    return best;
}

gdn_status run_small(const LinearArgs& a, const Operands& op, bool f8, Plan how, int dev, cudaStream_t s) {
    TcArgs t{};
    t.a = a;
    t.up = op.up;
    t.tops = op.tops;
    t.marks = op.marks;
    t.accs = op.accs;
    for (int q = 0; q < kMaxAccs; ++q) t.starts[q] = op.starts[q];
    t.plane = op.plane;
    const int elems = f8 ? 128 : 64, per = a.gated ? 64 : 128;
    t.slabs = (a.K + elems - 1) / elems;
    t.bn = how.bn;
    t.splits = how.splits;
    t.block = block_of((t.slabs + t.splits - 1) / t.splits, a.out_f32 && t.accs == 1);
    t.blocks = ((t.slabs + t.splits - 1) / t.splits + t.block - 1) / t.block;
    const long long tiles = ((long long)a.N + per - 1) / per, tiles_m = (a.M + t.bn - 1) / t.bn;
    if (tiles * t.splits > INT32_MAX || tiles_m > 65535) return GDN_ERR_DIMS;
    t.wide_out = a.N % 4 == 0 && (reinterpret_cast<uintptr_t>(a.out) & (a.out_f32 ? 15u : 7u)) == 0;
    t.stage_bytes = kWBytes + t.bn * kSlabBytes;
    t.stages = (int)(((op.plane ? kSmemLimit : 112 * 1024) - sizeof(SmallBars) - 1024) / t.stage_bytes);  // two CTAs an SM
    if (t.stages > kMaxStages) t.stages = kMaxStages;
    t.tmem_cols = 32;
    while (t.tmem_cols < (uint32_t)((t.blocks > 1 ? 2 : t.accs) * t.bn)) t.tmem_cols <<= 1;
    t.idesc = f8 ? make_idesc_e4m3(128, t.bn) : make_idesc_bf16(128, t.bn, a.nk ? 0 : 1, 0);
    gdn_status st = status_word_for_current_device(&t.status);
    if (st != GDN_OK) return st;
    CUtensorMap tw, tx;
    const long long depth = op.depth(a);
    if (!encode(&tw, f8, op.w, a.nk ? op.w_cols : depth, a.nk ? depth : op.w_cols, op.w_pitch, 64) ||
        !encode(&tx, f8, op.x, a.M, depth, op.x_pitch, t.bn))
        return GDN_ERR_CUDA;
    const size_t smem = (size_t)t.stages * t.stage_bytes + sizeof(SmallBars) + 1024;
    auto run = [&](auto e4m3, auto kn, auto parts) {
        constexpr bool kF8 = decltype(e4m3)::value, kKN = decltype(kn)::value, kParts3 = decltype(parts)::value;
        return launch_small<kF8, kKN, kParts3>(t, tw, tx, (int)tiles, (int)tiles_m, smem, dev, s);
    };
    const std::true_type yes{};
    const std::false_type no{};
    const cudaError_t e = f8              ? run(yes, no, no)
                          : op.accs == 1 ? (a.nk ? run(no, no, no) : run(no, yes, no))
                                         : (a.nk ? run(no, no, yes) : run(no, yes, yes));
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

template <bool F8, bool KN, bool PARTS, bool BLOCKED>
cudaError_t launch_large_as(const TcArgs& t, const CUtensorMap& tw, const CUtensorMap& tx, const CUtensorMap& to,
                            const CUtensorMap& tr, int pairs, size_t smem, int dev, cudaStream_t s) {
    static std::atomic<bool> done[kMaxDevices];
    return launch(linear_large_kernel<F8, KN, PARTS, BLOCKED>, done, dev, dim3((unsigned)(2 * pairs)), kThreads, smem, 2, s,
                  tw, tx, to, tr, t);
}

template <bool F8, bool KN, bool PARTS>
cudaError_t launch_large(const TcArgs& t, const CUtensorMap& tw, const CUtensorMap& tx, const CUtensorMap& to,
                         const CUtensorMap& tr, int pairs, size_t smem, int dev, cudaStream_t s) {
    if constexpr (!PARTS) {
        if (t.blocks > 1) return launch_large_as<F8, KN, false, true>(t, tw, tx, to, tr, pairs, smem, dev, s);
    }
    return launch_large_as<F8, KN, PARTS, false>(t, tw, tx, to, tr, pairs, smem, dev, s);
}

gdn_status run_large(const LinearArgs& a, const Operands& op, bool f8, Plan how, int dev, int sms, cudaStream_t s) {
    TcArgs t{};
    t.a = a;
    t.up = op.up;
    t.tops = op.tops;
    t.marks = op.marks;
    t.accs = op.accs;
    for (int q = 0; q < kMaxAccs; ++q) t.starts[q] = op.starts[q];
    t.plane = op.plane;
    const int elems = f8 ? 128 : 64, per = a.gated ? 128 : 256;
    t.slabs = (a.K + elems - 1) / elems;
    t.tiles_n = (int)(((long long)a.N + per - 1) / per);
    t.bn = how.bn;
    t.block = block_of(t.slabs, a.out_f32 && t.accs == 1);
    t.blocks = (t.slabs + t.block - 1) / t.block;
    t.ring = t.blocks == 1 ? 2 : 512 / t.bn < kMaxRing ? 512 / t.bn : kMaxRing;
    t.tiles_m = (a.M + t.bn - 1) / t.bn;
    if ((long long)t.tiles_n * t.tiles_m > INT32_MAX - sms) return GDN_ERR_DIMS;
    t.group = t.tiles_n < 16 ? t.tiles_n : 16;
    t.stage_bytes = kWBytes + t.bn / 2 * kSlabBytes;
    t.staged = !op.plane && !a.out_f32 && a.N % 8 == 0 &&
               ((reinterpret_cast<uintptr_t>(a.out) | reinterpret_cast<uintptr_t>(a.res)) & 15u) == 0;
    const size_t fixed = sizeof(LargeBars) + box_bytes(t) + (a.gated ? kSwapBytes : 0) + 1024;
    t.stages = (int)((kSmemLimit - fixed) / t.stage_bytes);
    if (t.stages > kLargeStages) t.stages = kLargeStages;
    t.tmem_cols = 128;
    while (t.tmem_cols < (uint32_t)((t.accs > t.ring ? t.accs : t.ring) * t.bn)) t.tmem_cols <<= 1;
    t.idesc = f8 ? make_idesc_e4m3(256, t.bn) : make_idesc_bf16(256, t.bn, a.nk ? 0 : 1, 0);
    gdn_status st = status_word_for_current_device(&t.status);
    if (st != GDN_OK) return st;
    CUtensorMap tw, tx;
    const long long depth = op.depth(a);
    if (!encode(&tw, f8, op.w, a.nk ? op.w_cols : depth, a.nk ? depth : op.w_cols, op.w_pitch, 64) ||
        !encode(&tx, f8, op.x, a.M, depth, op.x_pitch, t.bn / 2))
        return GDN_ERR_CUDA;
    CUtensorMap to{}, tr{};
    const int tokens = a.gated ? 16 : 32;
    if (t.staged && (!encode(&to, false, a.out, a.M, a.N, a.N, tokens) ||
                     (a.res && !encode(&tr, false, a.res, a.M, a.N, a.N, tokens))))
        return GDN_ERR_CUDA;
    const size_t smem = (size_t)t.stages * t.stage_bytes + fixed;
    const int tiles = t.tiles_n * t.tiles_m, most = sms > 1 ? sms / 2 : 1, pairs = tiles < most ? tiles : most;
    const cudaError_t e = f8              ? launch_large<true, false, false>(t, tw, tx, to, tr, pairs, smem, dev, s)
                          : op.accs == 1 ? (a.nk ? launch_large<false, false, false>(t, tw, tx, to, tr, pairs, smem, dev, s)
                                                 : launch_large<false, true, false>(t, tw, tx, to, tr, pairs, smem, dev, s))
                          : a.nk         ? launch_large<false, false, true>(t, tw, tx, to, tr, pairs, smem, dev, s)
                                         : launch_large<false, true, true>(t, tw, tx, to, tr, pairs, smem, dev, s);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

template <bool F8, bool KN, bool BLOCKED>
cudaError_t launch_joint_as(const TcArgs& t, const CUtensorMap& tw, const CUtensorMap& tx, int tiles, size_t smem, int dev,
                            cudaStream_t s) {
    static std::atomic<bool> done[kMaxDevices];
    return launch(linear_joint_kernel<F8, KN, BLOCKED>, done, dev, dim3((unsigned)(tiles * 2 * t.splits)), kThreads, smem,
                  2 * t.splits, s, tw, tx, t);
}
template <bool F8, bool KN>
cudaError_t launch_joint(const TcArgs& t, const CUtensorMap& tw, const CUtensorMap& tx, int tiles, size_t smem, int dev,
                         cudaStream_t s) {
    return t.blocks > 1 ? launch_joint_as<F8, KN, true>(t, tw, tx, tiles, smem, dev, s)
                        : launch_joint_as<F8, KN, false>(t, tw, tx, tiles, smem, dev, s);
}

gdn_status run_joint(const LinearArgs& a, const Operands& op, bool f8, Plan how, int dev, cudaStream_t s) {
    TcArgs t{};
    t.a = a;
    t.up = op.up;
    t.accs = 1;
    const int elems = f8 ? 128 : 64, per = a.gated ? 128 : 256;
    t.slabs = (a.K + elems - 1) / elems;
    t.tiles_n = (int)(((long long)a.N + per - 1) / per);
    t.bn = how.bn;
    t.splits = how.splits;
    t.block = block_of((t.slabs + t.splits - 1) / t.splits, a.out_f32);
    t.blocks = ((t.slabs + t.splits - 1) / t.splits + t.block - 1) / t.block;
    t.tiles_m = (a.M + t.bn - 1) / t.bn;
    t.stage_bytes = kWBytes + t.bn / 2 * kSlabBytes;
    // (the others' sums of a CTA's chunks, 96 KB at the most, fit the stages, 168 KB at the least)
    const size_t fixed = sizeof(LargeBars) + (a.gated ? kSwapBytes : 0) + 1024;
    t.stages = (int)((kSmemLimit - fixed) / t.stage_bytes);
    if (t.stages > kLargeStages) t.stages = kLargeStages;
    t.tmem_cols = 32;
    while (t.tmem_cols < (uint32_t)((t.blocks > 1 ? 2 : 1) * t.bn)) t.tmem_cols <<= 1;
    t.idesc = f8 ? make_idesc_e4m3(256, t.bn) : make_idesc_bf16(256, t.bn, a.nk ? 0 : 1, 0);
    gdn_status st = status_word_for_current_device(&t.status);
    if (st != GDN_OK) return st;
    CUtensorMap tw, tx;
    if (!encode(&tw, f8, op.w, a.nk ? op.w_cols : a.K, a.nk ? a.K : op.w_cols, op.w_pitch, 64) ||
        !encode(&tx, f8, op.x, a.M, a.K, op.x_pitch, t.bn / 2))
        return GDN_ERR_CUDA;
    const size_t smem = (size_t)t.stages * t.stage_bytes + fixed;
    const int tiles = t.tiles_n * t.tiles_m;
    const cudaError_t e = f8     ? launch_joint<true, false>(t, tw, tx, tiles, smem, dev, s)
                          : a.nk ? launch_joint<false, false>(t, tw, tx, tiles, smem, dev, s)
                                 : launch_joint<false, true>(t, tw, tx, tiles, smem, dev, s);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace

namespace {

// Rows of `cols` elements with any alignment, copied to rows `pitch` elements apart (whole 16-byte
// pieces): the first `half` columns to column 0, the others to column `up`.
struct CopyJob {
    const void* src;
    void* dst;
    long long rows, cols, pitch, half, up;
};

template <typename E>
__global__ void __launch_bounds__(256) linear_align_kernel(const __grid_constant__ CopyJob x,
                                                           const __grid_constant__ CopyJob w) {
    constexpr int V = 16 / (int)sizeof(E);
    griddep_launch_dependents();
    griddep_wait();
    const long long x_pieces = x.rows * (x.pitch / V), pieces = x_pieces + w.rows * (w.pitch / V);
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < pieces; i += (long long)gridDim.x * 256) {
        const CopyJob& c = i < x_pieces ? x : w;
        const long long at = i < x_pieces ? i : i - x_pieces, row = at / (c.pitch / V), d0 = at % (c.pitch / V) * V;
        const E* src = static_cast<const E*>(c.src) + row * c.cols;
        E e[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const long long d = d0 + j, from = d < c.half ? d : d >= c.up ? c.half + d - c.up : c.cols;
            e[j] = from < c.cols ? src[from] : E(0);
        }
        uint4 o;
        memcpy(&o, e, 16);
        reinterpret_cast<uint4*>(c.dst)[row * (c.pitch / V) + at % (c.pitch / V)] = o;
    }
}

// fp32 operands as three bf16 parts each: x = x1 + x2 + x3, every part the rounding of what the ones before
// leave (24 bits in three times 8, so the sum is exact).  Of the nine products of parts the six of 2^-16 and
// more are taken, the five small ones (x1 w3, x3 w1, x2 w2, x1 w2, x2 w1) into an accumulator of their own.
// The tensor cores truncate a sum at every step of 16 terms, always towards zero, so that it falls short by
// about K 1e-9 of itself (2.1e-6 at K = 2048; fp32 sums with rounding 0.8e-6).  The x1 w1, whose sum that is,
// therefore go to an accumulator for every 704 to 1024 of K (see accs_of), which are added with rounding: at K = 4096
// sums of one sign are off by 8.3e-7 (fp32 sums 8.4e-7; with three accumulators 1.57e-6).
constexpr int kParts = 3;

// Splits one operand: rows_in x cols fp32 -> rows_out x width parts, rows `pitch` apart and parts `plane`
// apart; columns as in CopyJob, what lies outside is zero.
struct SplitJob {
    const float* src;
    __nv_bfloat16* dst;
    long long rows_in, rows_out, cols, width, pitch, plane, half, up;
};

// tops[block], tops[gridDim.x + block]: the exponents of the largest elements of x and of the weight that the block
// met (see LinearMarks).
// 16 bytes are read at a time where a piece lies whole and on such a boundary (2048 x 2048 twice: 28 us by elements).
__global__ void __launch_bounds__(256) linear_split_kernel(const __grid_constant__ SplitJob x,
                                                           const __grid_constant__ SplitJob w, uint8_t* tops) {
    __shared__ uint32_t warp_tops[2][256 / 32];
    griddep_launch_dependents();
    griddep_wait();
    const long long x_pieces = x.rows_out * (x.width / 8), pieces = x_pieces + w.rows_out * (w.width / 8);
    uint32_t top_x = 0, top_w = 0;  // (magnitudes are ordered as their bits are, infinities and NaN above all)
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < pieces; i += (long long)gridDim.x * 256) {
        const SplitJob& c = i < x_pieces ? x : w;
        const long long at = i < x_pieces ? i : i - x_pieces, row = at / (c.width / 8), d0 = at % (c.width / 8) * 8;
        const float* src = c.src + row * c.cols;
        float in[8];
        const long long first = d0 < c.half ? d0 : c.half + d0 - c.up;  // the source column of d0, if it has one
        const bool whole = row < c.rows_in && (d0 + 8 <= c.half || d0 >= c.up) && first + 8 <= c.cols;
        if (whole && (reinterpret_cast<uintptr_t>(src + first) & 15u) == 0) {
            const float4* at16 = reinterpret_cast<const float4*>(src + first);
            const float4 p = at16[0], q = at16[1];
            in[0] = p.x, in[1] = p.y, in[2] = p.z, in[3] = p.w, in[4] = q.x, in[5] = q.y, in[6] = q.z, in[7] = q.w;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const long long d = d0 + j, from = d < c.half ? d : d >= c.up ? c.half + d - c.up : c.cols;
                in[j] = row < c.rows_in && from < c.cols ? src[from] : 0.f;
            }
        }
        __nv_bfloat16 part[3][8];
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float v = in[j];
            top = max(top, __float_as_uint(v) & 0x7fffffffu);
            __nv_bfloat16 p = __float2bfloat16_rn(v);
            part[0][j] = p;
            float left = v - __bfloat162float(p);
            part[1][j] = p = __float2bfloat16_rn(left);
            left -= __bfloat162float(p);
            part[2][j] = __float2bfloat16_rn(left);
        }
        uint4 o[3];
        memcpy(o, part, sizeof(o));
        uint4* dst = reinterpret_cast<uint4*>(c.dst + row * c.pitch + d0);
#pragma unroll
        for (int k = 0; k < kParts; ++k) dst[k * (c.plane / 8)] = o[k];
        if (i < x_pieces)
            top_x = max(top_x, top);
        else
            top_w = max(top_w, top);
    }
    top_x = __reduce_max_sync(0xffffffffu, top_x);
    top_w = __reduce_max_sync(0xffffffffu, top_w);
    if ((threadIdx.x & 31) == 0) warp_tops[0][threadIdx.x >> 5] = top_x, warp_tops[1][threadIdx.x >> 5] = top_w;
    __syncthreads();
    if (threadIdx.x < 2) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 256 / 32; ++i) top = max(top, warp_tops[threadIdx.x][i]);
        tops[threadIdx.x * gridDim.x + blockIdx.x] = (uint8_t)(top == 0 ? 0 : max(top >> 23, 1u));
    }
}

// Whether TMA can take an operand of `cols`-element rows as it lies.
bool takes(const void* p, long long cols, int size) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && cols * size % 16 == 0;
}

int slabs_of(int K, bool f8) { return (K + (f8 ? 127 : 63)) / (f8 ? 128 : 64); }

// The accumulators of a tile by parts: one for the small products and, for the x1 w1, one for every `share` slabs: 704 of
// K, up to 1024 where that would be more than three (and four of them past K = 3072).
int accs_of(int slabs, int* share) {
    const int wanted = slabs > 48 ? 4 : slabs > 22 ? 3 : (slabs + 10) / 11;
    *share = (slabs + wanted - 1) / wanted;
    return 1 + (slabs + *share - 1) / *share;
}

gdn_status run_tc(const LinearArgs& a, const Operands& op, bool f8, int dev, int sms, cudaStream_t s) {
    const Plan how = plan(a, slabs_of(a.K, f8), op.accs, sms);
    if (how.large && how.splits > 1) return run_joint(a, op, f8, how, dev, s);
    return how.large ? run_large(a, op, f8, how, dev, sms, s) : run_small(a, op, f8, how, dev, s);
}

// What the two routes that lay operands out anew need: the jobs (without their destinations), and their bytes.
void copy_jobs(const LinearArgs& a, int size, CopyJob* x, CopyJob* w) {
    const int piece = 16 / size;
    const long long wn = a.gated ? 2LL * a.N : a.N, w_row = a.nk ? a.K : wn;
    auto up_to = [&](long long n) { return (n + piece - 1) / piece * piece; };
    *x = CopyJob{a.x, nullptr, 0, a.K, up_to(a.K), a.K, up_to(a.K)};
    *w = CopyJob{a.w, nullptr, 0, w_row, up_to(w_row), w_row, up_to(w_row)};
    if (!takes(a.x, a.K, size)) x->rows = a.M;
    // the up half's boxes of a [K, 2 N] weight start at column N, which TMA wants on 16 bytes too
    const bool halves = !a.nk && a.gated;
    if (takes(a.w, w_row, size) && (!halves || a.N % piece == 0)) return;
    w->rows = a.nk ? wn : a.K;
    if (halves) {  // both halves start on a piece
        w->half = a.N;
        w->up = up_to(a.N);
        w->pitch = 2 * w->up;
    }
}
size_t job_bytes(const CopyJob& c, int size) { return (size_t)(c.rows * c.pitch * size); }

void split_jobs(const LinearArgs& a, SplitJob* x, SplitJob* w) {
    const long long wn = a.gated ? 2LL * a.N : a.N;
    auto up_to = [](long long n) { return (n + 7) / 8 * 8; };
    const long long kp = (a.K + 63) / 64 * 64LL;  // whole slabs a term
    *x = SplitJob{static_cast<const float*>(a.x), nullptr, a.M, a.M, a.K, kp, kParts * kp, kp, kp, kp};
    *w = *x;
    w->src = static_cast<const float*>(a.w);
    if (a.nk) {
        w->rows_in = w->rows_out = wn;
        return;
    }
    w->rows_in = a.K;
    w->rows_out = kp;
    w->cols = wn;
    w->half = a.gated ? a.N : up_to(wn);
    w->up = a.gated ? up_to(a.N) : up_to(wn);
    w->width = w->pitch = a.gated ? 2 * w->up : up_to(wn);
    w->plane = kp * w->pitch;
}
size_t job_bytes(const SplitJob& c, bool planes) {
    return (size_t)((planes ? kParts * c.plane : c.rows_out * c.pitch) * 2);
}
constexpr int kSplitBlocks = 1216;  // (8 a GB300's SM; a multiple of 4: see parts_fit_all)

gdn_status run_copies(const LinearArgs& a, bool f8, uint8_t* scratch, int dev, int sms, cudaStream_t s) {
    const int size = f8 ? 1 : 2;
    CopyJob x, w;
    copy_jobs(a, size, &x, &w);
    Operands op{a.x, a.w, a.K, w.cols, a.gated ? 2LL * a.N : a.N, a.N};
    if (x.rows) {
        op.x = x.dst = scratch;
        op.x_pitch = x.pitch;
    }
    if (w.rows) {
        op.w = w.dst = scratch + job_bytes(x, size);
        op.w_pitch = w.pitch;
        if (!a.nk && a.gated) {
            op.up = (int)w.up;
            op.w_cols = w.up + a.N;
        }
    }
    const cudaError_t e = f8 ? launch_plain(linear_align_kernel<uint8_t>, 8u * sms, s, x, w)
                             : launch_plain(linear_align_kernel<uint16_t>, 8u * sms, s, x, w);
    return e == cudaSuccess ? run_tc(a, op, f8, dev, sms, s) : GDN_ERR_CUDA;
}

gdn_status run_parts(const LinearArgs& a, uint8_t* scratch, int dev, int sms, cudaStream_t s, LinearMarks* marks) {
    SplitJob x, w;
    split_jobs(a, &x, &w);
    x.dst = reinterpret_cast<__nv_bfloat16*>(scratch);
    w.dst = reinterpret_cast<__nv_bfloat16*>(scratch + job_bytes(x, false));
    uint8_t* tops = scratch + job_bytes(x, false) + job_bytes(w, !a.nk);
    *marks = LinearMarks{tops, kSplitBlocks};
    if (launch_plain(linear_split_kernel, kSplitBlocks, s, x, w, tops) != cudaSuccess) return GDN_ERR_CUDA;
    const bool halves = !a.nk && a.gated;
    Operands op{x.dst, w.dst, x.pitch, w.pitch, halves ? w.up + a.N : a.gated ? 2LL * a.N : a.N, halves ? (int)w.up : a.N};
    op.tops = tops;
    op.marks = kSplitBlocks;
    const int slabs = slabs_of(a.K, false);
    int share = 0;
    op.accs = accs_of(slabs, &share);
    for (int q = 1; q < op.accs; ++q) op.starts[q] = (q - 1) * share;
    op.plane = 64 * slabs;
    return run_tc(a, op, false, dev, sms, s);
}

}  // namespace

LinearPlan plan_linear(const LinearArgs& a, int32_t dtype) {
    const double ops = 2.0 * a.M * (a.gated ? 2LL * a.N : a.N) * a.K;
    if (dtype == GDN_F32) {
        // Worth the split and two more launches from 3e8 operations.  By parts and on the FFMA kernel, us: M = 128,
        // K = N = 1024 (2.7e8) 14.1 and 11.6, M = 192 15.3 and 19.4; M = 64, K = N = 2048 19.8 and 19.7, M = 96 26.9 and
        // 34.9; M = 16, K = 4096, N = 8192 93 and 126.  Fewer rows than a tile's 16 stay on the FFMA kernel.  Up to
        // K = 4096 the accumulators of a tile are enough for the error to stay that of fp32 sums; past it nothing empties
        // them in between, and the FFMA kernel does the work at 53 TFLOP/s (M = N = 4096, K = 8192: 5.2 ms; 310 by parts
        // at K = 4096, and a library's fp32 product 67).
        if (ops < 3e8 || a.K > 4096 || a.M < 16) return LinearPlan{LinearRoute::kFfma, 0};
        SplitJob x, w;
        split_jobs(a, &x, &w);
        const size_t bytes = job_bytes(x, false) + job_bytes(w, !a.nk) + 2 * kSplitBlocks;
        return bytes > (size_t)4 << 30 ? LinearPlan{LinearRoute::kFfma, 0} : LinearPlan{LinearRoute::kParts, bytes};
    }
    const int size = dtype == GDN_BF16 ? 2 : 1;
    CopyJob x, w;
    copy_jobs(a, size, &x, &w);
    if (x.rows == 0 && w.rows == 0) return LinearPlan{LinearRoute::kTensor, 0};
    // Copies cost about 10 us and then HBM's rate, the FFMA kernel does 47 TFLOP/s: M = 4000, K = 3001, N = 5000
    // (bf16) 100 us and 2.6 ms.
    if (ops < 1e9) return LinearPlan{LinearRoute::kFfma, 0};
    return LinearPlan{LinearRoute::kCopies, job_bytes(x, size) + job_bytes(w, size)};
}

void linear_tc_tiles(const LinearArgs& a, int32_t dtype, LinearRoute route, int sms, gdn_linear_plan_info* info) {
    const int slabs = slabs_of(a.K, dtype == GDN_F8E4M3);
    int share = 0;
    const Plan how = plan(a, slabs, route == LinearRoute::kParts ? accs_of(slabs, &share) : 1, sms);
    info->kernel = !how.large         ? GDN_LINEAR_KERNEL_SMALL
                   : how.splits > 1 ? GDN_LINEAR_KERNEL_JOINT
                                    : GDN_LINEAR_KERNEL_PAIRS;
    info->tokens = how.bn;
    info->splits = how.splits;
}

gdn_status launch_linear_tc(const LinearArgs& a, int32_t dtype, LinearRoute route, void* scratch, int dev, int sms,
                            cudaStream_t s, LinearMarks* marks) {
    uint8_t* p = static_cast<uint8_t*>(scratch);
    const bool f8 = dtype == GDN_F8E4M3;
    if (route == LinearRoute::kParts) return run_parts(a, p, dev, sms, s, marks);
    if (route == LinearRoute::kCopies) return run_copies(a, f8, p, dev, sms, s);
    const long long wn = a.gated ? 2LL * a.N : a.N;
    return run_tc(a, Operands{a.x, a.w, a.K, a.nk ? a.K : wn, wn, a.N}, f8, dev, sms, s);
}

}  // namespace gdn
