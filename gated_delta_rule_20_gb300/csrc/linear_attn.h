// linear_attn.h -- declarations shared by the parts of linear attention with a decay for each head
// (linear_attn.cu: entry points, the single-token step and the fp32 kernel; linear_attn_tc.cu: the
// tensor-core kernel).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "gdn.h"

namespace gdn {

// One call's arguments after host-side validation.
struct LinearAttn {
    const void* q;
    const void* k;
    const void* v;
    const float* g_log;      // [B, Hv, S], or [Hv] with head_decay
    const int32_t* lengths;  // [B], or null: S tokens each
    const float* state_in;   // null: zeros
    float* state_out;
    void* out;
    float scale;
    int B, Hk, Hv, S, Dk, Dv;
    bool bf16, head_decay;
    bool zero_rest;  // rows of out behind a sequence's length are zeroed (only with lengths)
    int Pk, Pv;      // channels from a row to the next, of q and k and of v and out (the FMA units: Dk and Dv)
};

// Least log-decay that is told from the others: e^-100 = 3.7e-44 is (nearly) the least fp32 number, so that
// nothing is left of a state behind it, and sums of a chunk's log-decays stay finite (a g_log of -inf
// starts a new sequence).
constexpr float kMinLogDecay = -100.f;
__device__ __forceinline__ float least_decay(float g) { return g < kMinLogDecay ? kMinLogDecay : g; }  // (NaN stays)

// n / d for 0 <= n < 2^31 as the high half of a product: m = ceil(2^(31 + s) / d), 2^(s - 1) < d <= 2^s.
struct Divisor {
    uint32_t m;
    int s;
    __device__ __forceinline__ int of(int n) const { return (int)(__umulhi(2u * (uint32_t)n, m) >> s); }
};
inline Divisor divisor(int d) {
    int s = 0;
    while ((1ll << s) < d) ++s;
    return Divisor{(uint32_t)(((1ull << (31 + s)) + d - 1) / d), s};
}

// Segments of every sequence (P = 1: whole).  Segment j holds tokens [j len, (j + 1) len) of S.  A first launch runs
// segments 0 .. P - 2 from zero (segment 0: from state_in) and leaves their end states X_j in `parts` [P][B Hv][Dk Dv]
// and their decays F_j in `decays` [P][B Hv]; a second adds them up in place, X_j += F_j X_{j-1}, so that slot j is the
// start state of segment j + 1; a third runs all segments.  Slot P - 1 keeps a copy of state_in for segment 0, since
// segment P - 1 may write state_out in its place before segment 0 has read it.
struct LinearAttnSplit {
    int P, len;
    float* parts;
    float* decays;
    // P = 1 on the tensor cores, where the heads are some rounds of all SMs and a few more: CTAs that run parts of `len` tokens of
    // these, handing the state on (0: none), and their flags
    int handed;
    uint32_t* flags;
    __device__ const float* start(int seg, long long bh, long long heads, long long n) const {
        return parts + ((seg ? seg - 1 : P - 1) * heads + bh) * n;
    }
};
inline size_t linear_attn_split_bytes(const LinearAttn& p, int P) {
    return P <= 1 ? 0 : (size_t)P * p.B * p.Hv * ((size_t)p.Dk * p.Dv + 1) * sizeof(float);
}

inline size_t linear_attn_flag_bytes(int handed) { return handed ? ((size_t)handed * 8 + 1) * sizeof(uint32_t) : 0; }

// bf16, rows (of Pk and Pv channels) and pointers of whole 16 bytes: all launches of a split, or the one of P = 1.
gdn_status launch_linear_attn_tc(const LinearAttn& p, const LinearAttnSplit& s, int dev, int sms, int32_t* status,
                                 cudaStream_t stream);

// The second launch (nothing for P = 2).
cudaError_t launch_linear_attn_combine(const LinearAttn& p, const LinearAttnSplit& s, cudaStream_t stream);

}  // namespace gdn
