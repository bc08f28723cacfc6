// Arguments shared by the kernels of dsa_sparse_mla_decode_fp4 (mla_fp4.cu).
#pragma once

#include "fp4.cuh"

namespace dsa {

constexpr float kLog2e4 = 1.4426950408889634f;

struct MlaF4Args {
    const uint16_t* qlat;
    const int32_t* row_seq;
    const uint8_t* codes;   // [cache rows, 256]
    const uint8_t* scales;  // [cache rows, 32]
    const int32_t* token_ids;
    float* part_o;    // ns > 1: [rows, ns, heads, 512] unnormalised
    float* part_ml;   // ... and [rows, ns, heads, 2]: m and the sum of the weights 2^(s - m)
    float* olat;      // ns == 1, nullable
    uint16_t* olat16; // ns == 1, nullable (bf16)
    int32_t* status;
    Paging pg;
    int rows;
    int heads;
    int ow;
    int ns;
    int tps;
    float scale;   // softmax_scale
    float vscale;  // 2^cache_exp
};

// The tensor-core kernel (mla_fp4_tc.cu): out_width > 0, cache rows below 2^31, splits of
// a multiple of mla_f4_tc_chunk() tokens.
int mla_f4_tc_chunk();
int mla_f4_tc_launch(const MlaF4Args& a, cudaStream_t st);

// The cache row of token t of sequence seq (L tokens), or -1 where there is none; bad ids
// and block entries are flagged.
__device__ __forceinline__ long long f4_token_row(const MlaF4Args& a, int seq, int L, int t) {
    if (t >= 0 && t < L) {
        const long long row = token_row(a.pg, seq, t);
        if (row < 0) flag_status(a.status, DSA_STATUS_BAD_BLOCK);
        return row;
    }
    if (t != -1) flag_status(a.status, DSA_STATUS_BAD_TOKEN);
    return -1;
}

// The power of two that brings the largest finite magnitude (bf16 bits amax) of one head's
// query to [2^14, 2^15): its values convert to f16 without overflow, and exactly from there
// down to 2^-28 of it. Below, they lose bits that the head's f32 sums have no room for. One
// per head: heads of one row may differ by any factor, and each has a softmax of its own. 0
// where the head is all zeros.
__device__ __forceinline__ int f4_q_exp(uint32_t amax) {
    if (amax == 0u) return 0;
    const int e = max((int)(amax >> 7), 1) - 127;  // subnormals: their largest exponent
    return min(14 - e, 126);
}
// Finite magnitudes of two packed bf16, Inf and NaN as 0.
__device__ __forceinline__ uint32_t f4_finite_abs2(uint32_t u) {
    const uint32_t lo = u & 0x7fffu, hi = (u >> 16) & 0x7fffu;
    return (lo < 0x7f80u ? lo : 0u) | (hi < 0x7f80u ? hi << 16 : 0u);
}
__device__ __forceinline__ uint32_t f4_q_half2(uint32_t u, float mul) {
    const __half2 h = __floats2half2_rn(bf16_lo(u) * mul, bf16_hi(u) * mul);
    return *reinterpret_cast<const uint32_t*>(&h);
}

}  // namespace dsa
