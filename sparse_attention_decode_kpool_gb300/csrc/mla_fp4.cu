// dsa_sparse_mla_decode_fp4: latent attention over the selected tokens of an FP4 cache.
//
// Page: metrale_model_arch/glm5next_dsa/mod.rs, "Shape of the pipeline" (last stage) and
// build.rs module doc, transforms 1 and 3 (absorbed Q; each latent row is both key and
// value). Per row r and head h over the selected tokens t, with v[t, :] the decoded row:
//
//   s[t] = softmax_scale * <q[h, :], v[t, :]>,  p = softmax(s),  olat[h, :] = sum_t p[t] v[t, :]
//
// The cache's power of two 2^cache_exp is taken out of v: it multiplies the logits'
// scale and the output once, and the matrix products run on code * scale, which is exact
// in f16. Q goes to f16 too, times a power of two per row and head (f4_q_exp), and the
// probabilities are kept in f16 shifted up by kUp (they reach 2^kUp): a weight is then
// rounded by at most 2^-11 of itself down to 2^(-14 - kUp) of the row's largest, where bf16
// weights would carry 2^-8. Sums (of the rounded weights), maxima and the output
// accumulate in f32.
//
// mla_f4_split_kernel -- one CTA of eight warps per (split of the token list, row, group
// of up to 32 heads), mma.sync m16n8k16. A chunk is 64 tokens; warp w owns tokens
// 8w .. 8w + 7: it resolves them, gathers their 288 bytes with cp.async into its part of
// a three-stage ring, decodes them into the swizzled f16 tile and computes their scores,
// all without the other warps. Then the heads' maxima are exchanged, P goes to shared
// memory, and warp w adds P V for latent columns 64w .. 64w + 63.
#include "mla_fp4.cuh"

namespace dsa {
namespace {

constexpr int KVL = DSA_KV_LORA_RANK;
constexpr int CH = 64;               // tokens per chunk
constexpr int NW = 8;                // warps
constexpr int NTH = NW * 32;
constexpr int ROWB = KVL * 2;        // bytes of a decoded row
constexpr int RAWB = KVL / 2 + KVL / kF4Block;  // 288
constexpr int STAGES = 3;
constexpr int kMaxSplits = 64;       // what the combine kernel takes
constexpr float kUp = 14.f;          // probabilities reach 2^kUp in f16
static_assert(CH == 8 * NW, "a warp owns eight tokens");

// D += A * B, m16n8k16, f16 inputs, f32 accumulate.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t swz(int row, int chunk) {
    return (uint32_t)(row * ROWB + ((chunk ^ (row & 7)) << 4));
}

template <int MT>
struct Smem {
    static constexpr int HP = 16 * MT;
    static constexpr int Q = 0;
    static constexpr int TILE = Q + HP * ROWB;
    static constexpr int RAW = TILE + CH * ROWB;
    static constexpr int P = RAW + STAGES * CH * RAWB;
    static constexpr int RED = P + HP * CH * 2;   // [NW][HP] f32
    static constexpr int MASK = RED + NW * HP * 4;  // [STAGES][CH]
    static constexpr int SCALE = MASK + STAGES * CH;  // [HP] factors of the scores
    static constexpr int BYTES = SCALE + HP * 4;
};

template <int MT>
__global__ void __launch_bounds__(NTH, 1) mla_f4_split_kernel(MlaF4Args a) {
    pdl_wait();
    using S = Smem<MT>;
    constexpr int HP = S::HP;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* Qs = smem + S::Q;
    uint8_t* tile = smem + S::TILE;
    uint8_t* raw = smem + S::RAW;
    uint8_t* Ps = smem + S::P;
    float* red = reinterpret_cast<float*>(smem + S::RED);
    uint8_t* vmask = smem + S::MASK;
    float* scale = reinterpret_cast<float*>(smem + S::SCALE);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, q = lane & 3;
    const int split = blockIdx.x, r = blockIdx.y, head0 = blockIdx.z * HP;
    const int nh = min(HP, a.heads - head0);

    int seq = a.row_seq ? __ldg(a.row_seq + r) : r;
    int L = 0;
    if (seq >= 0 && seq < a.pg.batch) {
        L = min(__ldg(a.pg.seq_lens + seq), seq_capacity(a.pg));
    } else {
        if (tid == 0 && split == 0 && blockIdx.z == 0) flag_status(a.status, DSA_STATUS_BAD_TOKEN);
        seq = 0;
    }
    const int t_begin = split * a.tps;
    const int t_end = min(t_begin + a.tps, a.ow);
    const int nch = t_end > t_begin ? (t_end - t_begin + CH - 1) / CH : 0;

    // This warp's eight tokens of chunk c into ring stage c % STAGES (absent ones as zeros:
    // a masked token's row is never read, so nothing in it can reach the sums).
    auto gather = [&](int c) {
        const int st = c % STAGES;
        long long prow = -1;
        if (lane < 8) {
            const int pos = t_begin + c * CH + warp * 8 + lane;
            if (pos < t_end)
                prow = f4_token_row(a, seq, L, __ldg(a.token_ids + (long long)r * a.ow + pos));
            vmask[st * CH + warp * 8 + lane] = prow >= 0 ? 1 : 0;
        }
        uint8_t* dst = raw + (st * CH + warp * 8) * RAWB;
#pragma unroll
        for (int k = 0; k < (8 * (RAWB / 16) + 31) / 32; ++k) {
            const int i = lane + 32 * k;
            const int j = min(i / (RAWB / 16), 7), c16 = i - j * (RAWB / 16);
            const long long pr = __shfl_sync(0xffffffffu, prow, j);
            if (i < 8 * (RAWB / 16)) {
                const long long row = pr >= 0 ? pr : 0;
                const uint8_t* src = c16 < 16
                                         ? a.codes + row * (KVL / 2) + c16 * 16
                                         : a.scales + row * (KVL / kF4Block) + (c16 - 16) * 16;
                cp_async16(smem_u32(dst + j * RAWB + c16 * 16), src, pr >= 0 ? 16 : 0);
            }
        }
    };
#pragma unroll
    for (int c = 0; c < STAGES - 1; ++c) {
        if (c < nch) gather(c);
        cp_async_commit();
    }

    // Q to f16 (zero rows past the last head), each head times its power of two; warp w has
    // heads 2 MT w .. + 2 MT - 1, a lane two pieces of each.
    {
        const uint16_t* qb = a.qlat + ((long long)r * a.heads + head0) * KVL;
        const float base = a.scale * kLog2e4 * a.vscale;
        uint4 v[2 * MT][2];
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int h = 2 * MT * warp + i;
                v[i][k] = h < nh ? ldg16(qb + h * KVL + (lane + 32 * k) * 8) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) {
            uint32_t m = 0;
#pragma unroll
            for (int k = 0; k < 2; ++k)
                m = __vmaxu2(m, __vmaxu2(__vmaxu2(f4_finite_abs2(v[i][k].x), f4_finite_abs2(v[i][k].y)),
                                         __vmaxu2(f4_finite_abs2(v[i][k].z), f4_finite_abs2(v[i][k].w))));
            const int h = 2 * MT * warp + i;
            const int qe = f4_q_exp(__reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16)));
            const float mul = pow2f(qe);
#pragma unroll
            for (int k = 0; k < 2; ++k)
                *reinterpret_cast<uint4*>(Qs + swz(h, lane + 32 * k)) =
                    make_uint4(f4_q_half2(v[i][k].x, mul), f4_q_half2(v[i][k].y, mul),
                               f4_q_half2(v[i][k].z, mul), f4_q_half2(v[i][k].w, mul));
            if (lane == 0) scale[h] = base * pow2f(-qe);
        }
        __syncthreads();
    }
    float sl0[MT], sl1[MT];  // scores to logits in log2 units, heads 16 i + g and + 8
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        sl0[i] = scale[16 * i + g];
        sl1[i] = scale[16 * i + g + 8];
    }

    float m0[MT], m1[MT], l0[MT], l1[MT];  // heads 16 i + g and + 8: running max, this warp's sums
    float oacc[MT][8][4];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        m0[i] = m1[i] = -INFINITY;
        l0[i] = l1[i] = 0.f;
#pragma unroll
        for (int n = 0; n < 8; ++n)
            oacc[i][n][0] = oacc[i][n][1] = oacc[i][n][2] = oacc[i][n][3] = 0.f;
    }
    const int mi = lane >> 3;
    const int arow = (lane & 7) + ((lane >> 3) & 1) * 8;

    for (int c = 0; c < nch; ++c) {
        const int st = c % STAGES;
        if (c + STAGES - 1 < nch) gather(c + STAGES - 1);
        cp_async_commit();
        cp_async_wait<STAGES - 1>();
        __syncthreads();  // Q in place (c == 0); the tile's readers of chunk c - 1 are done

        // ---- decode this warp's tokens: 16-channel block b of token j, 8 bytes each
        {
            const uint8_t* rb = raw + (st * CH + warp * 8) * RAWB;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint8_t* row = rb + k * RAWB;
                const uint2 cw = *reinterpret_cast<const uint2*>(row + lane * 8);
                const uint32_t s = row[KVL / 2 + lane];
                const uint32_t s2 = e4m3x2_to_f16x2(s | (s << 8));
                *reinterpret_cast<uint4*>(tile + swz(warp * 8 + k, 2 * lane)) = fp4_decode8(cw.x, s2);
                *reinterpret_cast<uint4*>(tile + swz(warp * 8 + k, 2 * lane + 1)) =
                    fp4_decode8(cw.y, s2);
            }
        }
        __syncwarp();

        // ---- S = Q K^T: MT x 16 heads by this warp's 8 tokens
        float sacc[MT][4];
#pragma unroll
        for (int i = 0; i < MT; ++i) sacc[i][0] = sacc[i][1] = sacc[i][2] = sacc[i][3] = 0.f;
#pragma unroll 4
        for (int kk = 0; kk < KVL / 32; ++kk) {
            uint32_t bf[4];  // k-steps 2 kk and 2 kk + 1
            ldsm_x4(bf, smem_u32(tile + swz(warp * 8 + (lane & 7), 4 * kk + mi)));
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                uint32_t a0[4], a1[4];
                ldsm_x4(a0, smem_u32(Qs + swz(16 * i + arow, 4 * kk + (lane >> 4))));
                ldsm_x4(a1, smem_u32(Qs + swz(16 * i + arow, 4 * kk + 2 + (lane >> 4))));
                mma_f16(sacc[i], a0, bf[0], bf[1]);
                mma_f16(sacc[i], a1, bf[2], bf[3]);
            }
        }
        const bool ok0 = vmask[st * CH + warp * 8 + 2 * q] != 0;
        const bool ok1 = vmask[st * CH + warp * 8 + 2 * q + 1] != 0;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            sacc[i][0] = ok0 ? sacc[i][0] * sl0[i] : -INFINITY;
            sacc[i][1] = ok1 ? sacc[i][1] * sl0[i] : -INFINITY;
            sacc[i][2] = ok0 ? sacc[i][2] * sl1[i] : -INFINITY;
            sacc[i][3] = ok1 ? sacc[i][3] * sl1[i] : -INFINITY;
            float x0 = fmaxf(sacc[i][0], sacc[i][1]), x1 = fmaxf(sacc[i][2], sacc[i][3]);
            x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
            x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
            x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
            x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2));
            if (q == 0) {
                red[warp * HP + 16 * i + g] = x0;
                red[warp * HP + 16 * i + g + 8] = x1;
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            float n0 = m0[i], n1 = m1[i];
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                n0 = fmaxf(n0, red[w * HP + 16 * i + g]);
                n1 = fmaxf(n1, red[w * HP + 16 * i + g + 8]);
            }
            // all logits so far absent (or -inf): any finite stand-in gives weights 0
            const float u0 = n0 == -INFINITY ? 0.f : n0, u1 = n1 == -INFINITY ? 0.f : n1;
            const float al0 = exp2f(m0[i] - u0), al1 = exp2f(m1[i] - u1);
            m0[i] = n0;
            m1[i] = n1;
            const __half2 p0 = __floats2half2_rn(exp2f(sacc[i][0] - u0 + kUp),
                                                 exp2f(sacc[i][1] - u0 + kUp));
            const __half2 p1 = __floats2half2_rn(exp2f(sacc[i][2] - u1 + kUp),
                                                 exp2f(sacc[i][3] - u1 + kUp));
            const float2 f0 = __half22float2(p0), f1 = __half22float2(p1);
            l0[i] = l0[i] * al0 + (f0.x + f0.y);
            l1[i] = l1[i] * al1 + (f1.x + f1.y);
            const int h0 = 16 * i + g, h1 = h0 + 8;
            *reinterpret_cast<__half2*>(Ps + h0 * (CH * 2) + ((warp ^ (h0 & 7)) << 4) + 4 * q) = p0;
            *reinterpret_cast<__half2*>(Ps + h1 * (CH * 2) + ((warp ^ (h1 & 7)) << 4) + 4 * q) = p1;
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                oacc[i][n][0] *= al0;
                oacc[i][n][1] *= al0;
                oacc[i][n][2] *= al1;
                oacc[i][n][3] *= al1;
            }
        }
        __syncthreads();

        // ---- O += P V, latent columns 64 warp .. + 63
#pragma unroll
        for (int kk = 0; kk < CH / 16; ++kk) {
            uint32_t af[MT][4];
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int h = 16 * i + arow;
                ldsm_x4(af[i], smem_u32(Ps + h * (CH * 2) + (((2 * kk + (lane >> 4)) ^ (h & 7)) << 4)));
            }
            const int tok = kk * 16 + (mi & 1) * 8 + (lane & 7);
#pragma unroll
            for (int dp = 0; dp < 4; ++dp) {
                uint32_t bf[4];
                ldsm_x4_t(bf, smem_u32(tile + swz(tok, warp * 8 + 2 * dp + (mi >> 1))));
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    mma_f16(oacc[i][2 * dp], af[i], bf[0], bf[1]);
                    mma_f16(oacc[i][2 * dp + 1], af[i], bf[2], bf[3]);
                }
            }
        }
    }
    cp_async_wait<0>();

    // ---- the warps' sums, in warp order
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        l0[i] += __shfl_xor_sync(0xffffffffu, l0[i], 1);
        l1[i] += __shfl_xor_sync(0xffffffffu, l1[i], 1);
        l0[i] += __shfl_xor_sync(0xffffffffu, l0[i], 2);
        l1[i] += __shfl_xor_sync(0xffffffffu, l1[i], 2);
        if (q == 0) {
            red[warp * HP + 16 * i + g] = l0[i];
            red[warp * HP + 16 * i + g + 8] = l1[i];
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int h = 16 * i + g + 8 * half;
            if (h >= nh) continue;
            float l = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) l += red[w * HP + h];
            const int d0 = warp * 64 + 2 * q;
            if (a.ns == 1) {
                // a NaN sum (a NaN in q or in a selected row) keeps its NaN
                const float k = l == 0.f ? 0.f : a.vscale / l;
                const long long o = ((long long)r * a.heads + head0 + h) * KVL + d0;
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                    const float x = oacc[i][n][2 * half] * k, y = oacc[i][n][2 * half + 1] * k;
                    if (a.olat) *reinterpret_cast<float2*>(a.olat + o + 8 * n) = make_float2(x, y);
                    if (a.olat16)
                        *reinterpret_cast<uint32_t*>(a.olat16 + o + 8 * n) = pack_bf16x2(x, y);
                }
            } else {
                const long long u = ((long long)r * a.ns + split) * a.heads + head0 + h;
#pragma unroll
                for (int n = 0; n < 8; ++n)
                    *reinterpret_cast<float2*>(a.part_o + u * KVL + d0 + 8 * n) = make_float2(
                        oacc[i][n][2 * half] * a.vscale, oacc[i][n][2 * half + 1] * a.vscale);
                if (warp == 0 && q == 0)
                    *reinterpret_cast<float2*>(a.part_ml + u * 2) =
                        make_float2(half ? m1[i] : m0[i], l);
            }
        }
}

// Merges the splits of a row: a warp per 128 C latent columns of a (row, head), a lane per
// C four-column pieces, E splits at a time. C E = 16 loads of 16 bytes are under way per
// lane, whether the splits are many (a few rows) or two (many rows): with C = 1 and two
// splits the 64-row merge took 11 us, with a block per (row, head) 8. They are asked for
// before the weights 2^(m_s - max) are known, which the warp takes from the splits' (m, l)
// pairs, a lane per pair. Sums in split order.
constexpr int kMergeWarps = 4;
template <int C>
__global__ void __launch_bounds__(kMergeWarps * 32) mla_f4_merge_kernel(
    const float* __restrict__ part_o, const float* __restrict__ part_ml, long long rh, int heads,
    int ns, float* olat, uint16_t* olat16) {
    pdl_trigger();  // the projection after it streams weights that do not depend on it
    pdl_wait();
    constexpr int E = 16 / C, W = 4 / C;  // splits at a time, warps per (row, head)
    const int lane = threadIdx.x & 31;
    const long long u = (long long)blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
    const long long i = u / W;  // row * heads + head
    if (i >= rh) return;
    const int r = (int)(i / heads), h = (int)(i - (long long)r * heads);
    const long long first = ((long long)r * ns) * heads + h;  // split 0's entry, + heads each
    const int col = (int)(u % W) * (32 * C) + lane;           // in pieces of four columns
    const float4* po = reinterpret_cast<const float4*>(part_o) + first * (KVL / 4) + col;
    const long long step = (long long)heads * (KVL / 4);
    float4 o[E][C];
    auto load = [&](int s0) {
#pragma unroll
        for (int s = 0; s < E; ++s)
#pragma unroll
            for (int c = 0; c < C; ++c)
                o[s][c] = s0 + s < ns ? __ldg(po + (s0 + s) * step + 32 * c)
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    load(0);
    float w[2], l[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int s = lane + 32 * k;
        const float2 ml = s < ns ? __ldg(reinterpret_cast<const float2*>(part_ml) + first +
                                         (long long)s * heads)
                                 : make_float2(-INFINITY, 0.f);
        w[k] = ml.x;
        l[k] = ml.y;
    }
    float top = fmaxf(w[0], w[1]);
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        w[k] = w[k] == -INFINITY ? 0.f : exp2f(w[k] - top);
        sum += w[k] * l[k];  // NaN where a split's sum is NaN
    }
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
    float4 acc[C];
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < ns; s0 += E) {
        if (s0 > 0) load(s0);
#pragma unroll
        for (int s = 0; s < E; ++s) {
            const float ws = __shfl_sync(0xffffffffu, s0 + s < 32 ? w[0] : w[1], (s0 + s) & 31);
            if (s0 + s < ns) {
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    acc[c].x = fmaf(ws, o[s][c].x, acc[c].x);
                    acc[c].y = fmaf(ws, o[s][c].y, acc[c].y);
                    acc[c].z = fmaf(ws, o[s][c].z, acc[c].z);
                    acc[c].w = fmaf(ws, o[s][c].w, acc[c].w);
                }
            }
        }
    }
    const float k = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const long long at = i * KVL + 4 * (col + 32 * c);
        const float4 x = make_float4(acc[c].x * k, acc[c].y * k, acc[c].z * k, acc[c].w * k);
        if (olat) *reinterpret_cast<float4*>(olat + at) = x;
        if (olat16)
            *reinterpret_cast<uint2*>(olat16 + at) =
                make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
    }
}

template <int C>
int launch_merge(const MlaF4Args& a, float* olat, uint16_t* olat16, cudaStream_t st) {
    const long long rh = (long long)a.rows * a.heads, warps = rh * (4 / C);
    cudaError_t e = launch_pdl(mla_f4_merge_kernel<C>,
                               dim3((unsigned)((warps + kMergeWarps - 1) / kMergeWarps)),
                               dim3(kMergeWarps * 32), 0, st, (const float*)a.part_o,
                               (const float*)a.part_ml, rh, a.heads, a.ns, olat, olat16);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "dsa_sparse_mla_decode_fp4 merge launch");
    return DSA_OK;
}

// ---------------------------------------------------------------------------
struct F4Plan {
    bool tc;  // the tcgen05 kernel (mla_fp4_tc.cu), else the mma.sync kernel above
    int mt, hgroups, ns, tps;
    long long cost;  // estimated time, tenths of a microsecond
    size_t off_part_o, off_part_ml, off_xbf, off_proj, bytes;
};
size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }

F4Plan f4_plan(bool tc, int rows, int heads, int ow, int hidden, bool with_oabs, int sms) {
    F4Plan p;
    p.tc = tc;
    p.mt = heads <= 16 ? 1 : 2;
    p.hgroups = tc ? (heads + 63) / 64 : (heads + 16 * p.mt - 1) / (16 * p.mt);
    const int chunk = tc ? mla_f4_tc_chunk() : CH;
    const long long base = (long long)rows * p.hgroups;
    const long long cpr = ow > 0 ? (ow + chunk - 1) / chunk : 1;  // chunks per row
    p.tps = (int)cpr * chunk;
    p.ns = 1;
    // Estimated time, in tenths of a microsecond, fitted to a sweep of 1 to 128 heads, 1 to
    // 2,048 rows and 64 to 2,048 tokens: the busiest CTA walks ceil(units / sms) units of
    // ceil(chunks / ns) chunks. A chunk takes the tcgen05 kernel (128 tokens, any number
    // of heads up to 64) 2.8 us and a unit 4.5 us more (its first chunk's latencies, Q)
    // plus up to 2 for the output; the mma.sync kernel 2.8 us (64 tokens, 16 heads) or 4.4
    // (32 heads) and a unit 1 or 1.5. Splitting costs the merge, 1.8 us and its bytes at
    // 6 TB/s. The split count that makes this smallest, the fewest on ties.
    const long long per_chunk = tc ? 28 : p.mt == 1 ? 28 : 44;
    const long long per_unit = tc ? 45 + 20 * (heads < 64 ? heads : 64) / 64 : p.mt == 1 ? 10 : 15;
    p.cost = -1;
    for (long long t = 1; t <= cpr && t <= kMaxSplits; ++t) {
        const long long tps = (cpr + t - 1) / t;
        const long long ns = (cpr + tps - 1) / tps;
        long long cost = (tc ? 15 : 20) + (base * ns + sms - 1) / sms * (tps * per_chunk + per_unit);
        if (ns > 1) cost += 18 + rows * ns * heads * (KVL * 4LL) / 600000;
        if (p.cost < 0 || cost < p.cost) {
            p.cost = cost;
            p.tps = (int)tps * chunk;
            p.ns = (int)ns;
        }
    }
    size_t off = 0;
    p.off_part_o = off;
    if (p.ns > 1) off += al256((size_t)rows * p.ns * heads * KVL * 4);
    p.off_part_ml = off;
    if (p.ns > 1) off += al256((size_t)rows * p.ns * heads * 2 * 4);
    p.off_xbf = off;
    if (with_oabs) off += al256((size_t)rows * heads * KVL * 2);
    p.off_proj = off;
    if (with_oabs) off += al256(project_workspace_bytes(rows, heads * KVL, hidden, sms));
    p.bytes = off;
    return p;
}

// Enough for either kernel: the call's choice depends on the cache's size too, and a
// workspace serves whichever kernel the option names when it is used.
size_t f4_bytes(int rows, int heads, int ow, int hidden, bool with_oabs, int sms) {
    const size_t b0 = f4_plan(false, rows, heads, ow, hidden, with_oabs, sms).bytes;
    const size_t b1 = f4_plan(true, rows, heads, ow, hidden, with_oabs, sms).bytes;
    return b0 > b1 ? b0 : b1;
}

// Which kernel: DSA_OPT_MLA_KERNEL's, else the one with the smaller estimate. Measured, mma
// against tcgen05: 16 heads, 8 rows of 2,048 tokens 10.6 us against 11.8; 24 heads 13.4
// against 12.0; 4 heads, 64 rows of 256 tokens 9.9 against 11.8, of 1,000 26 against 19;
// 64 heads, 8 rows of 256 tokens 9.8 against 12.4, of 2,048 21 against 14.0.
bool f4_use_tc(int rows, int heads, int ow, long long cache_rows, int sms) {
    if (ow < 1 || cache_rows > 0x7fffffffLL) return false;
    switch (mla_kernel_choice()) {
        case DSA_MLA_KERNEL_TCGEN05: return true;
        case DSA_MLA_KERNEL_MMA: return false;
        default:
            return f4_plan(true, rows, heads, ow, 0, false, sms).cost <
                   f4_plan(false, rows, heads, ow, 0, false, sms).cost;
    }
}

int check_f4(int rows, int heads, int kvl, int ow, int hidden, bool with_oabs) {
    if (rows < 0 || heads < 1 || ow < 0)
        return fail(DSA_ERR_INVALID_ARG,
                    "dsa_sparse_mla_decode_fp4: rows %d, heads %d, out_width %d", rows, heads, ow);
    if (kvl != KVL)
        return fail(kvl == 0 ? DSA_ERR_CONFIG : DSA_ERR_UNSUPPORTED,
                    "dsa_sparse_mla_decode_fp4: kv_lora_rank %d, kernels are built for %d", kvl,
                    KVL);
    if (rows > 65535)
        return fail(DSA_ERR_UNSUPPORTED, "dsa_sparse_mla_decode_fp4: rows %d > 65535", rows);
    if (heads > 4096)
        return fail(DSA_ERR_UNSUPPORTED, "dsa_sparse_mla_decode_fp4: heads %d > 4096", heads);
    if (with_oabs && !project_supported(heads * KVL, hidden))
        return fail(DSA_ERR_UNSUPPORTED,
                    "dsa_sparse_mla_decode_fp4: hidden %d must be a positive multiple of 64",
                    hidden);
    return DSA_OK;
}

template <int MT>
int launch_split(const MlaF4Args& a, const F4Plan& p, cudaStream_t st) {
    static_assert(Smem<MT>::BYTES <= 227 * 1024, "split kernel shared memory");
    int rc = set_max_smem((const void*)mla_f4_split_kernel<MT>, Smem<MT>::BYTES);
    if (rc) return rc;
    cudaError_t e = launch_pdl(mla_f4_split_kernel<MT>, dim3(p.ns, a.rows, p.hgroups), dim3(NTH),
                               Smem<MT>::BYTES, st, a);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "dsa_sparse_mla_decode_fp4 split launch");
    return DSA_OK;
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" int dsa_sparse_mla_decode_fp4_workspace(int rows, int heads, int kv_lora_rank,
                                                   int out_width, int hidden, int with_o_absorb,
                                                   size_t* bytes) {
    if (!bytes)
        return fail(DSA_ERR_INVALID_ARG, "dsa_sparse_mla_decode_fp4_workspace: bytes is NULL");
    int rc = check_f4(rows, heads, kv_lora_rank, out_width, hidden, with_o_absorb != 0);
    if (rc) return rc;
    const int sms = sm_count();
    if (sms <= 0)
        return fail(DSA_ERR_CUDA, "dsa_sparse_mla_decode_fp4_workspace: no CUDA device");
    *bytes = f4_bytes(rows, heads, out_width, hidden, with_o_absorb != 0, sms);
    return DSA_OK;
}

extern "C" int dsa_sparse_mla_decode_fp4_splits(int rows, int heads, int kv_lora_rank,
                                                int out_width, long long cache_rows,
                                                int* splits) {
    if (!splits)
        return fail(DSA_ERR_INVALID_ARG, "dsa_sparse_mla_decode_fp4_splits: splits is NULL");
    int rc = check_f4(rows, heads, kv_lora_rank, out_width, 0, false);
    if (rc) return rc;
    const int sms = sm_count();
    if (sms <= 0)
        return fail(DSA_ERR_CUDA, "dsa_sparse_mla_decode_fp4_splits: no CUDA device");
    const bool tc = f4_use_tc(rows, heads, out_width, cache_rows, sms);
    *splits = f4_plan(tc, rows, heads, out_width, 0, false, sms).ns;
    return DSA_OK;
}

extern "C" int dsa_sparse_mla_decode_fp4(const dsa_bf16* qlat, int rows, int heads,
                                         int kv_lora_rank, const int32_t* row_seq,
                                         const uint8_t* ckv_codes, const uint8_t* ckv_scales,
                                         int cache_exp, const dsa_paging* pg,
                                         const int32_t* token_ids, int out_width,
                                         float softmax_scale, const dsa_bf16* o_absorb, int hidden,
                                         dsa_bf16* y, float* olat, dsa_bf16* olat16,
                                         int32_t* status, void* workspace, size_t workspace_bytes,
                                         void* stream) {
    const bool with_oabs = o_absorb != nullptr;
    int rc = check_f4(rows, heads, kv_lora_rank, out_width, hidden, with_oabs);
    if (rc) return rc;
    if (cache_exp < -kF4MaxExp || cache_exp > kF4MaxExp)
        return fail(DSA_ERR_INVALID_ARG,
                    "dsa_sparse_mla_decode_fp4: cache_exp %d outside [-%d, %d]", cache_exp,
                    kF4MaxExp, kF4MaxExp);
    if (with_oabs != (y != nullptr))
        return fail(DSA_ERR_INVALID_ARG,
                    "dsa_sparse_mla_decode_fp4: o_absorb and y must be both given or both NULL");
    Paging P;
    rc = check_paging(pg, 0, &P);
    if (rc) return rc;
    if (rows == 0) return DSA_OK;
    if (!qlat || !ckv_codes || !ckv_scales || (out_width > 0 && !token_ids))
        return fail(DSA_ERR_INVALID_ARG, "dsa_sparse_mla_decode_fp4: NULL tensor");
    if ((((uintptr_t)qlat) | ((uintptr_t)ckv_codes) | ((uintptr_t)ckv_scales) |
         ((uintptr_t)o_absorb) | ((uintptr_t)olat) | ((uintptr_t)olat16) | ((uintptr_t)y) |
         ((uintptr_t)workspace)) & 15)
        return fail(DSA_ERR_INVALID_ARG,
                    "dsa_sparse_mla_decode_fp4: tensors must be 16-byte aligned");
    if (!olat && !olat16 && !with_oabs) return DSA_OK;  // nothing requested
    const int sms = sm_count();
    if (sms <= 0) return fail(DSA_ERR_CUDA, "dsa_sparse_mla_decode_fp4: no CUDA device");
    const long long cache_rows = P.block_table ? P.num_blocks * P.block_size
                                               : (long long)P.batch * P.max_seq_len;
    const F4Plan p = f4_plan(f4_use_tc(rows, heads, out_width, cache_rows, sms), rows, heads, out_width,
                             hidden, with_oabs, sms);
    const size_t need = f4_bytes(rows, heads, out_width, hidden, with_oabs, sms);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(DSA_ERR_INVALID_ARG,
                    "dsa_sparse_mla_decode_fp4: workspace %zu B < %zu B needed", workspace_bytes,
                    need);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    cudaStream_t st = (cudaStream_t)stream;
    // the projection reads a bf16 olat: the caller's where there is one
    uint16_t* x16 = olat16 ? olat16
                           : with_oabs ? reinterpret_cast<uint16_t*>(ws + p.off_xbf) : nullptr;
    MlaF4Args a;
    a.qlat = qlat;
    a.row_seq = row_seq;
    a.codes = ckv_codes;
    a.scales = ckv_scales;
    a.token_ids = token_ids;
    a.part_o = p.ns > 1 ? reinterpret_cast<float*>(ws + p.off_part_o) : nullptr;
    a.part_ml = p.ns > 1 ? reinterpret_cast<float*>(ws + p.off_part_ml) : nullptr;
    a.olat = olat;
    a.olat16 = x16;
    a.status = status;
    a.pg = P;
    a.rows = rows;
    a.heads = heads;
    a.ow = out_width;
    a.ns = p.ns;
    a.tps = p.tps;
    a.scale = softmax_scale;
    a.vscale = ldexpf(1.f, cache_exp);
    rc = p.tc ? mla_f4_tc_launch(a, st)
              : p.mt == 1 ? launch_split<1>(a, p, st) : launch_split<2>(a, p, st);
    if (rc) return rc;
    if (p.ns > 1) {
        rc = p.ns <= 4   ? launch_merge<4>(a, olat, x16, st)
             : p.ns <= 8 ? launch_merge<2>(a, olat, x16, st)
                         : launch_merge<1>(a, olat, x16, st);
        if (rc) return rc;
    }
    if (with_oabs)
        return project_launch(x16, false, rows, heads * KVL, o_absorb, hidden, y, status,
                              ws + p.off_proj, workspace_bytes - p.off_proj, st);
    return DSA_OK;
}
