// dsa_sparse_mla_decode_fp4 on the tensor cores (tcgen05): 64 heads at a time, a
// persistent grid over (row, head group, split) units, 128 tokens per chunk.
//
//   S^T = V Q^T     M = 128 tokens, N = 64 heads, K = 512 latent columns
//   O^T += V^T P^T  M = 512 latent columns (four tiles), N = 64 heads, K = 128 tokens
//
// V is the chunk's decoded rows in f16 (128 x 512, 128 KB of shared memory in 128-byte
// swizzle atoms): one tile serves both products, K-major for the scores and MN-major for
// the values. With Q (64 KB) and P (16 KB) there is no room for a second tile, nor for a
// stage of undecoded rows; instead the next chunk's 288 bytes per token wait in registers
// (18 of them in each of 512 threads), loaded a chunk ahead, so the tile's refill is
// arithmetic and shared-memory stores only. It is refilled a quarter (128 columns) at a
// time, as the value product of the chunk before leaves it, and the score product starts
// on a quarter as soon as it is filled.
//
// Sixteen worker warps do everything but addresses and MMA issue; what they do in a chunk
// follows from what is ready: decode the four quarters, request the next chunk's rows,
// softmax. In the softmax warp w has tensor-memory lane quarter w & 3 (32 tokens) and
// heads 16 (w >> 2) .. + 15. A head's running maximum is moved only when a score exceeds
// it by more than kLazy (or there is none yet): one vote per chunk among the four warps
// of a head group, and only after such a vote are maxima exchanged and O^T rescaled.
// Weights are held at 2^kUpTc over the maximum, so with the lag they reach 2^15 in f16; the
// sums that divide the output take them unrounded.
//
// Warps 16 and 18 resolve token ids to cache rows, chunks ahead; warp 17 issues the MMAs.
//
// Waits are bounded: one that runs out sets DSA_STATUS_TIMEOUT and a flag that makes all
// later waits return at once; every role then runs its loops to the end (rows stay
// checked ones), so named barriers stay matched, and the tensor memory is released.
#include <float.h>

#include "mla_fp4.cuh"
#include "tc.cuh"

namespace dsa {
namespace {

constexpr int kT = 128;  // tokens per chunk
constexpr int kH = 64;   // heads per unit
constexpr int kKVL = 512;
constexpr int kAtoms = kKVL / 64;
constexpr uint32_t kLatAtom = kT * 128;
constexpr uint32_t kQAtom = kH * 128;
constexpr int kRing = 4;  // chunks of resolved rows
constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffLat = kOffQ + kAtoms * kQAtom;
constexpr uint32_t kOffP = kOffLat + kAtoms * kLatAtom;
constexpr uint32_t kOffRows = kOffP + kT * 128;         // [kRing][kT] cache row, or -1
constexpr uint32_t kOffRed = kOffRows + kRing * kT * 4;  // [4][kH] chunk maxima
constexpr uint32_t kOffSums = kOffRed + 4 * kH * 4;      // [4][kH] head sums
constexpr uint32_t kOffK = kOffSums + 4 * kH * 4;        // [kH] factors of the output
constexpr uint32_t kOffQmax = kOffK + kH * 4;            // [16] a warp's largest and smallest head
constexpr uint32_t kOffScale = kOffQmax + 16 * 4;        // [kH] factors of the scores
constexpr uint32_t kOffOwn = kOffScale + kH * 4;         // [16] whether `scale` counts
constexpr uint32_t kOffBar = kOffOwn + 16 * 4;
constexpr int ROWS_FULL = 0;                    // [kRing]
constexpr int ROWS_EMPTY = ROWS_FULL + kRing;   // [kRing]
constexpr int LAT_FULL = ROWS_EMPTY + kRing;    // [4] quarter decoded
constexpr int LAT_EMPTY = LAT_FULL + 4;         // [4] quarter's value product done
constexpr int Q_FULL = LAT_EMPTY + 4;
constexpr int S_FULL = Q_FULL + 1;
constexpr int P_FULL = S_FULL + 1;
constexpr int O_DONE = P_FULL + 1;
constexpr int O_FREE = O_DONE + 1;
constexpr int DRAIN = O_FREE + 1;
constexpr int kBars = DRAIN + 1;
constexpr uint32_t kOffMisc = kOffBar + kBars * 8;
constexpr uint32_t kBytes = kOffMisc + 16;
constexpr uint32_t kDyn = kBytes + 1024;
static_assert(kDyn <= 227 * 1024, "shared memory");
static_assert(kOffBar % 8 == 0 && kOffRows % 16 == 0 && kOffScale % 16 == 0, "alignment");
constexpr uint32_t kTmemCols = 512;  // S^T: columns [0, 64); O^T tile i: [64 + 64 i, + 64)
constexpr int kWorkers = 16;
constexpr int kThreads = (kWorkers + 4) * 32;
// Launched at 96 registers a thread (640 x 96 of the SM's 65,536); the four worker
// warpgroups take 104 and the fifth 64: 4 x 104 + 64 = 5 x 96.
constexpr int kRegLow = 64, kRegHigh = 104;
static_assert(4 * kRegHigh + kRegLow <= 5 * 96, "register split");
constexpr float kLazy = 8.f;
// Heads whose maxima of |q| are within 2^kSame share one power of two: the smallest one's
// values are then exact in f16 down to 2^-23 of its maximum and off by 2^-31 of it below.
constexpr int kSame = 8;
constexpr float kUpTc = 7.f;  // weights reach 2^(kUpTc + kLazy) = 2^15

// The descriptor `bytes` further on (an operand's next 16 columns or rows).
__device__ __forceinline__ uint64_t desc_at(uint64_t d, uint32_t bytes) { return d + (bytes >> 4); }
// D f32, A and B f16.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// 16 consecutive f32 columns of this thread's lane, loaded and complete.
__device__ __forceinline__ void tc_ld16(uint32_t (&v)[16], uint32_t taddr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15}, [%16];\n"
        "tcgen05.wait::ld.sync.aligned;\n"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]),
          "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16};\n" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
        "r"(v[15])
        : "memory");
}
// Reduce-scatter of 16 values over a warp: lane l ends with op over all lanes of value
// l / 2.
template <typename Op>
__device__ __forceinline__ float scatter16(float (&v)[16], int lane, Op op) {
#pragma unroll
    for (int w = 8, m = 16; w >= 1; w >>= 1, m >>= 1) {
        const bool hi = (lane & m) != 0;
#pragma unroll
        for (int i = 0; i < w; ++i) {
            const float got = __shfl_xor_sync(0xffffffffu, hi ? v[i] : v[w + i], m);
            v[i] = op(hi ? v[w + i] : v[i], got);
        }
    }
    return op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
}
// The smaller of the two, NaN where one is.
__device__ __forceinline__ float min_nan(float x, float y) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void prefetch_l2(const void* p) {
    asm volatile("prefetch.global.L2 [%0];\n" ::"l"(p));
}
__device__ __forceinline__ void bar_sync(int id, int threads) {
    asm volatile("barrier.cta.sync %0, %1;\n" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ bool bar_any(int id, int threads, bool p) {
    uint32_t r;
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\n"
        "barrier.cta.red.or.pred q, %2, %3, p;\nselp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"((uint32_t)p), "r"(id), "r"(threads)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void sts16(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};\n" ::"r"(addr), "r"(v.x), "r"(v.y),
                 "r"(v.z), "r"(v.w)
                 : "memory");
}
// A warp waits for a phase, for about a second at most; after a timeout (here or in another
// role) it returns at once. The whole warp waits and stays converged: with one lane
// waiting for the others the warp came out in two parts, and each decoded by itself.
__device__ __forceinline__ void warp_wait_or_go(uint64_t* bar, uint32_t parity,
                                                volatile int* abort_flag, int32_t* status) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return;
    const uint64_t t0 = global_ns();
    for (;;) {
        if (__any_sync(0xffffffffu, *abort_flag != 0)) return;
        if (__all_sync(0xffffffffu, mbar_try_wait_sleep(bar, parity, 20000u))) return;
        if (__any_sync(0xffffffffu, global_ns() - t0 > 1000000000ull)) {
            *abort_flag = 1;
            flag_status(status, DSA_STATUS_TIMEOUT);
            return;
        }
    }
}

// The 16 heads of S^T at taddr times their factors, in place. A function of its own: seldom
// needed, and within the loop over chunks its instructions cost 0.3 % of a prefill.
__device__ __noinline__ void own_scores(uint32_t taddr, const float* scale) {
    uint32_t v[16];
    tc_ld16(v, taddr);
#pragma unroll
    for (int h = 0; h < 16; ++h) v[h] = __float_as_uint(__uint_as_float(v[h]) * scale[h]);
    tc_st16(taddr, v);
    tc_wait_st();
}
struct Unit {
    int r, hg, split, t_begin, t_end, nch;
};
__device__ __forceinline__ Unit unit_of(const MlaF4Args& a, int hgroups, int u) {
    Unit w;
    const int rh = a.ns == 1 ? u : u / a.ns;
    w.split = u - rh * a.ns;
    w.r = hgroups == 1 ? rh : rh / hgroups;
    w.hg = rh - w.r * hgroups;
    w.t_begin = w.split * a.tps;
    w.t_end = min(w.t_begin + a.tps, a.ow);
    w.nch = (w.t_end - w.t_begin + kT - 1) / kT;
    return w;
}

__global__ void __launch_bounds__(kThreads, 1) mla_f4_tc_kernel(MlaF4Args a, int hgroups, int units) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    volatile int* rows = reinterpret_cast<volatile int*>(smem + kOffRows);
    float* red = reinterpret_cast<float*>(smem + kOffRed);
    float* sums = reinterpret_cast<float*>(smem + kOffSums);
    float* kout = reinterpret_cast<float*>(smem + kOffK);
    uint32_t* qmax = reinterpret_cast<uint32_t*>(smem + kOffQmax);
    float* scale = reinterpret_cast<float*>(smem + kOffScale);
    int* owns = reinterpret_cast<int*>(smem + kOffOwn);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);
    // the same in every lane of a warp, which the shuffle shows to the compiler
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int b = 0; b < kRing; ++b) {
            mbar_init(bars + ROWS_FULL + b, 1);
            mbar_init(bars + ROWS_EMPTY + b, kWorkers);
        }
        for (int q = 0; q < 4; ++q) {
            mbar_init(bars + LAT_FULL + q, kWorkers);
            mbar_init(bars + LAT_EMPTY + q, 1);
        }
        mbar_init(bars + Q_FULL, kWorkers);
        mbar_init(bars + S_FULL, 1);
        mbar_init(bars + P_FULL, kWorkers);
        mbar_init(bars + O_DONE, 1);
        mbar_init(bars + O_FREE, kWorkers);
        mbar_init(bars + DRAIN, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    for (int i = threadIdx.x; i < kRing * kT; i += kThreads) rows[i] = -1;
    if (warp == kWorkers + 1) tc_alloc(tmem_slot, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();

    auto wait = [&](int bar, uint32_t parity) {
        warp_wait_or_go(bars + bar, parity, abort_flag, a.status);
    };
    auto arrive = [&](int bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + bar);
    };

    if (warp < kWorkers) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kRegHigh));
        const int qd = warp & 3, hb = (warp >> 2) * 16;  // lane quarter, first head
        const int j = 32 * qd + lane;                    // softmax: this thread's token
        const uint32_t lrow = (uint32_t)(32 * qd) << 16;
        // decode: token dj, 32-column piece dp of each quarter (four lanes share a token, so a
        // quarter of a warp's 16-byte loads covers two lines of 64 bytes; eight lanes on
        // eight tokens cost four times the L1 cycles, which the MMAs' operand reads lose)
        const int dj = 8 * warp + (lane >> 2), dp = lane & 3;
        const uint32_t drow = smem_u32(smem + kOffLat) + (dp >> 1) * kLatAtom + dj * 128;
        const float NEG_INF = __int_as_float(0xff800000);
        // This thread's part of a chunk's undecoded rows: per quarter k 16 bytes of codes
        // (channels 128 k + 32 dp .. + 31), and the eight scales of channels 128 dp .. + 127
        // (quarter dp; the token's four lanes exchange them at the decode).
        uint4 code[4];
        uint2 scl;
        auto request = [&](int n) {
            const int row = rows[(n & (kRing - 1)) * kT + dj];
            if (row >= 0) {
                const uint8_t* c = a.codes + (long long)row * (kKVL / 2) + dp * 16;
                const uint8_t* s = a.scales + (long long)row * (kKVL / kF4Block) + dp * 8;
#pragma unroll
                for (int k = 0; k < 4; ++k) code[k] = ldg16(c + 64 * k);
                scl = __ldg(reinterpret_cast<const uint2*>(s));
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) code[k] = make_uint4(0, 0, 0, 0);
                scl = make_uint2(0, 0);
            }
        };

        // O^T of a unit, times its heads' factors, to the output or the split's partials
        auto write_out = [&](const Unit& w, int k) {
            const int nh = min(kH, a.heads - w.hg * kH);
            float f[16];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 x = *reinterpret_cast<const float4*>(kout + hb + 4 * i);
                f[4 * i] = x.x, f[4 * i + 1] = x.y, f[4 * i + 2] = x.z, f[4 * i + 3] = x.w;
            }
            wait(O_DONE, (uint32_t)(k & 1));
            tc_fence_after();
            const long long head = a.ns > 1 ? ((long long)w.r * a.ns + w.split) * a.heads
                                            : (long long)w.r * a.heads;
            const long long o0 = (head + w.hg * kH + hb) * kKVL + j;
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
                uint32_t v[16];
                tc_ld16(v, tmem + lrow + 64 + 64 * i + hb);
                float* o32 = (a.ns > 1 ? a.part_o : a.olat) + o0 + 128 * i;
                uint16_t* o16 = a.olat16 + o0 + 128 * i;
                if (a.ns > 1 || a.olat) {
#pragma unroll
                    for (int h = 0; h < 16; ++h)
                        if (hb + h < nh) o32[h * kKVL] = __uint_as_float(v[h]) * f[h];
                }
                if (a.ns == 1 && a.olat16) {
#pragma unroll
                    for (int h = 0; h < 16; ++h)
                        if (hb + h < nh)
                            o16[h * kKVL] = __bfloat16_as_ushort(
                                __float2bfloat16_rn(__uint_as_float(v[h]) * f[h]));
                }
            }
            tc_fence_before();
            arrive(O_FREE);
        };

        int n = 0, ku = 0;
        Unit prev = {};
        for (int u = blockIdx.x; u < units; u += gridDim.x, ++ku) {
            const Unit w = unit_of(a, hgroups, u);
            const int nh = min(kH, a.heads - w.hg * kH);
            // ---- Q of the unit: f16, times a power of two; warp w has heads 4 w .. 4 w + 3.
            // One power for all heads, that of the largest, unless a head's own is more than
            // 2^kSame above it; then every head has its own, and each chunk's scores are first
            // multiplied by their heads' factors. (A factor per head throughout made a prefill
            // 6 % slower, this 1.3 %.) The last unit's score products are complete (its last
            // S^T was read), so the buffer is free; its value product may still run, and its
            // output is written after this unit's first decode.
            float sl2;  // scores to logits in log2 units
            {
                const uint16_t* qb = a.qlat + ((long long)w.r * a.heads + w.hg * kH) * kKVL;
                auto piece = [&](int k) {  // head 4 warp + k / 2, channels 8 lane + 256 (k & 1)
                    return ldg16(qb + (4 * warp + (k >> 1)) * kKVL + 8 * lane + 256 * (k & 1));
                };
                auto store = [&](int k, const uint4& x, float mul) {
                    const int h = 4 * warp + (k >> 1), c = lane + 32 * (k & 1);
                    sts16(smem_u32(smem + kOffQ) + (c >> 3) * kQAtom + h * 128 +
                              (((c & 7) ^ (h & 7)) << 4),
                          make_uint4(f4_q_half2(x.x, mul), f4_q_half2(x.y, mul),
                                     f4_q_half2(x.z, mul), f4_q_half2(x.w, mul)));
                };
                auto finite = [&](int h) {  // the largest finite |q| of head 4 warp + h
                    uint32_t x = 0;
                    for (int k = 2 * h; k < 2 * h + 2 && 4 * warp + h < nh; ++k) {
                        const uint4 y = piece(k);
                        x = __vmaxu2(x, __vmaxu2(__vmaxu2(f4_finite_abs2(y.x), f4_finite_abs2(y.y)),
                                                 __vmaxu2(f4_finite_abs2(y.z), f4_finite_abs2(y.w))));
                    }
                    return __reduce_max_sync(0xffffffffu, max(x & 0xffffu, x >> 16));
                };
                uint4 v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    v[k] = make_uint4(0, 0, 0, 0);
                    if (4 * warp + (k >> 1) < nh) v[k] = piece(k);
                }
                if (ku == 0) {  // the first chunk's rows, beside the first Q
                    wait(ROWS_FULL, 0);
                    request(0);
                }
                // the largest |q| of the warp's heads, and the smallest but for all-zero ones
                uint32_t hi = 0, lo = 0x7fffu;
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    uint32_t x = 0;
#pragma unroll
                    for (int k = 2 * h; k < 2 * h + 2; ++k)
                        x = __vmaxu2(x, __vmaxu2(__vmaxu2(v[k].x & 0x7fff7fffu, v[k].y & 0x7fff7fffu),
                                                 __vmaxu2(v[k].z & 0x7fff7fffu, v[k].w & 0x7fff7fffu)));
                    x = __reduce_max_sync(0xffffffffu, max(x & 0xffffu, x >> 16));
                    hi = max(hi, x);
                    lo = min(lo, x ? x : 0x7fffu);
                }
                if (hi >= 0x7f80u) {  // an Inf or NaN: the finite ones
                    hi = 0, lo = 0x7fffu;
#pragma unroll 1
                    for (int h = 0; h < 4; ++h) {
                        const uint32_t x = finite(h);
                        hi = max(hi, x);
                        lo = min(lo, x ? x : 0x7fffu);
                    }
                }
                if (lane == 0) qmax[warp] = hi << 16 | lo;
                bar_sync(1, kWorkers * 32);
                const uint32_t hl = qmax[lane & 15];
                const int qe = f4_q_exp(__reduce_max_sync(0xffffffffu, hl >> 16));
                const float base = a.scale * kLog2e4 * a.vscale, mul = pow2f(qe);
#pragma unroll
                for (int k = 0; k < 8; ++k) store(k, v[k], mul);
                const bool own = f4_q_exp(__reduce_min_sync(0xffffffffu, hl & 0xffffu)) - qe > kSame;
                sl2 = own ? 1.f : base * pow2f(-qe);
                if (lane == 0) owns[warp] = own;  // read by this warp alone
                if (own) {
#pragma unroll 1
                    for (int h = 0; h < 4; ++h) {
                        const int x = f4_q_exp(finite(h));
                        if (4 * warp + h < nh) {
                            store(2 * h, piece(2 * h), pow2f(x));
                            store(2 * h + 1, piece(2 * h + 1), pow2f(x));
                        }
                        if (lane == 0) scale[4 * warp + h] = base * pow2f(-x);
                    }
                    bar_sync(1, kWorkers * 32);  // `scale` is in place
                }
                fence_async_smem();
                arrive(Q_FULL);
            }
            if (u + (int)gridDim.x < units) {  // the next unit's Q into L2, a line a thread
                const Unit x = unit_of(a, hgroups, u + gridDim.x);
                const int i = threadIdx.x;  // 64 channels of head i / 8
                if (x.hg * kH + (i >> 3) < a.heads)
                    prefetch_l2(a.qlat + ((long long)x.r * a.heads + x.hg * kH) * kKVL + 64 * i);
            }

            // maximum less kUpTc, this lane's sum of weights, per head. None yet: the lowest
            // number, so that a logit that overflowed to -inf has weight 0 and not NaN.
            float e[16], l[16];
#pragma unroll
            for (int h = 0; h < 16; ++h) {
                e[h] = -FLT_MAX;
                l[h] = 0.f;
            }
            for (int c = 0; c < w.nch; ++c, ++n) {
                // ---- decode, quarter by quarter. First the token's scales: lane dp holds the
                // four 16-bit pairs of quarter dp and needs pair dp of every quarter (a 4 x 4
                // transpose in two exchanges): ev = quarters 0 and 2, od = 1 and 3.
                uint32_t ev, od;
                {
                    const bool hi = (dp & 2) != 0, odd = (dp & 1) != 0;
                    const uint32_t r = __shfl_xor_sync(0xffffffffu, hi ? scl.x : scl.y, 2);
                    const uint32_t x = hi ? r : scl.x, y = hi ? scl.y : r;
                    const uint32_t lo2 = __byte_perm(x, y, 0x5410), hi2 = __byte_perm(x, y, 0x7632);
                    const uint32_t t = __shfl_xor_sync(0xffffffffu, odd ? lo2 : hi2, 1);
                    ev = odd ? t : lo2;
                    od = odd ? hi2 : t;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t s = e4m3x2_to_f16x2(((k & 1) ? od : ev) >> (8 * (k & 2)));
                    const uint32_t s0 = __byte_perm(s, s, 0x1010), s1 = __byte_perm(s, s, 0x3232);
                    // lanes 2 and 3 of a token store their blocks in the other order: the
                    // eight lanes of a store then hit eight different 16-byte columns
                    const uint4 cw = (dp & 2) ? make_uint4(code[k].z, code[k].w, code[k].x, code[k].y)
                                              : code[k];
                    const uint32_t sa = (dp & 2) ? s1 : s0, sb = (dp & 2) ? s0 : s1;
                    const uint4 d0 = fp4_decode8(cw.x, sa), d1 = fp4_decode8(cw.y, sa),
                                d2 = fp4_decode8(cw.z, sb), d3 = fp4_decode8(cw.w, sb);
                    // decoded before the wait: the product that frees the quarter still runs
                    wait(LAT_EMPTY + k, (uint32_t)(n & 1) ^ 1u);
                    const uint32_t base = drow + 2 * k * kLatAtom;
                    const int c0 = 4 * (dp & 1) + (dp & 2), x = dj & 7;
                    sts16(base + ((c0 ^ x) << 4), d0);
                    sts16(base + (((c0 + 1) ^ x) << 4), d1);
                    sts16(base + (((c0 ^ 2) ^ x) << 4), d2);
                    sts16(base + ((((c0 ^ 2) + 1) ^ x) << 4), d3);
                    fence_async_smem();
                    arrive(LAT_FULL + k);
                }
                // ---- request the next chunk's rows (the next unit's first, at the end)
                if (c + 1 < w.nch || u + (int)gridDim.x < units) {
                    wait(ROWS_FULL + ((n + 1) & (kRing - 1)), (uint32_t)(((n + 1) / kRing) & 1));
                    request(n + 1);
                }
                // ---- the last unit's output, while this one's first score product runs
                if (c == 0 && ku > 0) {
                    bar_sync(2 + (warp >> 2), 128);  // kout is in place
                    write_out(prev, ku - 1);
                }
                // ---- softmax
                const int rb = n & (kRing - 1);
                const bool valid = rows[rb * kT + j] >= 0;
                const uint32_t prow = smem_u32(smem + kOffP) + j * 128;
                const uint32_t pc0 = prow + (((hb >> 3) ^ (j & 7)) << 4);
                const uint32_t pc1 = prow + ((((hb >> 3) + 1) ^ (j & 7)) << 4);
                uint32_t sv[16];  // scores, then weights, of heads hb .. hb + 15
                // weights 2^(score - maximum + kUpTc) of this thread's token into its row of P
                auto weights = [&]() {
                    uint32_t pk[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float p0 = ex2_sfu(__uint_as_float(sv[2 * i]));
                        const float p1 = ex2_sfu(__uint_as_float(sv[2 * i + 1]));
                        sv[2 * i] = __float_as_uint(p0);
                        sv[2 * i + 1] = __float_as_uint(p1);
                        const __half2 p = __floats2half2_rn(p0, p1);
                        pk[i] = valid ? *reinterpret_cast<const uint32_t*>(&p) : 0u;
                    }
                    sts16(pc0, make_uint4(pk[0], pk[1], pk[2], pk[3]));
                    sts16(pc1, make_uint4(pk[4], pk[5], pk[6], pk[7]));
                    fence_async_smem();
                };
                const bool own = owns[warp] != 0;
                wait(S_FULL, (uint32_t)(n & 1));
                tc_fence_after();
                if (own) {  // this warp's part of S^T times its heads' factors, in place
                    own_scores(tmem + lrow + hb, scale + hb);
                }
                tc_ld16(sv, tmem + lrow + hb);
                bool moving = c == 0;
                if (!moving) {
                    // With the maxima as they are; the vote on whether they may stay comes
                    // when the weights are stored, so that it does not delay them.
                    float top = NEG_INF;
#pragma unroll
                    for (int h = 0; h < 16; ++h) {
                        const float y = fmaf(__uint_as_float(sv[h]), sl2, -e[h]);
                        sv[h] = __float_as_uint(y);
                        top = fmaxf(top, y);
                    }
                    weights();
                    moving = bar_any(2 + (warp >> 2), 128, valid && top > kUpTc + kLazy);
                    if (moving) tc_ld16(sv, tmem + lrow + hb);
                }
                if (moving) {
                    // move the maxima that a score of this chunk exceeds by more than kLazy
                    float f[16];
#pragma unroll
                    for (int h = 0; h < 16; ++h)
                        f[h] = valid ? __fmul_rn(__uint_as_float(sv[h]), sl2) : NEG_INF;
                    const float mine =
                        scatter16(f, lane, [](float x, float y) { return fmaxf(x, y); });
                    if ((lane & 1) == 0) red[qd * kH + hb + (lane >> 1)] = mine;
                    bar_sync(2 + (warp >> 2), 128);
                    bool resc = false;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float4 r[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            r[q] = *reinterpret_cast<const float4*>(red + q * kH + hb + 4 * i);
                        const float t[4] = {
                            fmaxf(fmaxf(r[0].x, r[1].x), fmaxf(r[2].x, r[3].x)) - kUpTc,
                            fmaxf(fmaxf(r[0].y, r[1].y), fmaxf(r[2].y, r[3].y)) - kUpTc,
                            fmaxf(fmaxf(r[0].z, r[1].z), fmaxf(r[2].z, r[3].z)) - kUpTc,
                            fmaxf(fmaxf(r[0].w, r[1].w), fmaxf(r[2].w, r[3].w)) - kUpTc};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int h = 4 * i + k;
                            const bool moved = t[k] > e[h] + kLazy;
                            f[h] = moved ? ex2_sfu(e[h] - t[k]) : 1.f;
                            e[h] = moved ? t[k] : e[h];
                            l[h] *= f[h];
                            resc = resc || moved;
                        }
                    }
                    if (resc && c > 0) {  // the chunk before's O^T is complete (S_FULL)
#pragma unroll 1
                        for (int i = 0; i < 4; ++i) {
                            uint32_t v[16];
                            const uint32_t addr = tmem + lrow + 64 + 64 * i + hb;
                            tc_ld16(v, addr);
#pragma unroll
                            for (int h = 0; h < 16; ++h)
                                v[h] = __float_as_uint(__uint_as_float(v[h]) * f[h]);
                            tc_st16(addr, v);
                        }
                        tc_wait_st();
                    }
                    tc_ld16(sv, tmem + lrow + hb);
                    // The rounded logits that e was taken from, not the exact ones: above
                    // 2^24, where f32's steps are coarser than kUpTc, the largest weight
                    // would else be anything. So it is 2^0 or more; e itself may round
                    // down, hence the bound (2^16 overflows f16).
#pragma unroll
                    for (int h = 0; h < 16; ++h)
                        sv[h] = __float_as_uint(
                            min_nan(__fsub_rn(__fmul_rn(__uint_as_float(sv[h]), sl2), e[h]),
                                    kUpTc + kLazy));
                    weights();
                }
                tc_fence_before();
                arrive(P_FULL);
                if (lane == 0) mbar_arrive(bars + ROWS_EMPTY + rb);
#pragma unroll
                for (int h = 0; h < 16; ++h) l[h] += valid ? __uint_as_float(sv[h]) : 0.f;
            }

            // ---- head sums over the lanes, then over the four lane quarters; the factors
            // of the output follow from them
            float first = e[0];  // lane h: head hb + h's
#pragma unroll
            for (int h = 1; h < 16; ++h) first = lane == h ? e[h] : first;
            const float sum = scatter16(l, lane, [](float x, float y) { return x + y; });
            if ((lane & 1) == 0) sums[qd * kH + hb + (lane >> 1)] = sum;
            bar_sync(2 + (warp >> 2), 128);
            if (qd == 0 && lane < 16) {
                const int h = hb + lane;
                const float t = (sums[h] + sums[kH + h]) + (sums[2 * kH + h] + sums[3 * kH + h]);
                // a NaN sum keeps its NaN; a split's weights are relative to e itself
                kout[h] = a.ns > 1 ? a.vscale : (t == 0.f ? 0.f : a.vscale / t);
                if (a.ns > 1 && h < nh) {
                    const long long p =
                        ((long long)w.r * a.ns + w.split) * a.heads + w.hg * kH + h;
                    *reinterpret_cast<float2*>(a.part_ml + p * 2) = make_float2(first, t);
                }
            }
            prev = w;
        }
        if (ku > 0) {
            bar_sync(2 + (warp >> 2), 128);
            write_out(prev, ku - 1);
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRegLow));
        if (warp == kWorkers + 1) {
            // ---- MMA issue
            constexpr uint32_t IDESC_QK = idesc_f16(kT, kH);
            constexpr uint32_t IDESC_PV = idesc_f16(128, kH) | (1u << 15) | (1u << 16);
            // Loops, not straight-line code: this warp's few instructions then stay in the
            // instruction cache beside the workers' many. Shared memory ends below 2^18
            // bytes, so stepping a descriptor's address never carries out of its field.
            const uint64_t q0 = sw128_desc(smem_u32(smem + kOffQ));
            const uint64_t k0 = sw128_desc(smem_u32(smem + kOffLat));
            const uint64_t v0 = sw128_desc_mn(smem_u32(smem + kOffLat), kLatAtom, 1024);
            const uint64_t p0 = sw128_desc_mn(smem_u32(smem + kOffP), kQAtom, 1024);
            int n = 0, ku = 0;
            for (int u = blockIdx.x; u < units; u += gridDim.x, ++ku) {
                const Unit w = unit_of(a, hgroups, u);
                wait(Q_FULL, (uint32_t)(ku & 1));
                for (int c = 0; c < w.nch; ++c, ++n) {
#pragma unroll 1
                    for (int at = 0; at < kAtoms; ++at) {
                        if ((at & 1) == 0) {
                            wait(LAT_FULL + (at >> 1), (uint32_t)(n & 1));
                            tc_fence_after();
                        }
                        const uint64_t ka = desc_at(k0, at * kLatAtom);
                        const uint64_t qa = desc_at(q0, at * kQAtom);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            warp_mma(tmem, desc_at(ka, 32 * kk), desc_at(qa, 32 * kk), IDESC_QK,
                                     (at | kk) != 0 ? 1u : 0u);
                    }
                    warp_commit(bars + S_FULL);
                    wait(P_FULL, (uint32_t)(n & 1));
                    if (c == 0 && ku > 0) wait(O_FREE, (uint32_t)((ku - 1) & 1));
                    tc_fence_after();
#pragma unroll 1
                    for (int i = 0; i < 4; ++i) {
                        const uint64_t vi = desc_at(v0, 2 * i * kLatAtom);
#pragma unroll
                        for (int kk = 0; kk < kT / 16; ++kk)
                            warp_mma(tmem + 64 + 64 * i, desc_at(vi, kk * 2048),
                                     desc_at(p0, kk * 2048), IDESC_PV, (c > 0 || kk > 0) ? 1u : 0u);
                        warp_commit(bars + LAT_EMPTY + i);
                    }
                    if (c == w.nch - 1) warp_commit(bars + O_DONE);
                }
            }
            // every MMA issued has completed before tensor memory is released
            warp_commit(bars + DRAIN);
            if (lane == 0) mbar_wait(bars + DRAIN, 0);
        } else if (warp != kWorkers + 3) {
            // ---- cache rows: warps 16 and 18 take every other chunk
            const int mine = warp == kWorkers ? 0 : 1;
            int n = 0;
            for (int u = blockIdx.x; u < units; u += gridDim.x) {
                const Unit w = unit_of(a, hgroups, u);
                int seq = -1, L = 0;
                for (int c = 0; c < w.nch; ++c, ++n) {
                    if ((n & 1) != mine) continue;
                    const int b = n & (kRing - 1);
                    int id[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int pos = w.t_begin + c * kT + 32 * k + lane;
                        id[k] = pos < w.t_end ? __ldg(a.token_ids + (long long)w.r * a.ow + pos) : -1;
                    }
                    if (c < 2) {  // this warp's first chunk of the unit; the ids are on their way
                        seq = a.row_seq ? __ldg(a.row_seq + w.r) : w.r;
                        if (seq >= 0 && seq < a.pg.batch) {
                            L = min(__ldg(a.pg.seq_lens + seq), seq_capacity(a.pg));
                        } else {
                            if (lane == 0) flag_status(a.status, DSA_STATUS_BAD_TOKEN);
                            seq = 0;
                            L = 0;
                        }
                    }
                    int prow[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) prow[k] = (int)f4_token_row(a, seq, L, id[k]);
                    wait(ROWS_EMPTY + b, (uint32_t)((n / kRing) & 1) ^ 1u);
#pragma unroll
                    for (int k = 0; k < 4; ++k) rows[b * kT + 32 * k + lane] = prow[k];
                    arrive(ROWS_FULL + b);
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kWorkers + 1) {
        tc_fence_after();
        tc_dealloc(tmem, kTmemCols);
    }
}

}  // namespace

int mla_f4_tc_chunk() { return kT; }

int mla_f4_tc_launch(const MlaF4Args& a, cudaStream_t st) {
    const int sms = sm_count();
    if (sms <= 0) return fail(DSA_ERR_CUDA, "dsa_sparse_mla_decode_fp4: no CUDA device");
    const int hgroups = (a.heads + kH - 1) / kH;
    const long long units = (long long)a.rows * hgroups * a.ns;
    if (units > 0x7fffffffLL - sms)
        return fail(DSA_ERR_UNSUPPORTED, "dsa_sparse_mla_decode_fp4: too many rows");
    int rc = set_max_smem((const void*)mla_f4_tc_kernel, (int)kDyn);
    if (rc) return rc;
    // setmaxnreg's split adds up to 96 registers a thread: with fewer at launch its raise
    // would wait for ever
    static const int regs = [] {
        cudaFuncAttributes at;
        return cudaFuncGetAttributes(&at, mla_f4_tc_kernel) == cudaSuccess ? at.numRegs : 0;
    }();
    if (regs < 96)
        return fail(DSA_ERR_CUDA, "dsa_sparse_mla_decode_fp4: built at %d registers", regs);
    cudaError_t e = launch_pdl(mla_f4_tc_kernel, dim3((unsigned)(units < sms ? units : sms)),
                               dim3(kThreads), kDyn, st, a, hgroups, (int)units);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "dsa_sparse_mla_decode_fp4 tensor-core launch");
    return DSA_OK;
}

}  // namespace dsa
