// dsa_experts: the chosen experts' gated products and their weighted sum.
//
//   z = w13[e] . x[r]  (I gate rows, I up rows)      h = silu(gate) * up
//   y[r] = bf16(sum_j weight[r, j] * (w2[e_j] . h_j))        e_j = ids[r, j]
//
// h is rounded to bf16, or with FP8 weights to E4M3 under one 2^k per 32 channels: it is
// the second product's tensor-core operand. All sums are f32.
//
// Launches: (1) dispatch: one block per expert finds its (row, j) pairs in order and how many
// pairs lie before them (none for few pairs, see kOwnPairs). (2) For large tiles, a copy of x
// in the pairs' order. (3) Gate and up products with the activation, (4) the down products,
// both by the same persistent tensor-core kernel, (5) the weighted sums.
//
// Experts of 4,096 x 1,024, eight a row: 8 rows of 128 experts, bf16, read 1.3 GB of weights in
// 200 us (HBM bounds it); 4,096 rows of 64 take 729 us in bf16 (353 and 256 for the products: 0.82
// and 0.57 of the measured bf16 rate, waiting for L2) and 537 us in FP8 (243 and 195: the scale
// copies between the MMAs).
//
// Each product has the weights as the MMA's M operand and the pairs as N: D^T [128 weight
// rows x N pairs], N a multiple of 16 up to the tile's limit, so that few pairs cost few
// tensor-core cycles and no padding, and the weights stream as in the projection. A work
// item is 128 weight rows times up to kN pairs of one expert over all of K; items go to
// the blocks round robin, the weight rows of one expert and pair tile next to each other
// in time. A tile of the first product is 64 gate rows and the 64 up rows of the same
// channels (one three-dimensional TMA box). The rows of x are gathered by TMA (four rows a
// copy) for small tiles; else they, as those of h, are contiguous in the pairs' order and one
// copy (in four, a prefill's products took 6 to 8 % longer).
//
// Roles: warp 0 copies, warp 1 issues the MMAs, warps 4-11 take the accumulators (two, so
// that the tensor cores run on meanwhile), with FP8 warps 12-15 lay out the scales: one byte (the
// exponent) per row and 32 K values for the block-scaled MMA, which warp 1 copies to tensor
// memory in order with its MMAs. (Such a copy takes the tensor pipe about 170 cycles; stored
// by the warps instead, with tcgen05.st, the scales came so late behind the MMAs in flight
// that the first product of 4,096 rows took 294 us instead of 243.) Waits are bounded; one that gives up sets DSA_STATUS_TIMEOUT and every role leaves its loop.
#include <atomic>

#include "fp8.cuh"
#include "tc.cuh"

namespace dsa {
namespace {

constexpr int kMaxDevices = 64;
constexpr uint32_t kABytes = 128 * 128;  // 128 weight rows x 128 bytes of K
constexpr int kSfStages = 8;             // K stages whose scales travel together: a chunk
constexpr uint32_t kSfBlock = 512;       // scale words of 128 rows, [32][4]: word [l][j] is row 32 j + l
constexpr int kEpiWarps = 8;             // warps 4-11 take the accumulators, in two groups
constexpr int kSfWarp = 4 + kEpiWarps;   // FP8: warps 12-15 lay out the scales
// The epilogue's staging in shared memory: 16 pairs x 128 weight rows, f32, each 32 rows four
// floats further on: the eight threads of a pair read 16 bytes each from different banks.
constexpr int kChunk = 16;
constexpr int kStgLd = 144;  // floats per pair
constexpr uint32_t kStgBytes = 4 * kChunk * kStgLd;

// A pair of blocks shares its MMAs where a tile is that large: each holds its own 128 weight
// rows and half of the pairs' rows, and gets its weight rows' products with all pairs. Shared
// memory then carries per multiply two thirds of what it does for one block's 128 x 256 tile,
// which is what bounds that one.
constexpr bool paired(int n) { return n > 128; }

// The first product gathers rows of x itself for small tiles. A gathering copy takes about 60
// cycles for its four rows: 16 of them (64 pairs) would take longer than the weights of their
// stage do to arrive, so larger tiles read a copy of x in the pairs' order.
constexpr bool gathers(int n) { return n < 64; }

// Up to so many pairs every block of the products orders them for itself, without the dispatch
// before it (2 to 3 us of a call that reads eight experts' weights in 33).
constexpr int kOwnPairs = 256;

template <bool F8, bool UP, int N>
struct EL {  // shared and tensor memory of one block
    static constexpr int BR = paired(N) ? (N / 2 + 31) / 32 * 32 : N;  // rows of x or h of a stage
    static constexpr uint32_t STAGE = kABytes + BR * 128;
    // Staging of the epilogue's groups of warps (a small tile is one group's), twice in the second
    // product, whose K is shorter.
    static constexpr int STG_BUFS = UP ? 1 : 2;
    static constexpr int STG_GROUPS = N > kChunk ? 2 : 1;
    // FP8: two chunks of scales. A word holds four bytes along K: those of four stages where a
    // scale spans one (weights, x), those of one stage for h.
    static constexpr int SFN = (N + 127) / 128;                 // blocks of N pairs
    static constexpr int SFC = SFN * (UP ? 1 : 4);              // of four stages
    static constexpr uint32_t SF_B = kSfStages / 4 * kSfBlock;  // where the pairs' part of a chunk starts
    static constexpr uint32_t SFBUF = !F8 ? 0 : SF_B + kSfStages / 4 * SFC * kSfBlock;
    static constexpr int COLS = 2 * N + (F8 ? 4 + 4 * SFC : 0);
    static constexpr uint32_t TMEM = COLS <= 32 ? 32 : COLS <= 64 ? 64 : COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
    static_assert(COLS <= 512, "tensor memory");
    // The rest is the ring's. (512: barriers; 1024: the ring's alignment.)
    static constexpr uint32_t OWN = gathers(N) ? 8 * kOwnPairs : 0;  // int[2][kOwnPairs]
    static constexpr uint32_t TAB_MAX = 8 * (DSA_MAX_EXPERTS + DSA_MAX_TOPK + 1) + OWN;
    static constexpr uint32_t OTHER = STG_GROUPS * STG_BUFS * kStgBytes + 2 * SFBUF + TAB_MAX + 512 + 1024;
    static constexpr int S = (int)((227 * 1024 - OTHER) / STAGE);  // ring stages
    static constexpr uint32_t STG = S * STAGE;
    static constexpr uint32_t SF = STG + STG_GROUPS * STG_BUFS * kStgBytes;
    static constexpr uint32_t BARS = SF + 2 * SFBUF;
    static constexpr int NBARS = 2 * S + 9;  // full, empty; 2 + 2 scales, accumulators; drain
    static constexpr uint32_t MISC = BARS + 8 * NBARS;
    static constexpr uint32_t TAB = MISC + 16 + OWN;  // int[2][n_experts + 1]
    static_assert(8 * NBARS + 16 <= 512 && SF % 128 == 0 && BARS % 8 == 0 && STAGE % 1024 == 0, "layout");
};

struct GemmArgs {
    const int32_t* ids;      // [pairs], where the blocks order the pairs; else NULL
    int32_t* place_of;       // [pairs] ... and the first product's first block says in which order
    const int32_t* counts;   // [E] pairs of each expert
    const int32_t* starts;   // [E] pairs before them
    const int32_t* pair_of;  // [pairs] pair (row * topk + j) at a place of the order
    int n_experts, topk, pairs;
    int hidden, inter;
    int n_m;   // items per pair tile (row tiles of the weights)
    int nst;   // K stages
    // first product
    uint16_t* h;         // bf16 [pairs, inter]
    uint8_t* h8;         // E4M3 [pairs, inter]
    uint8_t* h_scales;   // [pairs, inter / 32]
    // second product
    float* part;  // [pairs in their order, hidden]
    // FP8 scales
    const float* a_scales;  // weights, [E * rows, K / 128]
    const float* x_scales;  // [rows, hidden / 128]
    int32_t* status;
};

struct Item {
    int e, m, pos, n;  // expert, weight row tile, first place in the order, pairs
};
// Item w: tab[e] pair tiles lie before expert e's.
template <int N>
__device__ __forceinline__ Item item_of(const GemmArgs& a, const int* tab, const int* start, int w) {
    Item it;
    const int tile = w / a.n_m;
    it.m = w - tile * a.n_m;
    int lo = 0, hi = a.n_experts;  // tab[lo] <= tile < tab[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tab[mid] <= tile)
            lo = mid;
        else
            hi = mid;
    }
    // The expert's pairs in equal tiles (a small rest would take a third of a full tile's time).
    constexpr int kRound = paired(N) ? 32 : 16;
    const int cnt = start[lo + 1] - start[lo], tiles = tab[lo + 1] - tab[lo];
    const int size = ((cnt + tiles - 1) / tiles + kRound - 1) / kRound * kRound;
    it.e = lo;
    it.pos = start[lo] + (tile - tab[lo]) * size;
    it.n = min(size, start[lo + 1] - it.pos);
    return it;
}

// g / (1 + exp(-g)) with the division and the exponential of the special-function unit: off by about
// 2 + |g| units of 2^-23 of the result (the exponential's argument is rounded), and 0 below g of -87,
// where the formula gives less than 2^-118. Where |g| is large the result is g itself (the exponential
// adds nothing to 1) or below |g| e^g, so 2^-17 of it at g = -50 is still far below what h is rounded to:
// 2^-9 of itself, or 2^-4 with FP8.
__device__ __forceinline__ float silu(float g) { return __fdividef(g, 1.f + __expf(-g)); }

__device__ __forceinline__ void tc_ld16(uint32_t (&v)[16], uint32_t taddr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
}
// Waits for this thread's tensor-memory loads, as tc_wait_ld.
__device__ __forceinline__ void tc_wait_ld16(uint32_t (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;\n"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
                 :
                 : "memory");
}

// Barrier `id` of 128 threads (a warpgroup's); whether every one of them comes with ok.
__device__ __forceinline__ bool group_barrier(int id, bool ok) {
    int all;
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.s32 p, %1, 0;\n"
        "barrier.cta.red.and.pred q, %2, 128, p;\nselp.s32 %0, 1, 0, q;\n}\n"
        : "=r"(all)
        : "r"((int)ok), "r"(id)
        : "memory");
    return all != 0;
}
__device__ __forceinline__ void group_sync(int id) { asm volatile("bar.sync %0, 128;\n" ::"r"(id) : "memory"); }

// One block of scales (no swizzle, 8-row groups of 16-byte rows 128 bytes apart) from shared
// memory to four columns of tensor memory, a copy in each lane quarter. In order with the
// MMAs that the same thread issues before and after it. (Here and below: by one elected lane
// of a converged warp, see warp_mma.)
__device__ __forceinline__ uint64_t sf_desc(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
}
template <bool PAIR>
__device__ __forceinline__ void warp_cp_sf(uint32_t taddr, uint32_t saddr) {
    if constexpr (PAIR)
        asm volatile(
            "{\n.reg .pred e;\nelect.sync _|e, 0xffffffff;\n"
            "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n}\n" ::"r"(taddr), "l"(sf_desc(saddr)) : "memory");
    else
        asm volatile(
            "{\n.reg .pred e;\nelect.sync _|e, 0xffffffff;\n"
            "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n}\n" ::"r"(taddr), "l"(sf_desc(saddr)) : "memory");
}

// Instruction descriptor, kind::mxf8f6f4: E4M3 x E4M3 -> f32, both K-major, UE8M0 scales,
// bytes ida and idb of each row's scale word.
__device__ __forceinline__ uint32_t idesc_mxf8(int M, int N, int ida, int idb) {
    return ((uint32_t)idb << 4) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 4) << 24) |
           ((uint32_t)ida << 29);
}
template <bool PAIR>
__device__ __forceinline__ void warp_mma_mx(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa,
                                            uint32_t sb, uint32_t accumulate) {
    if constexpr (PAIR)
        asm volatile(
            "{\n.reg .pred p, e;\nelect.sync _|e, 0xffffffff;\nsetp.ne.b32 p, %6, 0;\n"
            "@e tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::
                "r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n.reg .pred p, e;\nelect.sync _|e, 0xffffffff;\nsetp.ne.b32 p, %6, 0;\n"
            "@e tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::
                "r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
}
// A converged warp waits for a phase, for about a second at most; false after a timeout (here or
// in another role).
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int32_t* status) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    const uint64_t t0 = global_ns();
    for (uint32_t i = 1;; ++i) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        if ((i & 255u) == 0u) {
            if (__any_sync(0xffffffffu, *abort_flag != 0)) return false;
            if (__any_sync(0xffffffffu, global_ns() - t0 > 1000000000ull)) {
                *abort_flag = 1;
                if ((threadIdx.x & 31) == 0) flag_status(status, DSA_STATUS_TIMEOUT);
                return false;
            }
        }
    }
}

// UP: the first product (rows of x gathered, activation); else the second.
template <bool F8, bool UP, int N>
__global__ void __launch_bounds__(F8 ? 512 : 384, 1)
    experts_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, GemmArgs a) {
    using L = EL<F8, UP, N>;
    constexpr int S = L::S;
    constexpr bool kGather = UP && gathers(N), kPair = paired(N);
    constexpr int kRound = kPair ? 32 : 16;  // pairs of an MMA: multiples of it
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::BARS);
    uint64_t* empty = full + S;
    uint64_t* sf_full = empty + S;
    uint64_t* sf_empty = sf_full + 2;
    uint64_t* acc_full = sf_empty + 2;
    uint64_t* acc_empty = acc_full + 2;
    uint64_t* drain = acc_empty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* tab = reinterpret_cast<int*>(smem + L::TAB);
    int* start = tab + a.n_experts + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // The leader (the even block of a pair, or the only one) issues the MMAs; full, scales and
    // accumulator-empty barriers are its own, the others each block's.
    const uint32_t rank = kPair ? cluster_rank() : 0;
    const int w0 = kPair ? blockIdx.x >> 1 : blockIdx.x, wstep = kPair ? gridDim.x >> 1 : gridDim.x;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(sf_full + i, kPair ? 8 : 4);
            mbar_init(sf_empty + i, 1);
            mbar_init(acc_full + i, 1);
            mbar_init(acc_empty + i, (kPair ? 2 : 1) * kEpiWarps);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        if constexpr (kPair)
            tc_alloc2(tmem_slot, L::TMEM);
        else
            tc_alloc(tmem_slot, L::TMEM);
    }
    // The tables of the dispatch. The first product waits for it (or for the ids); the second
    // starts early (its predecessor lets it once it has itself seen them finished) and waits
    // below, before it touches h.
    if constexpr (UP) {
        pdl_wait();
        pdl_trigger();
    }
    const int32_t* pair_of = a.pair_of;
    const bool own = gathers(N) && a.ids;
    int* const own_ids = reinterpret_cast<int*>(smem + L::MISC + 16);
    int* const own_pairs = own_ids + kOwnPairs;
    if (own) {
        for (int i = threadIdx.x; i < a.n_experts; i += blockDim.x) start[i] = 0;
        __syncthreads();
        const int q = threadIdx.x;  // (there are more threads than pairs)
        if (q < a.pairs) {
            int id = __ldg(a.ids + q);
            if (id < 0 || id >= a.n_experts) {
                if (UP && blockIdx.x == 0 && id != -1) flag_status(a.status, DSA_STATUS_BAD_EXPERT);
                id = -1;
            }
            own_ids[q] = id;
            if (id >= 0) atomicAdd(start + id, 1);
        }
        __syncthreads();
        for (int i = threadIdx.x; i < a.n_experts; i += blockDim.x) tab[i] = (start[i] + N - 1) / N;
    } else {
        for (int i = threadIdx.x; i < a.n_experts; i += blockDim.x) {
            const int n = a.counts[i];
            tab[i] = (n + N - 1) / N;
            start[i] = n;
        }
    }
    __syncthreads();
    if (warp < 2) {  // exclusive scans of the tile counts and the pair counts
        int* const list = warp == 0 ? tab : start;
        int run = 0;
        for (int i0 = 0; i0 < a.n_experts; i0 += 32) {
            const int i = i0 + lane;
            const int v = i < a.n_experts ? list[i] : 0;
            int x = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (i < a.n_experts) list[i] = run + x - v;
            run += __shfl_sync(0xffffffffu, x, 31);
        }
        if (lane == 0) list[a.n_experts] = run;
    }
    if (UP && own) {
        __syncthreads();
        const int q = threadIdx.x;
        if (q < a.pairs && own_ids[q] >= 0) {
            int place = start[own_ids[q]];
            for (int j = 0; j < q; ++j) place += own_ids[j] == own_ids[q];
            own_pairs[place] = q;
            if (blockIdx.x == 0) a.place_of[q] = place;
        }
        pair_of = own_pairs;
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (kPair) cluster_barrier();  // the peer's barriers exist
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    auto arrive_leader = [&](uint64_t* bar) {
        if constexpr (kPair)
            mbar_arrive_cluster(cluster_addr(bar, 0));
        else
            mbar_arrive(bar);
    };
    const int items = tab[a.n_experts] * a.n_m;

    if (warp == 0) {
        // ---------------- copies ----------------
        int i = 0;  // stages issued
        bool ok = true;
        auto load_a = [&](const Item& it, int st, int s) {  // (one lane)
            const uint32_t dst = smem_u32(smem + s * L::STAGE);
            const int k = st * (F8 ? 128 : 64), mt = kPair ? 2 * it.m + (int)rank : it.m;
            if constexpr (kPair) {
                const uint32_t bar = cluster_addr(full + s, 0);
                if constexpr (UP)
                    tma_load_3d_pair(dst, &tmA, k, mt * 64, 2 * it.e, bar);
                else
                    tma_load_2d_pair(dst, &tmA, k, it.e * a.hidden + mt * 128, bar);
            } else {
                if constexpr (UP)
                    tma_load_3d(dst, &tmA, k, mt * 64, 2 * it.e, full + s);
                else
                    tma_load_2d(dst, &tmA, k, it.e * a.hidden + mt * 128, full + s);
            }
        };
        for (int w = w0; w < items && ok; w += wstep) {
            const Item it = item_of<N>(a, tab, start, w);
            int row[4];
            if constexpr (kGather) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int p = lane * 4 + j;
                    row[j] = pair_of[it.pos + (p < it.n ? p : 0)] / a.topk;
                }
            }
            const int half = (it.n + 31) / 32 * 16;  // of a pair of blocks: columns from each
            const int quads = (it.n + 3) >> 2;
            const int pos = it.pos + (kPair ? (int)rank * half : 0);
            const uint32_t bytes = (kABytes + (kGather ? quads * 512 : L::BR * 128)) * (kPair ? 2 : 1);
            auto load_b = [&](int st, int s) {  // (all lanes)
                const uint32_t dst = smem_u32(smem + s * L::STAGE) + kABytes;
                const int k = st * (F8 ? 128 : 64);
                if constexpr (kGather) {
                    if (lane < quads)
                        tma_gather4(dst + lane * 512, &tmB, k, row[0], row[1], row[2], row[3], full + s);
                } else if (lane == 0) {
                    if constexpr (kPair)
                        tma_load_2d_pair(dst, &tmB, k, pos, cluster_addr(full + s, 0));
                    else
                        tma_load_2d(dst, &tmB, k, pos, full + s);
                }
            };
            int st = 0;
            if constexpr (!UP) {
                if (w == w0) {
                    // the first ring's weights do not wait for h
                    const int pre = a.nst < S ? a.nst : S;
                    if (lane == 0)
                        for (int s = 0; s < pre; ++s) {
                            if (rank == 0) mbar_arrive_expect_tx(full + s, bytes);
                            load_a(it, s, s);
                        }
                    pdl_wait();
                    __syncwarp();
                    for (; st < pre; ++st, ++i) load_b(st, st);
                }
            }
            for (; st < a.nst; ++st, ++i) {
                const int s = i % S;
                int go = 1;
                if (lane == 0) {
                    go = wait_or_abort(empty + s, (uint32_t)(((i / S) & 1) ^ 1), abort_flag, a.status);
                    if (go) {
                        if (rank == 0) mbar_arrive_expect_tx(full + s, bytes);
                        load_a(it, st, s);
                    }
                }
                go = __shfl_sync(0xffffffffu, go, 0);
                if (!go) {
                    ok = false;
                    break;
                }
                load_b(st, s);
            }
        }
        if constexpr (!UP)
            if (w0 >= items) pdl_wait();
        // the copies issued have landed before the block may leave its memory
        // (a pair's: the leader sees both blocks' copies, and neither leaves before the other)
        if (lane == 0 && rank == 0)
            for (int j = i > S ? i - S : 0; j < i; ++j)
                if (!mbar_wait(full + (j % S), (uint32_t)((j / S) & 1))) break;
        __syncwarp();
    } else if (warp == 1) {
        // ---------------- MMA issue (the whole warp) ----------------
        if (rank == 0) {
            int i = 0, t = 0, chunk = 0;
            bool ok = true;
            auto commit = [&](uint64_t* bar) {
                if constexpr (kPair)
                    warp_commit2(bar);
                else
                    warp_commit(bar);
            };
            constexpr int M = kPair ? 256 : 128;
            const uint32_t sf = tmem + 2 * N;
            for (int w = w0; w < items && ok; w += wstep, ++t) {
                const Item it = item_of<N>(a, tab, start, w);
                const int n = (it.n + kRound - 1) / kRound * kRound;
                const uint32_t d = tmem + (t & 1) * N;
                ok = warp_wait(acc_empty + (t & 1), (uint32_t)(((t >> 1) & 1) ^ 1), abort_flag, a.status);
                for (int st = 0; st < a.nst && ok; ++st, ++i) {
                    const int s = i % S;
                    if (F8 && (st & (kSfStages - 1)) == 0) {
                        ok = warp_wait(sf_full + (chunk & 1), (uint32_t)((chunk >> 1) & 1), abort_flag, a.status);
                        if (!ok) break;
                    }
                    ok = warp_wait(full + s, (uint32_t)((i / S) & 1), abort_flag, a.status);
                    if (!ok) break;
                    tc_fence_after();
                    if (F8 && (st & 3) == 0) {  // the next four stages' scales
                        const int g = (st >> 2) & (kSfStages / 4 - 1);
                        const uint32_t src = smem_u32(smem + L::SF + (chunk & 1) * L::SFBUF);
                        warp_cp_sf<kPair>(sf, src + g * kSfBlock);
#pragma unroll
                        for (int b = 0; b < L::SFC; ++b)
                            warp_cp_sf<kPair>(sf + 4 + 4 * b, src + L::SF_B + (g * L::SFC + b) * kSfBlock);
                    }
                    const uint32_t sa = smem_u32(smem + s * L::STAGE), sb = sa + kABytes;
                    const uint64_t da = sw128_desc(sa), db = sw128_desc(sb);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {  // 32 bytes of K each
                        const uint32_t more = (st | kk) != 0;
                        if constexpr (F8) {
                            // the byte of the scale words: the stage's, for h the K step's
                            warp_mma_mx<kPair>(d, da + 2 * kk, db + 2 * kk, idesc_mxf8(M, n, st & 3, UP ? st & 3 : kk), sf,
                                               sf + 4 + (UP ? 0 : (st & 3) * 4 * L::SFN), more);
                        } else if constexpr (kPair) {
                            warp_mma2(d, da + 2 * kk, db + 2 * kk, idesc_bf16(M, n), more);
                        } else {
                            warp_mma(d, da + 2 * kk, db + 2 * kk, idesc_bf16(M, n), more);
                        }
                    }
                    commit(empty + s);
                    if (F8 && ((st & (kSfStages - 1)) == kSfStages - 1 || st + 1 == a.nst)) {
                        commit(sf_empty + (chunk & 1));
                        ++chunk;
                    }
                }
                if (ok) commit(acc_full + (t & 1));
            }
            commit(drain);  // every MMA issued: all of them, or those before an abort
            if (lane == 0 && !mbar_wait(drain, 0)) flag_status(a.status, DSA_STATUS_TIMEOUT);
        }
        __syncwarp();
    } else if (warp >= 4 && warp < kSfWarp) {
        // ---------------- accumulators ----------------
        // Two groups of four warps take a chunk of 16 columns (pairs) in turn: out of tensor
        // memory a chunk ahead, transposed through shared memory, a pair's channels to eight
        // threads. (The second product's straight from the registers, a lane its channel of one pair, took
        // half as long again: the stores are too many.)
        const int ew = warp & 3, eg = (warp - 4) >> 2, et = threadIdx.x & 127;
        float* stg0 = reinterpret_cast<float*>(smem + L::STG + eg * L::STG_BUFS * kStgBytes);
        const int p = et >> 3, seg = et & 7;  // pair of the chunk; 8 or 16 channels
        int t = 0, turn = 0;
        for (int w = w0; w < items; w += wstep, ++t) {
            const Item it = item_of<N>(a, tab, start, w);
            const int mt = kPair ? 2 * it.m + (int)rank : it.m;
            int got = 1;
            if (lane == 0) got = wait_or_abort(acc_full + (t & 1), (uint32_t)((t >> 1) & 1), abort_flag, a.status);
            got = __shfl_sync(0xffffffffu, got, 0);
            got = group_barrier(1 + eg, got);  // the group shares barriers below: it leaves together
            if (!got) break;
            tc_fence_after();
            const uint32_t acc = tmem + ((uint32_t)(32 * ew) << 16) + (t & 1) * N;
            uint32_t v[16], nv[16];
            if (kChunk * eg < it.n) {
                tc_ld16(v, acc + kChunk * eg);
                tc_wait_ld16(v);
            }
            for (int c0 = kChunk * eg; c0 < it.n; c0 += 2 * kChunk, ++turn) {
                const bool more = c0 + 2 * kChunk < it.n;
                if (more) tc_ld16(nv, acc + c0 + 2 * kChunk);
                float* stg = stg0 + (L::STG_BUFS == 2 ? (turn & 1) * (kStgBytes / 4) : 0);
                if (L::STG_BUFS == 1) group_sync(1 + eg);  // the staging is free
#pragma unroll
                for (int c = 0; c < kChunk; ++c) stg[c * kStgLd + 36 * ew + lane] = __uint_as_float(v[c]);
                group_sync(1 + eg);
                const bool live = c0 + p < it.n;
                if constexpr (UP) {
                    float f[8], u[8];
                    const float* from = stg + p * kStgLd + seg * 8 + 4 * (seg >> 2);
#pragma unroll
                    for (int j = 0; j < 8; j += 4) {
                        *reinterpret_cast<float4*>(f + j) = *reinterpret_cast<const float4*>(from + j);
                        *reinterpret_cast<float4*>(u + j) = *reinterpret_cast<const float4*>(from + 72 + j);  // 64 rows on
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[j] = silu(f[j]) * u[j];
                    const long long at = (long long)(it.pos + c0 + p) * a.inter + mt * 64 + seg * 8;
                    if constexpr (F8) {
                        float m = 0.f;
#pragma unroll
                        for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(f[j]));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
                        const int e = fp8_scale_exp(m);
                        const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
                        if (live) {
                            *reinterpret_cast<uint2*>(a.h8 + at) =
                                make_uint2(e4m3x2(f[0] * inv, f[1] * inv) | (e4m3x2(f[2] * inv, f[3] * inv) << 16),
                                           e4m3x2(f[4] * inv, f[5] * inv) | (e4m3x2(f[6] * inv, f[7] * inv) << 16));
                            if (!(seg & 3)) a.h_scales[at >> 5] = (uint8_t)(e + 127);
                        }
                    } else if (live) {
                        *reinterpret_cast<uint4*>(a.h + at) =
                            make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                                       pack_bf16x2(f[6], f[7]));
                    }
                } else {
                    // channels 32 j + 4 seg .. + 3: eight threads write 128 bytes of a pair at a time
                    if (live && (!kPair || mt * 128 < a.hidden)) {  // (of an odd number of row tiles one too many)
                        const float* from = stg + p * kStgLd + seg * 4;
                        float* dst = a.part + (long long)(it.pos + c0 + p) * a.hidden + mt * 128 + seg * 4;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            *reinterpret_cast<float4*>(dst + 32 * j) = *reinterpret_cast<const float4*>(from + 36 * j);
                    }
                }
                if (more) {
                    tc_wait_ld16(nv);
#pragma unroll
                    for (int c = 0; c < kChunk; ++c) v[c] = nv[c];
                }
            }
            tc_fence_before();  // this warp's columns are in registers
            if (lane == 0) arrive_leader(acc_empty + (t & 1));
        }
    } else if (F8 && warp >= kSfWarp) {
        // ---------------- scales ----------------
        // The rows' scales along K are contiguous: eight threads take a chunk's eight stages
        // of one row, a chunk ahead of its use (the next item's first behind this one's last),
        // and store the bytes where the MMA warp's copies to tensor memory read them.
        const int t = threadIdx.x - 32 * kSfWarp, sub = t >> 3, sst = t & 7;
        constexpr int NB = N / 16;
        const long long ks = a.nst;  // scales per row: one per stage
        const long long da = UP ? (long long)a.inter * ks : 16 * ks;
        const float* bsrc = UP ? a.x_scales : reinterpret_cast<const float*>(a.h_scales);
        const float* pa = nullptr;
        uint32_t pb[NB];
        auto rows_of = [&](int w) {  // row sub + 16 k of the item's tiles
            const Item it = item_of<N>(a, tab, start, w);
            int mt = kPair ? 2 * it.m + (int)rank : it.m;
            if (!UP && mt * 128 >= a.hidden) mt = 0;  // the tile too many: any scales
            pa = a.a_scales + (UP ? (long long)it.e * 2 * a.inter + mt * 64 + sub
                                  : (long long)it.e * a.hidden + mt * 128 + sub) * ks + sst;
#pragma unroll
            for (int k = 0; k < NB; ++k) {
                const int p = it.pos + (sub + 16 * k < it.n ? sub + 16 * k : 0);
                pb[k] = (uint32_t)(UP ? pair_of[p] / a.topk : p);
            }
        };
        uint32_t va[8], vb[NB];
        uint32_t odd = 0;  // what the scales seen have beyond an exponent
        auto digits = [](uint32_t v) { return (v & 0x7fffffffu) > 0x7f800000u ? 0u : v & 0x807fffffu; };
        auto load = [&](int st0) {
            const bool in = st0 + sst < a.nst;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float* src = UP ? pa + (k >> 2) * da + (k & 3) * 16 * ks : pa + k * da;
                va[k] = in ? __float_as_uint(__ldg(src + st0)) : 0u;
            }
#pragma unroll
            for (int k = 0; k < NB; ++k) vb[k] = in ? __float_as_uint(bsrc[pb[k] * ks + st0 + sst]) : 0u;
        };
        if constexpr (!UP) pdl_wait();
        int w = w0, st0 = 0;
        if (w < items) {
            rows_of(w);
            load(0);
        }
        for (int chunk = 0; w < items; ++chunk) {
            int go = 1;
            if (lane == 0)
                go = wait_or_abort(sf_empty + (chunk & 1), (uint32_t)(((chunk >> 1) & 1) ^ 1), abort_flag, a.status);
            if (!__shfl_sync(0xffffffffu, go, 0)) break;
            uint8_t* buf = smem + L::SF + (chunk & 1) * L::SFBUF;
            // row sub + 16 k: word [sub + 16 (k % 2)][k / 2 % 4] of block k / 8
            uint8_t* to = buf + (sst >> 2) * kSfBlock + sub * 16 + (sst & 3);
#pragma unroll
            for (int k = 0; k < 8; ++k) to[(k & 1) * 256 + (k >> 1) * 4] = (uint8_t)(va[k] >> 23);
#pragma unroll
            for (int k = 0; k < NB; ++k) {
                const uint32_t at = (k >> 3) * kSfBlock + (k & 1) * 256 + ((k >> 1) & 3) * 4;
                if constexpr (UP)
                    buf[L::SF_B + (sst >> 2) * L::SFN * kSfBlock + sub * 16 + (sst & 3) + at] = (uint8_t)(vb[k] >> 23);
                else
                    *reinterpret_cast<uint32_t*>(buf + L::SF_B + sst * L::SFN * kSfBlock + sub * 16 + at) = vb[k];
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) arrive_leader(sf_full + (chunk & 1));
#pragma unroll
            for (int k = 0; k < 8; ++k) odd |= digits(va[k]);
            if constexpr (UP)
#pragma unroll
                for (int k = 0; k < NB; ++k) odd |= digits(vb[k]);
            st0 += kSfStages;
            if (st0 >= a.nst) {
                st0 = 0;
                w += wstep;
                if (w < items) rows_of(w);
            }
            if (w < items) load(st0);
        }
        if (odd) flag_status(a.status, DSA_STATUS_BAD_SCALE);
    }
    __syncthreads();
    if constexpr (kPair) cluster_barrier();  // neither leaves while the other may reach it
    if (warp == 1) {
        tc_fence_after();
        if constexpr (kPair)
            tc_dealloc2(tmem, L::TMEM);
        else
            tc_dealloc(tmem, L::TMEM);
    }
}

// One block per expert: its pairs in ascending order behind those of the experts before it.
// place_of: where a pair is in that order. Each warp looks at one contiguous part of the ids twice: how many are its expert's (and,
// over the block, how many belong to lower ones), then which.
__global__ void __launch_bounds__(1024) dispatch_kernel(const int32_t* __restrict__ ids, int pairs, int n_experts,
                                                        int32_t* counts, int32_t* starts, int32_t* pair_of,
                                                        int32_t* place_of, int32_t* status) {
    __shared__ int eq_w[32], lt_w[32];
    pdl_trigger();  // the products' blocks set themselves up meanwhile
    pdl_wait();
    const int e = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int per = (int)(((long long)pairs + 32 * warps - 1) / (32 * warps)) * 32;
    const long long p0 = (long long)warp * per;
    const int lo = (int)(p0 < pairs ? p0 : pairs), hi = (int)(p0 + per < pairs ? p0 + per : pairs);
    int eq = 0, lt = 0;
    bool bad = false;
#pragma unroll 8
    for (int p = lo + lane; p < hi; p += 32) {
        const int id = __ldg(ids + p);
        eq += id == e;
        lt += id >= 0 && id < e;
        bad |= id < -1 || id >= n_experts;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        eq += __shfl_xor_sync(0xffffffffu, eq, o);
        lt += __shfl_xor_sync(0xffffffffu, lt, o);
    }
    if (lane == 0) {
        eq_w[warp] = eq;
        lt_w[warp] = lt;
    }
    if (e == 0 && bad) flag_status(status, DSA_STATUS_BAD_EXPERT);
    __syncthreads();
    int before = 0, all = 0, base = 0;
    for (int i = 0; i < warps; ++i) {
        if (i < warp) before += eq_w[i];
        all += eq_w[i];
        base += lt_w[i];
    }
    if (threadIdx.x == 0) {
        counts[e] = all;
        starts[e] = base;
    }
    int at = base + before;
    if (eq == 0) return;
#pragma unroll 4
    for (int p = lo; p < hi; p += 32) {
        const bool mine = p + lane < hi && __ldg(ids + p + lane) == e;
        const uint32_t who = __ballot_sync(0xffffffffu, mine);
        if (mine) {
            const int place = at + __popc(who & ((1u << lane) - 1u));
            pair_of[place] = p + lane;
            place_of[p + lane] = place;
        }
        at += __popc(who);
    }
}

// The rows of x in the pairs' order, `vecs` 16-byte pieces each; a warp takes a row. Bound by
// memory: 32,768 rows of 8 KB written, 62 us with its wait for the dispatch.
__global__ void __launch_bounds__(256) permute_kernel(const uint4* __restrict__ x, const int32_t* __restrict__ counts,
                                                      const int32_t* __restrict__ starts, int n_experts,
                                                      const int32_t* __restrict__ pair_of, int topk, int vecs,
                                                      uint4* __restrict__ out) {
    pdl_wait();
    const int pos = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (pos >= starts[n_experts - 1] + counts[n_experts - 1]) return;
    const uint4* src = x + (long long)(pair_of[pos] / topk) * vecs;
    uint4* dst = out + (long long)pos * vecs;
    for (int v0 = lane; v0 < vecs; v0 += 128) {
        uint4 q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (v0 + 32 * j < vecs) q[j] = __ldg(src + v0 + 32 * j);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (v0 + 32 * j < vecs) dst[v0 + 32 * j] = q[j];
    }
}

// y[r] = sum over the row's experts, in their order in ids, of weight times product; four
// channels a thread. The products stay in f32 until here, as the sum of some that cancel needs their
// digits. Bound by memory: 4,096 rows of eight products of 4,096 channels (570 MB), 82 us; 8 rows 3.1 us
// (in blocks of 256 threads 3.5; eight channels a thread and four products at a time 6.3).
constexpr int kSumThreads = 128;
__global__ void __launch_bounds__(kSumThreads) combine_kernel(const float* __restrict__ part,
                                                              const int32_t* __restrict__ ids,
                                                              const int32_t* __restrict__ place_of,
                                                              const float* __restrict__ weights, int rows,
                                                              int topk, int n_experts, int hidden,
                                                              uint16_t* __restrict__ y) {
    pdl_wait();
    const int per_row = hidden / 4;
    const long long n = (long long)rows * per_row;
    for (long long i = (long long)blockIdx.x * kSumThreads + threadIdx.x; i < n; i += (long long)gridDim.x * kSumThreads) {
        const int r = (int)(i / per_row), c = (int)(i - (long long)r * per_row) * 4;
        float s[4] = {};
        for (int j0 = 0; j0 < topk; j0 += 8) {  // eight products are requested before the first is used
            uint4 q[8];
            float w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const long long p = (long long)r * topk + j0 + j;
                const int id = j0 + j < topk ? __ldg(ids + p) : -1;
                w[j] = 0.f;
                q[j] = make_uint4(0, 0, 0, 0);
                if (id >= 0 && id < n_experts) {
                    q[j] = ldg16_stream(part + (long long)__ldg(place_of + p) * hidden + c);
                    w[j] = __ldg(weights + p);
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                s[0] = fmaf(w[j], __uint_as_float(q[j].x), s[0]);
                s[1] = fmaf(w[j], __uint_as_float(q[j].y), s[1]);
                s[2] = fmaf(w[j], __uint_as_float(q[j].z), s[2]);
                s[3] = fmaf(w[j], __uint_as_float(q[j].w), s[3]);
            }
        }
        reinterpret_cast<uint2*>(y)[i] = make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
    }
}

size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }

// Pairs per tile, by what an expert gets on average (its tiles are cut to its own count, so a
// larger one costs shared memory for weights in flight rather than work). Measured with 64
// experts of 4,096 x 1,024, bf16, some more popular than others: 12 pairs each 272 us at 16 a
// tile, 258 at 32, 254 at 64; 20: 291 at 32, 261 at 64; 40: 281 at 64, 279 at 128, 282 at 256;
// 56: 298, 288, 292; 104: 334 at 128, 319 at 256. FP8: 12: 162 at 16, 149 at 32, 150 at 64; 56: 189
// at 64, 176 at 128, 186 at 224; 104: 210 and 210; 130: 237 and 227.
int tile_of(long long pairs, int n_experts, bool f8) {
    const long long mean = (pairs + n_experts - 1) / n_experts;
    return mean <= 8 ? 16 : mean <= 14 ? 32 : mean <= 48 ? 64 : mean <= 96 ? 128 : f8 ? 224 : 256;
}

struct Plan {
    size_t counts, starts, pair_of, place_of, x, h, h_scales, part, bytes;
};
Plan plan_of(long long pairs, int n_experts, int hidden, int inter, bool f8) {
    Plan p;
    size_t at = 0;
    p.counts = at;
    at += al256((size_t)n_experts * 4);
    p.starts = at;
    at += al256((size_t)n_experts * 4);
    p.pair_of = at;
    at += al256((size_t)pairs * 4);
    p.place_of = at;
    at += al256((size_t)pairs * 4);
    p.x = at;
    at += gathers(tile_of(pairs, n_experts, f8)) ? 0 : al256((size_t)pairs * hidden * (f8 ? 1 : 2));
    p.h = at;
    at += al256((size_t)pairs * inter * (f8 ? 1 : 2));
    p.h_scales = at;
    at += f8 ? al256((size_t)pairs * (inter / 32)) : 0;
    p.part = at;
    at += al256((size_t)pairs * hidden * 4);
    p.bytes = at;
    return p;
}

int check_experts(const char* name, int rows, int topk, int n_experts, int hidden, int inter) {
    if (rows < 0 || topk < 1 || n_experts < 1 || hidden < 1 || inter < 1)
        return fail(DSA_ERR_INVALID_ARG, "%s: rows %d, topk %d, n_experts %d, hidden %d, inter %d", name, rows, topk,
                    n_experts, hidden, inter);
    if (hidden % 128 != 0 || inter % 128 != 0)
        return fail(DSA_ERR_UNSUPPORTED, "%s: hidden %d and inter %d must be multiples of 128", name, hidden, inter);
    if (hidden > 65536 || inter > 65536)
        return fail(DSA_ERR_UNSUPPORTED, "%s: hidden %d and inter %d must be at most 65536", name, hidden, inter);
    if (n_experts > DSA_MAX_EXPERTS + DSA_MAX_TOPK)
        return fail(DSA_ERR_UNSUPPORTED, "%s: at most %d experts (got %d)", name, DSA_MAX_EXPERTS + DSA_MAX_TOPK,
                    n_experts);
    if ((long long)rows * topk > (1 << 24))
        return fail(DSA_ERR_UNSUPPORTED, "%s: rows * topk %lld > %d", name, (long long)rows * topk, 1 << 24);
    return DSA_OK;
}

// Clusters of the launch that fit the device at once, asked once per kernel (its `known`) and
// device.
cudaError_t max_clusters(const void* kernel, const cudaLaunchConfig_t& cfg, std::atomic<int>* known, int* n) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool keep = dev >= 0 && dev < kMaxDevices;
    *n = keep ? known[dev].load(std::memory_order_relaxed) : 0;
    if (*n > 0) return cudaSuccess;
    e = cudaOccupancyMaxActiveClusters(n, kernel, &cfg);
    if (e != cudaSuccess) return e;
    if (*n < 1) return cudaErrorLaunchOutOfResources;
    if (keep) known[dev].store(*n, std::memory_order_relaxed);
    return cudaSuccess;
}

template <bool F8, bool UP, int N>
int gemm_launch(const GemmArgs& a, const void* weights, const void* b, int b_rows, int sms, cudaStream_t st) {
    using L = EL<F8, UP, N>;
    static_assert(L::TAB + L::TAB_MAX + 1024 <= 227 * 1024, "shared memory");
    const int dyn = (int)(L::TAB + 8 * (a.n_experts + 1) + 1024);
    int rc = set_max_smem((const void*)experts_kernel<F8, UP, N>, 227 * 1024);
    if (rc) return rc;
    const CUtensorMapDataType dt = F8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const uint64_t es = F8 ? 1 : 2, H = a.hidden, I = a.inter, E = a.n_experts;
    const uint32_t bk = F8 ? 128 : 64;
    CUtensorMap tmA, tmB;
    if (UP) {
        const uint64_t dims[3] = {H, I, 2 * E};
        const uint64_t strides[2] = {H * es, I * H * es};
        const uint32_t box[3] = {bk, 64, 2};
        rc = make_tmap(&tmA, dt, weights, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
        if (rc) return rc;
        rc = make_tmap_2d(&tmB, dt, b, H, (uint64_t)b_rows, H * es, bk, gathers(N) ? 1 : L::BR,
                          CU_TENSOR_MAP_SWIZZLE_128B);
    } else {
        rc = make_tmap_2d(&tmA, dt, weights, I, E * H, I * es, bk, 128, CU_TENSOR_MAP_SWIZZLE_128B);
        if (rc) return rc;
        rc = make_tmap_2d(&tmB, dt, b, I, (uint64_t)b_rows, I * es, bk, L::BR, CU_TENSOR_MAP_SWIZZLE_128B);
    }
    if (rc) return rc;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)sms);
    cfg.blockDim = dim3(F8 ? 512 : 384);
    cfg.dynamicSmemBytes = (size_t)dyn;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = paired(N) ? 2 : 1;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (paired(N)) {
        cfg.gridDim.x &= ~1u;
        // One pair of blocks per pair of SMs; fewer where not all SMs come in pairs (a pair that
        // waited for others to leave would take its share of the items after theirs).
        int clusters = 0;
        static std::atomic<int> known[kMaxDevices];
        cudaError_t q = max_clusters((const void*)experts_kernel<F8, UP, N>, cfg, known, &clusters);
        if (q != cudaSuccess) return cuda_fail(q, "dsa_experts occupancy");
        if (2 * clusters < sms) cfg.gridDim.x = (unsigned)(2 * clusters);
    }
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, experts_kernel<F8, UP, N>, tmA, tmB, a);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "dsa_experts launch");
    return DSA_OK;
}

template <bool F8, bool UP>
int gemm_dispatch(const GemmArgs& a, const void* weights, const void* b, int b_rows, int sms, cudaStream_t st) {
    switch (tile_of(a.pairs, a.n_experts, F8)) {
        case 16: return gemm_launch<F8, UP, 16>(a, weights, b, b_rows, sms, st);
        case 32: return gemm_launch<F8, UP, 32>(a, weights, b, b_rows, sms, st);
        case 64: return gemm_launch<F8, UP, 64>(a, weights, b, b_rows, sms, st);
        case 128: return gemm_launch<F8, UP, 128>(a, weights, b, b_rows, sms, st);
        default: return gemm_launch<F8, UP, F8 ? 224 : 256>(a, weights, b, b_rows, sms, st);
    }
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" int dsa_experts_workspace(int rows, int topk, int n_experts, int hidden, int inter, int fp8,
                                     size_t* bytes) {
    if (!bytes) return fail(DSA_ERR_INVALID_ARG, "dsa_experts_workspace: bytes is NULL");
    int rc = check_experts("dsa_experts_workspace", rows, topk, n_experts, hidden, inter);
    if (rc) return rc;
    *bytes = plan_of((long long)rows * topk, n_experts, hidden, inter, fp8 != 0).bytes;
    return DSA_OK;
}

extern "C" int dsa_experts(const void* x, const float* x_scales, int rows, int hidden, const int32_t* ids,
                           const float* weights, int topk, const void* w13, const float* w13_scales, const void* w2,
                           const float* w2_scales, int n_experts, int inter, dsa_bf16* y, int32_t* status,
                           void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_experts("dsa_experts", rows, topk, n_experts, hidden, inter);
    if (rc) return rc;
    const bool f8 = x_scales || w13_scales || w2_scales;
    if (rows == 0) return DSA_OK;
    if (!x || !ids || !weights || !w13 || !w2 || !y) return fail(DSA_ERR_INVALID_ARG, "dsa_experts: NULL tensor");
    if (f8 && (!x_scales || !w13_scales || !w2_scales))
        return fail(DSA_ERR_INVALID_ARG, "dsa_experts: FP8 takes the scales of x, w13 and w2, bf16 none");
    if ((((uintptr_t)x) | ((uintptr_t)w13) | ((uintptr_t)w2) | ((uintptr_t)y) | ((uintptr_t)workspace)) & 15)
        return fail(DSA_ERR_INVALID_ARG, "dsa_experts: tensors must be 16-byte aligned");
    if ((((uintptr_t)x_scales) | ((uintptr_t)w13_scales) | ((uintptr_t)w2_scales) | ((uintptr_t)ids) |
         ((uintptr_t)weights)) & 3)
        return fail(DSA_ERR_INVALID_ARG, "dsa_experts: misaligned tensor");
    const int pairs = rows * topk;
    const Plan p = plan_of(pairs, n_experts, hidden, inter, f8);
    if (!workspace || workspace_bytes < p.bytes)
        return fail(DSA_ERR_INVALID_ARG, "dsa_experts: workspace %zu B < %zu B needed", workspace_bytes, p.bytes);
    const int sms = sm_count();
    if (sms <= 0) return fail(DSA_ERR_CUDA, "dsa_experts: no CUDA device");
    cudaStream_t st = (cudaStream_t)stream;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    int32_t* counts = reinterpret_cast<int32_t*>(ws + p.counts);
    int32_t* starts = reinterpret_cast<int32_t*>(ws + p.starts);
    int32_t* pair_of = reinterpret_cast<int32_t*>(ws + p.pair_of);
    int32_t* place_of = reinterpret_cast<int32_t*>(ws + p.place_of);
    const int threads = pairs >= 1024 ? 1024 : (pairs + 31) / 32 * 32;
    const bool own = pairs <= kOwnPairs && gathers(tile_of(pairs, n_experts, f8));
    cudaError_t e = cudaSuccess;
    if (!own) {
        e = launch_pdl(dispatch_kernel, dim3((unsigned)n_experts), dim3((unsigned)threads), 0, st, ids, pairs, n_experts,
                       counts, starts, pair_of, place_of, status);
        if (e == cudaSuccess) e = cudaGetLastError();
        if (e != cudaSuccess) return cuda_fail(e, "dsa_experts dispatch launch");
    }
    GemmArgs a = {};
    a.ids = own ? ids : nullptr;
    a.place_of = place_of;
    a.counts = counts;
    a.starts = starts;
    a.pair_of = pair_of;
    a.n_experts = n_experts;
    a.topk = topk;
    a.pairs = pairs;
    a.hidden = hidden;
    a.inter = inter;
    a.h = reinterpret_cast<uint16_t*>(ws + p.h);
    a.h8 = ws + p.h;
    a.h_scales = ws + p.h_scales;
    a.part = reinterpret_cast<float*>(ws + p.part);
    a.x_scales = x_scales;
    a.status = status;
    const bool two = paired(tile_of(pairs, n_experts, f8));
    a.n_m = inter / (two ? 128 : 64);
    a.nst = hidden / (f8 ? 128 : 64);
    a.a_scales = w13_scales;
    int x_rows = rows;
    if (!gathers(tile_of(pairs, n_experts, f8))) {
        e = launch_pdl(permute_kernel, dim3((unsigned)((pairs + 7) / 8)), dim3(256), 0, st, (const uint4*)x,
                       (const int32_t*)counts, (const int32_t*)starts, n_experts, (const int32_t*)pair_of, topk,
                       hidden / (f8 ? 16 : 8), (uint4*)(ws + p.x));
        if (e == cudaSuccess) e = cudaGetLastError();
        if (e != cudaSuccess) return cuda_fail(e, "dsa_experts permute launch");
        x = ws + p.x;
        x_rows = pairs;
    }
    rc = f8 ? gemm_dispatch<true, true>(a, w13, x, x_rows, sms, st)
            : gemm_dispatch<false, true>(a, w13, x, x_rows, sms, st);
    if (rc) return rc;
    a.n_m = two ? (hidden + 255) / 256 : hidden / 128;
    a.nst = inter / (f8 ? 128 : 64);
    a.a_scales = w2_scales;
    rc = f8 ? gemm_dispatch<true, false>(a, w2, a.h8, pairs, sms, st)
            : gemm_dispatch<false, false>(a, w2, a.h, pairs, sms, st);
    if (rc) return rc;
    const long long n = (long long)rows * (hidden / 4);
    long long blocks = (n + kSumThreads - 1) / kSumThreads;
    if (blocks > (long long)sms * 32) blocks = (long long)sms * 32;
    e = launch_pdl(combine_kernel, dim3((unsigned)blocks), dim3(kSumThreads), 0, st, (const float*)a.part, ids, (const int32_t*)place_of, weights, rows, topk, n_experts, hidden, y);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "dsa_experts combine launch");
    return DSA_OK;
}
