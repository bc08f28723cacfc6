// Pages of the paged caches: forking, freeing, growing (with copy-on-write) and compacting.
//
// A page is one block of dsa_paging's block table: block_size token rows in every token
// cache and block_size / kpool rows in every pooled-key cache, all found through one
// table. refs[p] counts the table entries that name page p; a page with refs[p] == 0 is
// free. All decisions are taken on the device from the tables and counts, so the calls
// can be captured in a graph and replayed as the sequences change.
//
// Determinism: pages are handed out lowest id first, to sequences in the order listed,
// and an integer count does not depend on the order of its additions.
//
// pages_free_kernel, pages_fork_kernel -- one block per (sequence, chunk of its table
// row). Latency bound: a row's entries are read and written once, with one atomic on
// each page's count. pages_serve_kernel -- one block per listed sequence.
//
// pages_reserve_kernel, pages_compact_kernel -- the planning steps. One cluster of eight
// CTAs scans the counts (4 bytes a page): each CTA sums its slice, the sums are
// exchanged through distributed shared memory, and a second pass over the slice (now in
// L2) gives every free (or live) page its rank. One launch, no grid-wide wait.
//
// pages_apply kernels -- the data. A page is cut into pieces of 4 KB per cache; a warp
// moves one piece at a time with eight 16-byte loads in flight per lane, so a few copied
// pages spread over the whole GPU and many stream at the memory's rate.
#include <cooperative_groups.h>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace dsa {
namespace {

constexpr int kPlanCtas = 8;
constexpr int kPlanThreads = 1024;
constexpr int kRowThreads = 256;
constexpr int kRowChunk = 1024;  // table entries per block of the free and fork kernels
constexpr int kCopyThreads = 256;
constexpr int kPiece = 4096;     // bytes a warp moves at a time

// ---------------------------------------------------------------------------
// Shared pieces.

// Drops one reference of page p (an entry of some table row).
__device__ __forceinline__ void page_release(int32_t* refs, long long num_pages, int p,
                                             int32_t* status) {
    if (p == -1) return;
    if (p < 0 || p >= num_pages) {
        flag_status(status, DSA_STATUS_BAD_BLOCK);
        return;
    }
    if (atomicSub(refs + p, 1) <= 0) {  // not held by anybody: the count stays
        atomicAdd(refs + p, 1);
        flag_status(status, DSA_STATUS_BAD_BLOCK);
    }
}

// Whether list[0, i) holds a, or list[0, n) holds b (block-wide).
__device__ __forceinline__ bool block_finds(const int32_t* list, int i, int a, int n, int b) {
    bool hit = false;
    for (int j = threadIdx.x; j < max(i, n); j += blockDim.x) {
        const int v = __ldg(list + j);
        hit = hit || (j < i && v == a) || (j < n && v == b);
    }
    return __syncthreads_or(hit) != 0;
}

// Two sums at once: the high and the low 32 bits (each sum below 2^31).
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair_of(int hi, int lo) {
    return ((Pair)(uint32_t)hi << 32) | (uint32_t)lo;
}
__device__ __forceinline__ int pair_hi(Pair p) { return (int)(p >> 32); }
__device__ __forceinline__ int pair_lo(Pair p) { return (int)(uint32_t)p; }

// Exclusive scan of one pair per thread over the block; *total gets the sum.
__device__ __forceinline__ Pair block_scan(Pair v, Pair* warp_sums, Pair* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Pair x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Pair y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();  // warp_sums is reused by consecutive calls
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    Pair w = warp_sums[lane];
    static_assert(kPlanThreads == 1024, "a lane per warp sum");
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Pair y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    const Pair before = warp == 0 ? 0 : __shfl_sync(0xffffffffu, w, warp - 1);
    return before + x - v;
}

// Every CTA's value to all CTAs of the cluster: returns the sum over lower ranks, *all is
// the sum over the cluster. slot: a [kPlanCtas] array used by this exchange alone.
__device__ __forceinline__ Pair cluster_scan(cg::cluster_group& cl, Pair v, Pair* slot,
                                             Pair* all) {
    if (threadIdx.x < kPlanCtas) cl.map_shared_rank(slot, threadIdx.x)[cl.block_rank()] = v;
    cl.sync();
    Pair before = 0, sum = 0;
#pragma unroll
    for (int k = 0; k < kPlanCtas; ++k) {
        if (k < (int)cl.block_rank()) before += slot[k];
        sum += slot[k];
    }
    *all = sum;
    return before;
}

// Four consecutive counts from page p0 on (p0 a multiple of 4); pages past hi read as `out`.
__device__ __forceinline__ int4 load_counts(const int32_t* refs, long long p0, long long hi, int out) {
    if (p0 + 4 <= hi && (reinterpret_cast<uintptr_t>(refs) & 15) == 0)
        return *reinterpret_cast<const int4*>(refs + p0);
    int4 r;
    r.x = p0 < hi ? refs[p0] : out;
    r.y = p0 + 1 < hi ? refs[p0 + 1] : out;
    r.z = p0 + 2 < hi ? refs[p0 + 2] : out;
    r.w = p0 + 3 < hi ? refs[p0 + 3] : out;
    return r;
}

// ---------------------------------------------------------------------------
// Page data: pairs of pages copied in every cache.

struct PageArrays {
    int n;
    int pieces;  // pieces of one page over all arrays
    uint8_t* base[DSA_MAX_PAGE_ARRAYS];
    long long bytes[DSA_MAX_PAGE_ARRAYS];  // bytes of a page, negative: not 16-byte aligned
    int first[DSA_MAX_PAGE_ARRAYS];        // index of the array's first piece
};

// A warp's walk over pieces: pair (which copied page), piece within the page, and the array
// that holds it. Consecutive pieces cost additions only; the start a division and a search.
struct PieceWalk {
    int pair, piece, array;
    __device__ __forceinline__ PieceWalk(const PageArrays& A, long long u) {
        const int per = max(A.pieces, 1);
        pair = (int)(u / per);
        piece = (int)(u - (long long)pair * per);
        int lo = 0, hi = A.n - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (A.first[mid] <= piece)
                lo = mid;
            else
                hi = mid - 1;
        }
        array = lo;
    }
    __device__ __forceinline__ void next(const PageArrays& A) {
        if (++piece >= max(A.pieces, 1)) {
            piece = 0;
            array = 0;
            ++pair;
        } else if (array + 1 < A.n && A.first[array + 1] == piece) {
            ++array;
        }
    }
};
// The walk's piece of page src to page dst, by a warp.
__device__ __forceinline__ void copy_piece(const PageArrays& A, const PieceWalk& w, long long src,
                                           long long dst) {
    const int lane = threadIdx.x & 31;
    const long long bytes = A.bytes[w.array];
    const long long stride = bytes < 0 ? -bytes : bytes;
    const long long off = (long long)(w.piece - A.first[w.array]) * kPiece;
    const int n = (int)min((long long)kPiece, stride - off);
    const uint8_t* s = A.base[w.array] + src * stride + off;
    uint8_t* d = A.base[w.array] + dst * stride + off;
    if (bytes >= 0) {
        const uint4* s4 = reinterpret_cast<const uint4*>(s);
        uint4* d4 = reinterpret_cast<uint4*>(d);
        const int m = n / 16;
        uint4 v[kPiece / 512];
#pragma unroll
        for (int k = 0; k < kPiece / 512; ++k)
            if (lane + 32 * k < m) v[k] = __ldcs(s4 + lane + 32 * k);
#pragma unroll
        for (int k = 0; k < kPiece / 512; ++k)
            if (lane + 32 * k < m) __stcs(d4 + lane + 32 * k, v[k]);
    } else {
        for (int i = lane; i < n; i += 32) d[i] = s[i];
    }
}
// This warp's share [*u0, *u1) of `total` pieces: equal runs of consecutive ones.
__device__ __forceinline__ void warp_share(long long total, long long* u0, long long* u1) {
    const long long warps = (long long)gridDim.x * (kCopyThreads / 32);
    const long long w = (long long)blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5);
    const long long each = (total + warps - 1) / warps;
    *u0 = min(total, w * each);
    *u1 = min(total, *u0 + each);
}

// ---------------------------------------------------------------------------
struct SeqArgs {
    const int32_t* list;     // sequences (free) or children (fork)
    const int32_t* parents;  // fork
    int n;
    int32_t* table;
    int32_t* seq_lens;
    int32_t* refs;
    int32_t* status;
    Paging pg;
};

__global__ void __launch_bounds__(kRowThreads) pages_free_kernel(SeqArgs a) {
    pdl_trigger();  // short kernels that often follow one another: the next may be resident
    pdl_wait();
    const int i = blockIdx.x;
    const int b = __ldg(a.list + i);
    if (b == -1) return;  // padding
    if (b < 0 || b >= a.pg.batch) {
        if (threadIdx.x == 0) flag_status(a.status, DSA_STATUS_BAD_SEQ);
        return;
    }
    if (block_finds(a.list, i, b, 0, 0)) return;  // listed before: freed by that entry
    int32_t* row = a.table + (long long)b * a.pg.max_blocks;
    const int e1 = min(a.pg.max_blocks, ((int)blockIdx.y + 1) * kRowChunk);
    for (int e = blockIdx.y * kRowChunk + threadIdx.x; e < e1; e += kRowThreads) {
        const int p = row[e];
        if (p == -1) continue;
        page_release(a.refs, a.pg.num_blocks, p, a.status);
        row[e] = -1;
    }
    if (blockIdx.y == 0 && threadIdx.x == 0) a.seq_lens[b] = 0;
}

__global__ void __launch_bounds__(kRowThreads) pages_fork_kernel(SeqArgs a) {
    pdl_trigger();
    pdl_wait();
    const int i = blockIdx.x;
    const int c = __ldg(a.list + i), p = __ldg(a.parents + i);
    if (c == -1) return;  // padding
    bool bad = c < 0 || c >= a.pg.batch || p < 0 || p >= a.pg.batch;
    // a child twice (the first pair counts), or a parent that the call overwrites
    bad = block_finds(a.list, i, c, a.n, p) || bad;
    if (bad) {
        if (threadIdx.x == 0) flag_status(a.status, DSA_STATUS_BAD_SEQ);
        return;
    }
    int32_t* child = a.table + (long long)c * a.pg.max_blocks;
    const int32_t* parent = a.table + (long long)p * a.pg.max_blocks;
    const int L = max(a.seq_lens[p], 0);
    const int held = (int)min((long long)a.pg.max_blocks,
                              ((long long)L + a.pg.block_size - 1) / a.pg.block_size);
    const int e1 = min(a.pg.max_blocks, ((int)blockIdx.y + 1) * kRowChunk);
    for (int e = blockIdx.y * kRowChunk + threadIdx.x; e < e1; e += kRowThreads) {
        const int old = child[e];
        int now = -1;
        if (e < held) {
            now = parent[e];
            if (now < 0 || now >= a.pg.num_blocks) {
                flag_status(a.status, DSA_STATUS_BAD_BLOCK);
                now = -1;
            } else {
                atomicAdd(a.refs + now, 1);
            }
        }
        page_release(a.refs, a.pg.num_blocks, old, a.status);
        if (old != now) child[e] = now;
    }
    if (blockIdx.y == 0 && threadIdx.x == 0) a.seq_lens[c] = L;
}

// dsa_pages_serve: one block per entry, for the search that fork's rule takes.
__global__ void __launch_bounds__(kRowThreads)
    pages_serve_kernel(const int32_t* parents, const int32_t* list, int n, int batch, int on,
                       int32_t* serving, int32_t* status) {
    pdl_trigger();
    pdl_wait();
    const int i = blockIdx.x;
    const int b = __ldg(list + i);
    if (b == -1) return;  // padding
    bool bad = b < 0 || b >= batch;
    if (parents) {  // the pairs that pages_fork_kernel skips
        const int p = __ldg(parents + i);
        bad = bad || p < 0 || p >= batch;
        bad = block_finds(list, i, b, n, p) || bad;
    }
    if (threadIdx.x != 0) return;
    if (bad)
        flag_status(status, DSA_STATUS_BAD_SEQ);
    else
        serving[b] = on ? b : -1;
}

// ---------------------------------------------------------------------------
// dsa_pages_reserve

struct ReserveArgs {
    const int32_t* list;  // nullable: all sequences
    int n;
    int new_tokens;
    int first_key;
    int kpool;  // 0: no pooled-key caches
    int32_t* table;
    int32_t* refs;
    int32_t* status;
    Paging pg;
    // workspace
    int32_t* count;  // ranks handed out
    int32_t* need;   // [n] pages of a listed sequence, then its first rank
    int32_t* owner;  // [batch] first entry of the list that names the sequence
    int32_t* free_list;  // [num_pages] free pages, ascending
    int32_t* src;        // [num_pages] page that rank's page is a copy of, or -1
};

// The pages that the next new_tokens of sequence b write: the token pages from t0 to t1
// and, where a pool becomes whole, the pooled-key pages from p0 to p1 (inclusive). With
// first_key > 0 a pool's page lies before its tokens' page.
struct Window {
    int t0, t1, p0, p1;
    bool partial;  // page t0 already holds tokens
};
__device__ __forceinline__ int pools_of(long long n, int first_key, int kpool) {
    return n > first_key ? (int)((n - first_key) / kpool) : 0;
}
__device__ __forceinline__ bool window_of(const ReserveArgs& a, int b, Window* w) {
    const int bs = a.pg.block_size;
    const int L = a.pg.seq_lens[b];
    if (L < 0 || (long long)L + a.new_tokens > (long long)a.pg.max_blocks * bs) {
        flag_status(a.status, DSA_STATUS_CACHE_FULL);
        return false;
    }
    const long long end = (long long)L + a.new_tokens;
    w->t0 = L / bs;
    w->t1 = (int)((end - 1) / bs);
    w->partial = L % bs != 0;
    w->p0 = 1;
    w->p1 = 0;
    if (a.kpool > 0) {
        const int q0 = pools_of(L, a.first_key, a.kpool), q1 = pools_of(end, a.first_key, a.kpool);
        if (q1 > q0) {
            const int ppb = bs / a.kpool;
            w->p0 = q0 / ppb;
            w->p1 = (q1 - 1) / ppb;
        }
    }
    return true;
}
// What entry j of the row needs: 0 nothing, 1 a fresh page, 2 a copy of *page.
__device__ __forceinline__ int entry_need(const ReserveArgs& a, const Window& w,
                                          const int32_t* row, int j, int* page) {
    const bool tok = j >= w.t0 && j <= w.t1;
    if (!tok && !(j >= w.p0 && j <= w.p1)) return 0;
    const int p = row[j];
    *page = p;
    if (p >= 0 && p < a.pg.num_blocks) return a.refs[p] > 1 ? 2 : 0;
    if (p == -1 && tok && !(j == w.t0 && w.partial)) return 1;
    flag_status(a.status, DSA_STATUS_BAD_BLOCK);
    return 0;
}

// G lanes per sequence (1 or 32): 32 where a call's window spans many pages. With one lane
// and at most one sequence per thread (kOne), what the first look at a sequence found
// stays in registers. The free pages are counted from loads issued before the sequences
// are looked at, and both sums travel together, so that a decode step's reservation waits
// for one chain of loads (length, table entry, count), one exchange and one barrier.
template <int G, bool kOne>
__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads, 1)
    pages_reserve_kernel(ReserveArgs a) {
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();  // every CTA has started: their shared memory may be written
    pdl_trigger();
    pdl_wait();
    __shared__ Pair warp_sums[kPlanThreads / 32];
    __shared__ Pair slots[kPlanCtas];
    const int rank = cl.block_rank();
    const int t = threadIdx.x;

    // this CTA's slice of the counts; its first tile stays in registers
    const long long num = a.pg.num_blocks;
    const long long slice = ((num + kPlanCtas - 1) / kPlanCtas + 3) & ~3LL;
    const long long s0 = min(num, rank * slice), s1 = min(num, s0 + slice);
    int4 c0 = make_int4(1, 1, 1, 1);
    if (s0 + 4LL * t < s1) c0 = load_counts(a.refs, s0 + 4LL * t, s1, 1);

    if (a.list) {  // the first entry that names a sequence serves it
        for (int b = rank * kPlanThreads + t; b < a.pg.batch; b += kPlanCtas * kPlanThreads)
            a.owner[b] = 0x7fffffff;
        cl.sync();
        for (int i = rank * kPlanThreads + t; i < a.n; i += kPlanCtas * kPlanThreads) {
            const int b = a.list[i];
            if (b >= 0 && b < a.pg.batch)
                atomicMin(a.owner + b, i);
            else if (b != -1)
                flag_status(a.status, DSA_STATUS_BAD_SEQ);
        }
        cl.sync();
    }
    // the sequence of list entry i, or -1
    auto seq_of = [&](int i) {
        if (!a.list) return i;
        const int b = a.list[i];
        return b >= 0 && b < a.pg.batch && __ldcg(a.owner + b) == i ? b : -1;
    };
    const int per = (a.n + kPlanCtas - 1) / kPlanCtas;
    const int i0 = min(a.n, rank * per), i1 = min(a.n, i0 + per);
    const int sub = t % G;  // lane within the sequence's group

    // ---- pages that each sequence of this CTA's slice needs
    int mine_need = 0, seq = -1, lo0 = 0, page0 = -1;
    uint32_t need_mask = 0;  // kOne: entries lo0 + bit; page0: the first one's page
    int run = 0;             // !kOne: the slice's sum
    if constexpr (kOne) {
        Window w;
        if (i0 + t < i1 && (seq = seq_of(i0 + t)) >= 0 && window_of(a, seq, &w)) {
            const int32_t* row = a.table + (long long)seq * a.pg.max_blocks;
            lo0 = w.p0 <= w.p1 ? min(w.p0, w.t0) : w.t0;
            for (int j = lo0; j <= w.t1; ++j) {
                int page;
                if (entry_need(a, w, row, j, &page) != 0) {
                    if (need_mask == 0) page0 = page;
                    need_mask |= 1u << (j - lo0);
                }
            }
            mine_need = __popc(need_mask);
        }
    } else {
        for (int i = i0 + t / G; i < i1; i += kPlanThreads / G) {
            const int b = seq_of(i);
            int need = 0;
            Window w;
            if (b >= 0 && window_of(a, b, &w)) {
                const int32_t* row = a.table + (long long)b * a.pg.max_blocks;
                const int lo = w.p0 <= w.p1 ? min(w.p0, w.t0) : w.t0;
                for (int j = lo + sub; j <= w.t1; j += G) {
                    int page;
                    need += entry_need(a, w, row, j, &page) != 0 ? 1 : 0;
                }
            }
            if (G > 1) need = __reduce_add_sync(0xffffffffu, need);
            if (sub == 0) a.need[i] = need;
        }
        __syncthreads();
        for (int i = i0; i < i1; i += kPlanThreads) {  // first ranks within the slice
            const bool in = i + t < i1;
            Pair total;
            const Pair before = block_scan(pair_of(in ? a.need[i + t] : 0, 0), warp_sums, &total);
            if (in) a.need[i + t] = run + pair_hi(before);
            run += pair_hi(total);
        }
        mine_need = t == 0 ? run : 0;
    }

    // ---- needs and free pages summed over the block and the cluster
    const int free0 = (c0.x == 0) + (c0.y == 0) + (c0.z == 0) + (c0.w == 0);
    int mine_free = free0;
    for (long long p = s0 + 4LL * (kPlanThreads + t); p < s1; p += 4LL * kPlanThreads) {
        const int4 c = load_counts(a.refs, p, s1, 1);
        mine_free += (c.x == 0) + (c.y == 0) + (c.z == 0) + (c.w == 0);
    }
    Pair here, all;
    const Pair mine = block_scan(pair_of(mine_need, mine_free), warp_sums, &here);
    const Pair before = cluster_scan(cl, here, slots, &all);
    const int want = pair_hi(all), free_all = pair_lo(all), base = pair_hi(before);
    if (rank == 0 && t == 0) *a.count = (int)min((long long)want, num);
    if (want == 0) return;  // every CTA of the cluster agrees

    // ---- free pages in ascending order, up to `want`
    int at = pair_lo(before);
    auto list_free = [&](const int4& c, long long q, int r) {
        if (c.x == 0 && r < want) a.free_list[r] = (int)q;
        r += c.x == 0;
        if (c.y == 0 && r < want) a.free_list[r] = (int)q + 1;
        r += c.y == 0;
        if (c.z == 0 && r < want) a.free_list[r] = (int)q + 2;
        r += c.z == 0;
        if (c.w == 0 && r < want) a.free_list[r] = (int)q + 3;
    };
    if (slice <= 4LL * kPlanThreads) {
        list_free(c0, s0 + 4LL * t, at + pair_lo(mine));
    } else {
        for (long long p = s0; p < s1 && at < want; p += 4LL * kPlanThreads) {
            const long long q = p + 4LL * t;
            int4 c = make_int4(1, 1, 1, 1);
            if (q < s1) c = load_counts(a.refs, q, s1, 1);
            Pair total;
            const Pair r = block_scan(
                pair_of(0, (c.x == 0) + (c.y == 0) + (c.z == 0) + (c.w == 0)), warp_sums, &total);
            list_free(c, q, at + pair_lo(r));
            at += pair_lo(total);
        }
    }
    cl.sync();  // the list is complete and visible to the cluster

    // ---- hand the pages out: all of a sequence's, or none. Counts of shared pages are
    // lowered by the apply step, so that every decision here sees the counts the needs were
    // taken from.
    if constexpr (kOne) {
        if (mine_need == 0) return;
        int32_t* row = a.table + (long long)seq * a.pg.max_blocks;
        int r = base + pair_hi(mine);
        const bool granted = r + mine_need <= free_all;
        if (!granted) flag_status(a.status, DSA_STATUS_NO_PAGES);
        bool first = true;
        for (uint32_t m = need_mask; m != 0; m &= m - 1, ++r, first = false) {
            const int j = lo0 + __ffs(m) - 1;
            const int page = first ? page0 : row[j];
            if (granted) {
                const int fresh = __ldcg(a.free_list + r);
                row[j] = fresh;
                a.refs[fresh] = 1;
                a.src[r] = page;  // -1: an unmapped entry, nothing to copy
            } else if (r < num) {
                a.src[r] = -1;
            }
        }
    } else {
        for (int i = i0 + t / G; i < i1; i += kPlanThreads / G) {
            const int b = seq_of(i);
            Window w;
            if (b < 0 || !window_of(a, b, &w)) continue;
            int32_t* row = a.table + (long long)b * a.pg.max_blocks;
            const int lo = w.p0 <= w.p1 ? min(w.p0, w.t0) : w.t0;
            const int r0 = base + a.need[i];
            // the first pass counts, the second writes
            int total = 0;
            for (int pass = 0; pass < 2; ++pass) {
                const bool granted = r0 + total <= free_all;
                int k = 0;
                for (int j0 = lo; j0 <= w.t1; j0 += G) {
                    const int j = j0 + sub;
                    int page = -1;
                    const int kind = j <= w.t1 ? entry_need(a, w, row, j, &page) : 0;
                    int mineat = k, step = kind != 0 ? 1 : 0;
                    if (G > 1) {
                        const uint32_t m = __ballot_sync(0xffffffffu, kind != 0);
                        mineat = k + __popc(m & ((1u << sub) - 1u));
                        step = __popc(m);
                    }
                    if (pass == 1 && kind != 0) {
                        const int r = r0 + mineat;
                        if (granted) {
                            const int fresh = __ldcg(a.free_list + r);
                            row[j] = fresh;
                            a.refs[fresh] = 1;
                            a.src[r] = kind == 2 ? page : -1;
                        } else if (r < num) {
                            a.src[r] = -1;
                        }
                    }
                    k += step;
                }
                if (pass == 0) total = k;
            }
            if (r0 + total > free_all && total > 0 && sub == 0)
                flag_status(a.status, DSA_STATUS_NO_PAGES);
        }
    }
}

__global__ void __launch_bounds__(kCopyThreads)
    pages_reserve_apply(const __grid_constant__ PageArrays A, const int32_t* count,
                        const int32_t* dst, const int32_t* src, int32_t* refs) {
    pdl_wait();
    long long u, end;
    warp_share((long long)*count * max(A.pieces, 1), &u, &end);
    if (u >= end) return;
    for (PieceWalk w(A, u); u < end; ++u, w.next(A)) {
        const int s = __ldg(src + w.pair);
        if (s < 0) continue;
        if (w.piece == 0 && (threadIdx.x & 31) == 0) atomicSub(refs + s, 1);
        if (w.piece < A.pieces) copy_piece(A, w, s, __ldg(dst + w.pair));
    }
}

// ---------------------------------------------------------------------------
// dsa_pages_compact

struct CompactArgs {
    int32_t* table;
    int32_t* refs;
    int32_t* remap;     // nullable [num_pages]
    int32_t* live_out;  // nullable [1]
    int32_t* status;
    Paging pg;
    // workspace
    int32_t* head;   // live pages, moved pages
    int32_t* hole;   // [num_pages] free pages below the live count, ascending
    int32_t* live;   // [num_pages] live page by rank (those at or above the live count)
    int32_t* order;  // [num_pages] rank of such a page
};

__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads, 1)
    pages_compact_kernel(CompactArgs a) {
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();  // every CTA has started: their shared memory may be written
    pdl_trigger();
    pdl_wait();
    __shared__ Pair warp_sums[kPlanThreads / 32];
    __shared__ Pair slots[kPlanCtas];
    const int rank = cl.block_rank();
    const int t = threadIdx.x;
    const long long num = a.pg.num_blocks;
    const long long slice = ((num + kPlanCtas - 1) / kPlanCtas + 3) & ~3LL;
    const long long s0 = min(num, rank * slice), s1 = min(num, s0 + slice);
    auto live_in = [](const int4& c) { return (c.x > 0) + (c.y > 0) + (c.z > 0) + (c.w > 0); };
    int4 c0 = make_int4(0, 0, 0, 0);  // the slice's first tile stays in registers
    if (s0 + 4LL * t < s1) c0 = load_counts(a.refs, s0 + 4LL * t, s1, 0);
    int mine = live_in(c0);
    for (long long p = s0 + 4LL * (kPlanThreads + t); p < s1; p += 4LL * kPlanThreads)
        mine += live_in(load_counts(a.refs, p, s1, 0));
    Pair here, all;
    const Pair scan0 = block_scan(pair_of(0, mine), warp_sums, &here);
    int at = pair_lo(cluster_scan(cl, here, slots, &all));
    const int live = pair_lo(all);
    // `before` live pages lie below page p: a free p < live is hole p - before, a live
    // p >= live has rank before; the moved pages are the last (live - those below `live`).
    for (long long p = s0; p < s1; p += 4LL * kPlanThreads) {
        const long long q = p + 4LL * t;
        int4 c4 = c0;
        int before = at + pair_lo(scan0);
        if (slice > 4LL * kPlanThreads) {
            if (p > s0) {
                c4 = make_int4(0, 0, 0, 0);
                if (q < s1) c4 = load_counts(a.refs, q, s1, 0);
            }
            Pair total;
            before = at + pair_lo(block_scan(pair_of(0, live_in(c4)), warp_sums, &total));
            at += pair_lo(total);
        }
        const int c[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int page = (int)(q + k);
            if (q + k < s1) {
                const bool alive = c[k] > 0;
                if (page == live) a.head[1] = live - before;
                if (page < live) {
                    if (!alive) a.hole[page - before] = page;
                    if (a.remap) a.remap[page] = alive ? page : -1;
                } else if (alive) {
                    a.live[before] = page;
                    a.order[page] = before;
                } else if (a.remap) {
                    a.remap[page] = -1;
                }
                before += alive;
            }
        }
    }
    if (rank == 0 && t == 0) {
        a.head[0] = live;
        if (live == num) a.head[1] = 0;
        if (a.live_out) *a.live_out = live;
    }
}

__global__ void __launch_bounds__(kCopyThreads)
    pages_compact_apply(const __grid_constant__ PageArrays A, CompactArgs a) {
    pdl_wait();
    const int live = a.head[0], moved = a.head[1];
    const int first = live - moved;  // rank of the first moved page
    const long long entries = (long long)a.pg.batch * a.pg.max_blocks;
    for (long long e = (long long)blockIdx.x * kCopyThreads + threadIdx.x; e < entries;
         e += (long long)gridDim.x * kCopyThreads) {
        const int p = a.table[e];
        if (p < live && p >= -1) continue;
        int to = -1;
        if (p >= 0 && p < a.pg.num_blocks) {
            const int r = a.order[p];  // meaningful only where live[r] is p
            if (r >= first && r < live && a.live[r] == p) to = a.hole[r - first];
        }
        if (to < 0)
            flag_status(a.status, DSA_STATUS_BAD_BLOCK);  // a page that nobody holds: left as it is
        else
            a.table[e] = to;
    }
    long long u, end;
    warp_share((long long)moved * max(A.pieces, 1), &u, &end);
    if (u >= end) return;
    for (PieceWalk w(A, u); u < end; ++u, w.next(A)) {
        const int s = a.live[first + w.pair], d = a.hole[w.pair];
        if (w.piece == 0 && (threadIdx.x & 31) == 0) {
            a.refs[d] = a.refs[s];
            a.refs[s] = 0;
            if (a.remap) a.remap[s] = d;
        }
        if (w.piece < A.pieces) copy_piece(A, w, s, d);
    }
}

// ---------------------------------------------------------------------------
size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }

struct PagesWs {
    size_t head, a, b, c, need, owner, bytes;
};
PagesWs pages_ws(long long num_pages, int n) {
    PagesWs w;
    const size_t list = al256((size_t)num_pages * 4);
    w.head = 0;
    w.a = 256;
    w.b = w.a + list;
    w.c = w.b + list;
    w.need = w.c + list;
    w.owner = w.need + al256((size_t)n * 4);
    w.bytes = w.owner + al256((size_t)n * 4);
    return w;
}

// The paging descriptor of a page call: paged, and naming the writable tensors given.
int check_pages(const char* name, const dsa_paging* pg, const int32_t* table,
                const int32_t* refs, Paging* out) {
    int rc = check_paging(pg, 0, out);
    if (rc) return rc;
    if (!out->block_table) return fail(DSA_ERR_INVALID_ARG, "%s: the cache is not paged", name);
    if (!table || table != pg->block_table)
        return fail(DSA_ERR_INVALID_ARG,
                    "%s: block_table must be the descriptor's (writable) table", name);
    if (!refs) return fail(DSA_ERR_INVALID_ARG, "%s: refs is NULL", name);
    if (out->num_blocks > 0x7fffffffLL)
        return fail(DSA_ERR_UNSUPPORTED, "%s: more than 2^31 - 1 pages", name);
    return DSA_OK;
}

int check_arrays(const char* name, const dsa_page_arrays* in, long long num_pages,
                 PageArrays* out) {
    out->n = 0;
    out->pieces = 0;
    if (!in) return DSA_OK;
    if (in->n < 0 || in->n > DSA_MAX_PAGE_ARRAYS)
        return fail(DSA_ERR_INVALID_ARG, "%s: %d page arrays (at most %d)", name, in->n,
                    DSA_MAX_PAGE_ARRAYS);
    if (in->n > 0 && in->num_pages != num_pages)
        return fail(DSA_ERR_INVALID_ARG, "%s: page arrays of %lld pages, the pool has %lld", name,
                    (long long)in->num_pages, num_pages);
    long long pieces = 0;
    for (int i = 0; i < in->n; ++i) {
        if (!in->base[i] || in->page_bytes[i] < 1)
            return fail(DSA_ERR_INVALID_ARG, "%s: page array %d: NULL or %lld bytes a page", name,
                        i, (long long)in->page_bytes[i]);
        const bool vec = (((uintptr_t)in->base[i]) | (uintptr_t)in->page_bytes[i]) % 16 == 0;
        out->base[i] = static_cast<uint8_t*>(in->base[i]);
        out->bytes[i] = vec ? in->page_bytes[i] : -in->page_bytes[i];
        out->first[i] = (int)pieces;
        pieces += (in->page_bytes[i] + kPiece - 1) / kPiece;
        if (pieces > 0x7fffffffLL)
            return fail(DSA_ERR_UNSUPPORTED, "%s: pages are too large", name);
    }
    out->n = in->n;
    out->pieces = (int)pieces;
    return DSA_OK;
}

int check_list(const char* name, int n, const Paging& P) {
    if (n < 0) return fail(DSA_ERR_INVALID_ARG, "%s: %d sequences", name, n);
    if (n > P.batch)
        return fail(DSA_ERR_INVALID_ARG, "%s: %d sequences listed, the batch has %d", name, n,
                    P.batch);
    return DSA_OK;
}

int launch_rows(const char* name, void (*kernel)(SeqArgs), const SeqArgs& a, cudaStream_t st) {
    const int chunks = (a.pg.max_blocks + kRowChunk - 1) / kRowChunk;
    if (chunks > 65535) return fail(DSA_ERR_UNSUPPORTED, "%s: max_blocks %d", name, a.pg.max_blocks);
    cudaError_t e = launch_pdl(kernel, dim3((unsigned)a.n, (unsigned)chunks), dim3(kRowThreads), 0,
                               st, a);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, name);
    return DSA_OK;
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" int dsa_pages_workspace(long long num_pages, int batch, size_t* bytes) {
    if (!bytes) return fail(DSA_ERR_INVALID_ARG, "dsa_pages_workspace: bytes is NULL");
    if (num_pages < 1 || num_pages > 0x7fffffffLL || batch < 1)
        return fail(DSA_ERR_INVALID_ARG, "dsa_pages_workspace: %lld pages, batch %d", num_pages,
                    batch);
    *bytes = pages_ws(num_pages, batch).bytes;
    return DSA_OK;
}

extern "C" int dsa_pages_free(const int32_t* seqs, int n, const dsa_paging* pg,
                              int32_t* block_table, int32_t* seq_lens, int32_t* refs,
                              int32_t* status, void* stream) {
    SeqArgs a;
    int rc = check_pages("dsa_pages_free", pg, block_table, refs, &a.pg);
    if (rc) return rc;
    if (!seq_lens || seq_lens != pg->seq_lens)
        return fail(DSA_ERR_INVALID_ARG,
                    "dsa_pages_free: seq_lens must be the descriptor's (writable) lengths");
    rc = check_list("dsa_pages_free", n, a.pg);
    if (rc) return rc;
    if (n == 0) return DSA_OK;
    if (!seqs) return fail(DSA_ERR_INVALID_ARG, "dsa_pages_free: NULL sequences");
    a.list = seqs;
    a.parents = nullptr;
    a.n = n;
    a.table = block_table;
    a.seq_lens = seq_lens;
    a.refs = refs;
    a.status = status;
    return launch_rows("dsa_pages_free launch", pages_free_kernel, a, (cudaStream_t)stream);
}

extern "C" int dsa_pages_fork(const int32_t* parents, const int32_t* children, int n,
                              const dsa_paging* pg, int32_t* block_table, int32_t* seq_lens,
                              int32_t* refs, int32_t* status, void* stream) {
    SeqArgs a;
    int rc = check_pages("dsa_pages_fork", pg, block_table, refs, &a.pg);
    if (rc) return rc;
    if (!seq_lens || seq_lens != pg->seq_lens)
        return fail(DSA_ERR_INVALID_ARG,
                    "dsa_pages_fork: seq_lens must be the descriptor's (writable) lengths");
    rc = check_list("dsa_pages_fork", n, a.pg);
    if (rc) return rc;
    if (n == 0) return DSA_OK;
    if (!parents || !children)
        return fail(DSA_ERR_INVALID_ARG, "dsa_pages_fork: NULL sequences");
    a.list = children;
    a.parents = parents;
    a.n = n;
    a.table = block_table;
    a.seq_lens = seq_lens;
    a.refs = refs;
    a.status = status;
    return launch_rows("dsa_pages_fork launch", pages_fork_kernel, a, (cudaStream_t)stream);
}

extern "C" int dsa_pages_serve(const int32_t* parents, const int32_t* seqs, int n, int batch,
                               int on, int32_t* serving, int32_t* status, void* stream) {
    if (batch < 1) return fail(DSA_ERR_INVALID_ARG, "dsa_pages_serve: batch %d < 1", batch);
    if (n < 0 || n > batch)
        return fail(DSA_ERR_INVALID_ARG, "dsa_pages_serve: %d sequences listed, the batch has %d",
                    n, batch);
    if (!serving) return fail(DSA_ERR_INVALID_ARG, "dsa_pages_serve: serving is NULL");
    if (n == 0) return DSA_OK;
    if (!seqs) return fail(DSA_ERR_INVALID_ARG, "dsa_pages_serve: NULL sequences");
    cudaError_t e = launch_pdl(pages_serve_kernel, dim3((unsigned)n), dim3(kRowThreads), 0,
                               (cudaStream_t)stream, parents, seqs, n, batch, on, serving, status);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "dsa_pages_serve launch");
    return DSA_OK;
}

extern "C" int dsa_pages_reserve(const int32_t* seqs, int n, const dsa_paging* pg,
                                 int32_t* block_table, int32_t* refs, int new_tokens,
                                 int first_key, int kpool, const dsa_page_arrays* arrays,
                                 int32_t* status, void* workspace, size_t workspace_bytes,
                                 void* stream) {
    ReserveArgs a;
    int rc = check_pages("dsa_pages_reserve", pg, block_table, refs, &a.pg);
    if (rc) return rc;
    if (!seqs) n = a.pg.batch;
    rc = check_list("dsa_pages_reserve", n, a.pg);
    if (rc) return rc;
    if (new_tokens < 1)
        return fail(DSA_ERR_INVALID_ARG, "dsa_pages_reserve: new_tokens %d < 1", new_tokens);
    if (kpool < 0 || kpool > DSA_MAX_KPOOL)
        return fail(DSA_ERR_UNSUPPORTED, "dsa_pages_reserve: kpool %d outside [0, %d]", kpool,
                    DSA_MAX_KPOOL);
    if (first_key < 0)
        return fail(DSA_ERR_INVALID_ARG, "dsa_pages_reserve: first_key %d < 0", first_key);
    if (kpool > 0 && (a.pg.block_size % kpool != 0 || first_key % kpool != 0))
        return fail(DSA_ERR_UNSUPPORTED,
                    "dsa_pages_reserve: block_size %d and first_key %d must be multiples of "
                    "kpool %d",
                    a.pg.block_size, first_key, kpool);
    // at most this many pages in a sequence's two windows; the needs are summed in 32 bits
    const long long window = 2LL * (new_tokens / a.pg.block_size + 2);
    if (n * (window < a.pg.max_blocks ? window : a.pg.max_blocks) > 0x7fffffffLL)
        return fail(DSA_ERR_UNSUPPORTED, "dsa_pages_reserve: %d sequences of %d new tokens", n,
                    new_tokens);
    PageArrays A;
    rc = check_arrays("dsa_pages_reserve", arrays, a.pg.num_blocks, &A);
    if (rc) return rc;
    const PagesWs w = pages_ws(a.pg.num_blocks, a.pg.batch);
    if (!workspace || workspace_bytes < w.bytes || ((uintptr_t)workspace & 15))
        return fail(DSA_ERR_INVALID_ARG,
                    "dsa_pages_reserve: workspace %zu B < %zu B needed (16-byte aligned)",
                    workspace_bytes, w.bytes);
    if (n == 0) return DSA_OK;
    const int sms = sm_count();
    if (sms <= 0) return fail(DSA_ERR_CUDA, "dsa_pages_reserve: no CUDA device");
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.list = seqs;
    a.n = n;
    a.new_tokens = new_tokens;
    a.first_key = first_key;
    a.kpool = kpool;
    a.table = block_table;
    a.refs = refs;
    a.status = status;
    a.count = reinterpret_cast<int32_t*>(ws + w.head);
    a.free_list = reinterpret_cast<int32_t*>(ws + w.a);
    a.src = reinterpret_cast<int32_t*>(ws + w.b);
    a.need = reinterpret_cast<int32_t*>(ws + w.need);
    a.owner = reinterpret_cast<int32_t*>(ws + w.owner);
    cudaStream_t st = (cudaStream_t)stream;
    // one lane per sequence while its window is a few pages (a decode step), a warp where
    // it may be many (the pages of a prompt); with one lane a sequence's entries, from its
    // pooled-key page to its last token page, have to fit a mask to stay in registers
    const bool wide = new_tokens / a.pg.block_size >= 4;
    const long long span = first_key / a.pg.block_size + new_tokens / a.pg.block_size + 3;
    const bool one = !wide && (long long)n <= (long long)kPlanCtas * kPlanThreads && span <= 32;
    auto plan = wide  ? pages_reserve_kernel<32, false>
                : one ? pages_reserve_kernel<1, true>
                      : pages_reserve_kernel<1, false>;
    cudaError_t e = launch_pdl(plan, dim3(kPlanCtas), dim3(kPlanThreads), 0, st, a);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "dsa_pages_reserve launch");
    e = launch_pdl(pages_reserve_apply, dim3((unsigned)sms * 4), dim3(kCopyThreads), 0, st, A,
                   (const int32_t*)a.count, (const int32_t*)a.free_list, (const int32_t*)a.src,
                   refs);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "dsa_pages_reserve copy launch");
    return DSA_OK;
}

extern "C" int dsa_pages_compact(const dsa_paging* pg, int32_t* block_table, int32_t* refs,
                                 const dsa_page_arrays* arrays, int32_t* remap, int32_t* live,
                                 int32_t* status, void* workspace, size_t workspace_bytes,
                                 void* stream) {
    CompactArgs a;
    int rc = check_pages("dsa_pages_compact", pg, block_table, refs, &a.pg);
    if (rc) return rc;
    PageArrays A;
    rc = check_arrays("dsa_pages_compact", arrays, a.pg.num_blocks, &A);
    if (rc) return rc;
    const PagesWs w = pages_ws(a.pg.num_blocks, a.pg.batch);
    if (!workspace || workspace_bytes < w.bytes || ((uintptr_t)workspace & 15))
        return fail(DSA_ERR_INVALID_ARG,
                    "dsa_pages_compact: workspace %zu B < %zu B needed (16-byte aligned)",
                    workspace_bytes, w.bytes);
    const int sms = sm_count();
    if (sms <= 0) return fail(DSA_ERR_CUDA, "dsa_pages_compact: no CUDA device");
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.table = block_table;
    a.refs = refs;
    a.remap = remap;
    a.live_out = live;
    a.status = status;
    a.head = reinterpret_cast<int32_t*>(ws + w.head);
    a.hole = reinterpret_cast<int32_t*>(ws + w.a);
    a.live = reinterpret_cast<int32_t*>(ws + w.b);
    a.order = reinterpret_cast<int32_t*>(ws + w.c);
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e = launch_pdl(pages_compact_kernel, dim3(kPlanCtas), dim3(kPlanThreads), 0, st, a);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "dsa_pages_compact launch");
    e = launch_pdl(pages_compact_apply, dim3((unsigned)sms * 8), dim3(kCopyThreads), 0, st, A, a);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "dsa_pages_compact copy launch");
    return DSA_OK;
}
