// dsa_route: a router's scores to the chosen experts and their weights.
// dsa_router_logits: the logits, x . w^T with f32 results (the projection of project.cu).
//
//   s_e = sigmoid(logit_e) or softmax(logits)_e        c_e = s_e + bias_e
//   groups: the topk_group groups whose group_top best c have the largest sum
//   experts: the topk largest c among those groups, ties to the lowest id, written in
//   ascending id; weight = s_e (over the sum of the chosen s when renorm) * scale
//
// One warp per row; expert e is lane e % 32's piece e / 32. Rows are few or short (a
// thousand bytes), so latency and instructions bound it, not memory (32,749 rows of 256 experts in 8
// groups: 41 us, the bytes' 5 us; 8 rows: 3.5 us): the best expert of
// a round is one warp reduction over the lanes' best, each lane's pieces sorted.
//
// The choice is the one that 64-bit arithmetic makes. It is first made in f32; every c
// computed so is within err of the exact one, so where the smallest chosen and the largest
// rejected value (of experts, or of groups) are further apart than the errors of both, the
// f32 choice is final. Else, one to two rows in a hundred for unrelated scores, what is not is
// compared in f64; a softmax with a bias, whose common factor matters, repeats the whole row.
// (A whole row in f64 takes about 20 us on this part's few FP64 units, half as long as 32,749 rows
// in f32: it was the tail that a batch waited for. Rows of equal logits, where all experts are in doubt
// and each round evaluates them again, take longest: 8 of 256 experts, topk 8, 68 us.)
#include "common.cuh"

namespace dsa {
namespace {

constexpr int kRouteWarps = 4;
constexpr uint32_t kAll = 0xffffffffu;
constexpr int kSets = (DSA_MAX_TOPK + 31) / 32;  // registers for one chosen expert per lane

struct RouteArgs {
    const float* logits;
    const float* bias;  // nullable
    int32_t* ids;
    float* weights;
    long long ld;
    int rows, n, groups, gsize, topk_group, group_top, topk, shared;
    int per_log;      // log2 of the lanes that scan a group: 32 / groups, rounded down
    uint32_t gmagic;  // 2^32 / gsize, rounded up; 0 for 1
    int softmax, renorm;
    float scale;
};

__device__ __forceinline__ float exp_t(float x) { return expf(x); }
__device__ __forceinline__ double exp_t(double x) { return exp(x); }
template <typename T>
__device__ __forceinline__ T neg_inf();
template <>
__device__ __forceinline__ float neg_inf<float>() { return __uint_as_float(0xff800000u); }
template <>
__device__ __forceinline__ double neg_inf<double>() { return __longlong_as_double(0xfff0000000000000ll); }

// Larger value, larger key; -0 and +0 alike; -inf has the lowest key of any number.
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t b = __float_as_uint(v + 0.f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ float warp_max_t(float v) { return of_key(__reduce_max_sync(kAll, key_of(v))); }
// (By integers: this part's FP64 units are few, a comparison there takes as long as dozens here.)
__device__ __forceinline__ double warp_max_t(double v) {
    unsigned long long b = (unsigned long long)__double_as_longlong(v + 0.0);
    b ^= (b >> 63) ? ~0ull : 1ull << 63;
    const uint32_t hi = __reduce_max_sync(kAll, (uint32_t)(b >> 32));
    const uint32_t lo = __reduce_max_sync(kAll, (uint32_t)(b >> 32) == hi ? (uint32_t)b : 0u);
    b = (unsigned long long)hi << 32 | lo;
    b ^= (b >> 63) ? 1ull << 63 : ~0ull;
    return __longlong_as_double((long long)b);
}
__device__ __forceinline__ float max_t(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ float min_t(float a, float b) { return fminf(a, b); }
__device__ __forceinline__ double max_t(double a, double b) { return fmax(a, b); }
__device__ __forceinline__ double min_t(double a, double b) { return fmin(a, b); }
// 2^x and 1 / x on the special-function unit, subnormals taken as zero.
__device__ __forceinline__ float ex2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <typename T>
__device__ __forceinline__ T warp_sum_t(T v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// e / a.gsize for e < 2^10.
__device__ __forceinline__ int group_of(const RouteArgs& a, int e) {
    return a.gmagic ? (int)__umulhi((uint32_t)e, a.gmagic) : e;
}

// The best two of each group's values, from the warp's staging area (value e at e + e / 32): 32 / groups lanes, rounded down to a power of two, scan one group. Lane g * per of
// group g has its score in *own and the smallest value in it in *least, the other lanes -inf.
// Returns the mask of the `most` best groups; *low: the worst of them, *next: the best other.
template <typename T>
__device__ __forceinline__ uint32_t best_groups(const RouteArgs& a, const T* buf, int lane, int most, T* own, T* least,
                                                T* low, T* next) {
    const T NI = neg_inf<T>();
    const int per = 1 << a.per_log, g = lane >> a.per_log, j0 = lane & (per - 1);
    T b1 = NI, b2 = NI;
    if (g < a.groups) {
        const int first = g * a.gsize;
        for (int e = first + j0; e < first + a.gsize; e += per) {
            const T v = buf[e + (e >> 5)];
            b2 = max_t(b2, min_t(b1, v));
            b1 = max_t(b1, v);
        }
    }
    for (int o = per >> 1; o > 0; o >>= 1) {
        const T o1 = __shfl_xor_sync(kAll, b1, o), o2 = __shfl_xor_sync(kAll, b2, o);
        b2 = max_t(max_t(b2, o2), min_t(b1, o1));
        b1 = max_t(b1, o1);
    }
    T score = b1;
    if (a.group_top == 2 && b2 > NI) score += b2;
    if (g >= a.groups || j0 != 0) score = NI;
    *own = score;
    *least = a.group_top == 2 && b2 > NI ? b2 : b1;
    uint32_t kept = 0;
    *low = NI;
    for (int k = 0; k < most; ++k) {
        const T m = warp_max_t(score);
        if (!(m > NI)) break;
        const int at = __ffs(__ballot_sync(kAll, score == m)) - 1;  // the lowest group of equal ones
        kept |= 1u << (at >> a.per_log);
        if (lane == at) score = NI;
        *low = m;
    }
    *next = warp_max_t(score);
    return kept;
}

// The topk largest c, ties to the lowest expert; bit i of the result: the lane's piece i is
// chosen.
template <typename T, int NPL>
__device__ __forceinline__ uint32_t best_experts(const RouteArgs& a, const T (&c)[NPL], int lane) {
    const T NI = neg_inf<T>();
    uint32_t taken = 0;
    T best = NI;
    int at = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i)
        if (c[i] > best) {
            best = c[i];
            at = i;
        }
    for (int k = 0; k < a.topk; ++k) {
        const T m = warp_max_t(best);
        if (!(m > NI)) break;
        const uint32_t who = __ballot_sync(kAll, best == m);
        bool mine = best == m;
        if (who & (who - 1))  // several lanes: the lowest expert
            mine = mine && __reduce_min_sync(who, (uint32_t)(lane + 32 * at)) == (uint32_t)(lane + 32 * at);
        if (mine) {
            taken |= 1u << at;
            best = NI;
#pragma unroll
            for (int i = 0; i < NPL; ++i)
                if (!((taken >> i) & 1u) && c[i] > best) {
                    best = c[i];
                    at = i;
                }
        }
    }
    return taken;
}

// The same in f32, for values that are certain: each lane sorts its pieces' keys into its column
// of `list`, and a round takes the largest head. A key is the value's order, its last bits
// replaced by the expert's number (piece and lane), the lower the larger; 0 for none. So keys
// differ, and one reduction a round says all. Lane j gets the key of the j-th best in
// mine[j / 32]. *low: the worst chosen value, *next: the best other (-inf if none), both cut
// down to a multiple of 32 NPL ulps. Returns how many there are.
template <int NPL>
__device__ __forceinline__ int best_keys(const RouteArgs& a, const float (&c)[NPL], int lane, uint32_t* list, float* low,
                                         float* next, uint32_t (&mine)[kSets]) {
    constexpr uint32_t kCut = 32 * NPL - 1;
    uint32_t k[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const uint32_t b = __float_as_uint(c[i]);  // (a -0 sorts below +0: their gap is 0, a doubt)
        const uint32_t o = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
        k[i] = c[i] > neg_inf<float>() ? (o & ~kCut) | (kCut - (uint32_t)(lane + 32 * i)) : 0u;
    }
    // Batcher's odd-even merge sort, largest first
#pragma unroll
    for (int p = 1; p < NPL; p <<= 1)
#pragma unroll
        for (int q = p; q >= 1; q >>= 1)
#pragma unroll
            for (int j = q % p; j + q < NPL; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i)
                    if (i + j + q < NPL && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
                        const uint32_t hi = max(k[i + j], k[i + j + q]);
                        k[i + j + q] = min(k[i + j], k[i + j + q]);
                        k[i + j] = hi;
                    }
#pragma unroll
    for (int i = 1; i < NPL; ++i) list[32 * (i - 1) + lane] = k[i];
    list[32 * (NPL - 1) + lane] = 0u;
    const uint32_t* then = list + lane;
    uint32_t head = k[0], worst = 0;
    int count = 0;
#pragma unroll
    for (int q = 0; q < kSets; ++q) {
        mine[q] = 0;
        const int rounds = min(32, a.topk - 32 * q);
        for (int j = 0; j < rounds; ++j) {
            const uint32_t m = __reduce_max_sync(kAll, head);
            if (m == 0) break;
            worst = m;
            ++count;
            mine[q] = lane == j ? m : mine[q];
            if (head == m) {
                head = *then;
                then += 32;
            }
        }
    }
    const uint32_t other = __reduce_max_sync(kAll, head);
    *low = worst ? of_key(worst & ~kCut) : neg_inf<float>();
    *next = other ? of_key(other & ~kCut) : neg_inf<float>();
    return count;
}

// c of expert e in f64 (a softmax score without the factor that all have: there is no bias then).
__device__ __forceinline__ double value_f64(const RouteArgs& a, long long r, float top, int e) {
    const double z = (double)__ldg(a.logits + r * a.ld + e);
    double v = a.softmax ? exp(z - (double)top) : 1 / (1 + exp(-z));
    if (a.bias) v += (double)__ldg(a.bias + e);
    return v;
}

// The best `most` of the pieces in `doubt`.
__device__ __noinline__ uint32_t choose_f64(const RouteArgs& a, long long r, int lane, float top, uint32_t doubt,
                                            int most) {
    uint32_t taken = 0;
    for (int round = 0; round < most; ++round) {
        double best = neg_inf<double>();
        int at = 0;
        for (uint32_t left = doubt & ~taken; left; left &= left - 1) {
            const int i = __ffs(left) - 1;
            const double v = value_f64(a, r, top, lane + 32 * i);
            if (v > best) {
                best = v;
                at = i;
            }
        }
        const double m = warp_max_t(best);
        const uint32_t who = __ballot_sync(kAll, best == m && best > neg_inf<double>());
        if (!who) break;
        if ((who >> lane) & 1u)
            if (__reduce_min_sync(who, (uint32_t)(lane + 32 * at)) == (uint32_t)(lane + 32 * at)) taken |= 1u << at;
        __syncwarp();
    }
    return taken;
}

// The best `most` of the groups in doubt, of which the pieces `needed` hold all that may be in
// their sums.
__device__ __noinline__ uint32_t choose_groups_f64(const RouteArgs& a, long long r, int lane, float top, uint32_t needed,
                                                   int pieces, int most, double* buf) {
    __syncwarp();
    for (int i = 0; i < pieces; ++i)
        buf[33 * i + lane] = (needed >> i) & 1u ? value_f64(a, r, top, lane + 32 * i) : neg_inf<double>();
    __syncwarp();
    double own, least, low, next;
    return best_groups(a, buf, lane, most, &own, &least, &low, &next);
}

// The chosen experts (count >= 0 of them, by their keys; else by the bits of `taken`),
// their scores and the row's outputs in ascending expert id; then padding and shared experts.
// Lane k takes the k-th chosen one; T: what the scores are computed in. In f32
// it gives up (false) where a ratio of scores, or a score to be scaled up, needs digits that numbers
// near f32's smallest lack, and where the scale over the sum of the scores passes its largest.
template <typename T, int NPL>
__device__ __forceinline__ bool emit(const RouteArgs& a, long long r, int lane, uint32_t taken, int count,
                                     const uint32_t (&mine)[kSets], T top, T inv, bool nan, int* chosen) {
    const int width = a.topk + a.shared;
    int32_t* ids = a.ids + r * width;
    float* weights = a.weights + r * width;
    const float* row = a.logits + r * a.ld;
    int n = count;
    __syncwarp();  // the staging area is free
    if (n >= 0) {  // each to the place of its rank: the larger the number in the key, the earlier
#pragma unroll
        for (int q = 0; q < kSets; ++q) {
            if (32 * q >= n) break;
            const uint32_t number = mine[q] & (32 * NPL - 1);
            int rank = 0;
#pragma unroll
            for (int p = 0; p < kSets; ++p)
                for (int j = 0; j < min(32, n - 32 * p); ++j)
                    rank += (__shfl_sync(kAll, mine[p], j) & (32 * NPL - 1)) > number;
            if (lane + 32 * q < n) chosen[rank] = 32 * NPL - 1 - number;
        }
    } else {
        n = 0;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const bool here = (taken >> i) & 1u;
            const uint32_t who = __ballot_sync(kAll, here);
            if (here) chosen[n + __popc(who & ((1u << lane) - 1u))] = lane + 32 * i;
            n += __popc(who);
        }
    }
    __syncwarp();
    T s[kSets], total = 0;
    bool tiny = false;
#pragma unroll
    for (int q = 0; q < kSets; ++q) {
        s[q] = 0;
        if (lane + 32 * q < n) {
            const T z = (T)__ldg(row + chosen[lane + 32 * q]);
            s[q] = a.softmax ? exp_t(z - top) * inv : (T)1 / ((T)1 + exp_t(-z));
            tiny |= s[q] < (T)1e-30;
        }
        total += s[q];
    }
    if (sizeof(T) == 4 && (a.renorm || fabsf(a.scale) > 1.f) && __any_sync(kAll, tiny)) return false;
    T f = (T)a.scale;
    if (a.renorm) {
        total = warp_sum_t(total);
        f = total > 0 ? f / total : (T)0;
        if (sizeof(T) == 4 && !(fabs(f) < (T)3.4e38)) return false;
    }
#pragma unroll
    for (int q = 0; q < kSets; ++q) {
        const int k = lane + 32 * q;
        if (k < n) {
            ids[k] = chosen[k];
            weights[k] = nan ? __uint_as_float(0x7fc00000u) : (float)(s[q] * f);
        }
    }
    for (int k = n + lane; k < width; k += 32) {
        const bool extra = k >= a.topk;
        ids[k] = extra ? a.n + (k - a.topk) : -1;
        weights[k] = extra ? 1.f : 0.f;
    }
    return true;
}

// A row in f64 throughout. A function of its own, seldom called: its registers and
// instructions stay out of the rows that f32 decides.
template <int NPL>
__device__ __noinline__ void route_row_f64(const RouteArgs& a, long long r, int lane, double* buf) {
    const double NI = neg_inf<double>();
    const float* row = a.logits + r * a.ld;
    double s[NPL], c[NPL], top = NI;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = lane + 32 * i;
        double z = e < a.n ? (double)__ldg(row + e) : NI;
        if (!(z == z) || (a.softmax && z > 3.5e38)) {
            bad = true;
            z = NI;
        }
        c[i] = z;  // the logit, until its score is known
        top = z > top ? z : top;
    }
    top = warp_max_t(top);
    double sum = 0, inv = 1;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        s[i] = 0;
        if (c[i] > NI) s[i] = a.softmax ? exp(c[i] - top) : 1 / (1 + exp(-c[i]));
        sum += s[i];
    }
    if (a.softmax) {
        sum = warp_sum_t(sum);
        inv = sum > 0 ? 1 / sum : 0;
#pragma unroll
        for (int i = 0; i < NPL; ++i) s[i] *= inv;
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = lane + 32 * i;
        const double b = a.bias && e < a.n ? (double)__ldg(a.bias + e) : 0;
        if (!(b == b)) {
            bad = true;
            c[i] = NI;
        }
        c[i] = c[i] > NI ? s[i] + b : NI;
    }
    const bool nan = __any_sync(kAll, bad);
    if (a.groups > 1) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < NPL; ++i) buf[33 * i + lane] = c[i];
        __syncwarp();
        double own, least, low, next;
        const uint32_t kept = best_groups(a, buf, lane, a.topk_group, &own, &least, &low, &next);
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = lane + 32 * i;
            if (e < a.n && !((kept >> group_of(a, e)) & 1u)) c[i] = NI;
        }
    }
    const uint32_t taken = best_experts(a, c, lane);
    const uint32_t none[kSets] = {};
    emit<double, NPL>(a, r, lane, taken, -1, none, top, inv, nan, reinterpret_cast<int*>(buf));
}

template <int NPL, bool SOFTMAX>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(RouteArgs a) {
    __shared__ __align__(8) unsigned char stage[kRouteWarps][33 * NPL * sizeof(double)];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float NI = neg_inf<float>();
    pdl_wait();
    const long long r = (long long)blockIdx.x * kRouteWarps + warp;
    if (r >= a.rows) return;
    {
        float z[NPL], c[NPL];
        bool bad = false;
        float top = NI, inv = 1.f, smax = 0.f, bmax = 0.f;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = lane + 32 * i;
            z[i] = e < a.n ? __ldg(a.logits + r * a.ld + e) : NI;
        }
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const bool odd = SOFTMAX ? !(z[i] < __uint_as_float(0x7f800000u)) : !(z[i] == z[i]);
            bad |= odd;
            z[i] = odd ? NI : z[i];
            if (SOFTMAX) top = fmaxf(top, z[i]);
        }
        // Scores by the special-function unit, for the choice: a softmax's within 2^-21 of the largest of
        // them, its common factor within 2^-18 of itself; a sigmoid's see below.
        constexpr float kLog2e = 1.4426950408889634f;
        if (SOFTMAX) {
            top = warp_max_t(top);
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                c[i] = z[i] > NI ? ex2_fast((z[i] - top) * kLog2e) : 0.f;
                sum += c[i];
            }
            sum = warp_sum_t(sum);
            inv = sum > 0.f ? 1.f / sum : 0.f;
            smax = inv;  // the largest logit's
        }
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const float s = SOFTMAX ? c[i] * inv : rcp_fast(1.f + ex2_fast(z[i] * -kLog2e));
            if (!SOFTMAX) smax = fmaxf(smax, s);
            c[i] = z[i] > NI ? s : NI;
        }
        if (!SOFTMAX) smax = warp_max_t(smax);
        if (a.bias) {
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                const int e = lane + 32 * i;
                const float b = e < a.n ? __ldg(a.bias + e) : 0.f;
                bad |= !(b == b);
                c[i] = c[i] > NI && b == b ? c[i] + b : NI;
                const float m = fabsf(b);
                bmax = m < 1e30f ? fmaxf(bmax, m) : bmax;  // (larger ones make no close call)
            }
            bmax = warp_max_t(bmax);
        }
        const bool nan = __any_sync(kAll, bad);
        // |c as computed - c|: the score's error (but for the softmax's common factor, which moves
        // no score past another), the addition's and half of a group sum's. A sigmoid's: 2^-22 by
        // the power of two, 2^-23 by the reciprocal, 2^-24 by the sum under it, and |z| (2^-24 + 2^-26)
        // by the rounding of z log2(e) and of that constant, less the more s exceeds 1/2. s |z| is
        // largest at the largest logit, whose -z is at most -ln(smax), or near 1. (1e-37: what the
        // unit takes for zero.)
        const float far = SOFTMAX ? 1.f : fmaxf(1.f, fminf(-__logf(smax), 128.f));
        const float err = (SOFTMAX ? (a.bias ? 3.8146973e-6f : 4.7683716e-7f) : 5.4e-7f + 7.6e-8f * far) * smax +
                          1.2e-7f * bmax + 1e-37f;
        bool sure = true;
        if (a.groups > 1) {
            float* buf = reinterpret_cast<float*>(stage[warp]);
            float own, least, low, next;
#pragma unroll
            for (int i = 0; i < NPL; ++i) buf[33 * i + lane] = c[i];
            __syncwarp();
            uint32_t kept = best_groups(a, buf, lane, a.topk_group, &own, &least, &low, &next);
            if (next > NI && !(low - next > 4 * err)) {
                sure = !(SOFTMAX && a.bias) && fabsf(low) < 1e30f;
                if (sure) {  // the groups near the border, by what may be in their sums
                    const int g = lane >> a.per_log;
                    const bool near = own > NI && ((kept >> g) & 1u ? own <= next + 4 * err : own >= low - 4 * err);
                    const uint32_t doubt = __reduce_or_sync(kAll, near ? 1u << g : 0u);
                    uint32_t needed = 0;
#pragma unroll
                    for (int i = 0; i < NPL; ++i) {
                        const int e = lane + 32 * i, h = e < a.n ? group_of(a, e) : 0;
                        const float from = __shfl_sync(kAll, least, h << a.per_log) - 2 * err;
                        if (e < a.n && ((doubt >> h) & 1u) && c[i] > NI && c[i] >= from) needed |= 1u << i;
                    }
                    kept = (kept & ~doubt) | choose_groups_f64(a, r, lane, top, needed, NPL, __popc(kept & doubt),
                                                               reinterpret_cast<double*>(stage[warp]));
                }
            }
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                const int e = lane + 32 * i;
                if (e < a.n && !((kept >> group_of(a, e)) & 1u)) c[i] = NI;
            }
        }
        __syncwarp();
        float low, next;
        uint32_t mine[kSets], taken = 0;
        int count = best_keys(a, c, lane, reinterpret_cast<uint32_t*>(stage[warp]), &low, &next, mine);
        // two errors, and what the keys cut off
        const float margin = 2 * err + (fabsf(low) + fabsf(next)) * (32 * NPL * 1.1920929e-7f);
        if (sure && next > NI && !(low - next > margin)) {
            sure = !(SOFTMAX && a.bias) && fabsf(low) < 1e30f;
            if (sure) {  // only what lies that near to the border is in doubt
#pragma unroll
                for (int q = 0; q < kSets; ++q)
                    for (int j = 0; j < min(32, count - 32 * q); ++j) {
                        const int e = 32 * NPL - 1 - (int)(__shfl_sync(kAll, mine[q], j) & (32 * NPL - 1));
                        taken |= (e & 31) == lane ? 1u << (e >> 5) : 0u;
                    }
                uint32_t doubt = 0;
#pragma unroll
                for (int i = 0; i < NPL; ++i)
                    if ((taken >> i) & 1u ? c[i] <= next + margin : c[i] > NI && c[i] >= low - margin) doubt |= 1u << i;
                const int most = (int)__reduce_add_sync(kAll, (uint32_t)__popc(taken & doubt));
                taken = (taken & ~doubt) | choose_f64(a, r, lane, top, doubt, most);
                count = -1;
            }
        }
        if (!sure || !emit<float, NPL>(a, r, lane, taken, count, mine, top, inv, nan, reinterpret_cast<int*>(stage[warp])))
            route_row_f64<NPL>(a, r, lane, reinterpret_cast<double*>(stage[warp]));
    }
}

template <int NPL>
cudaError_t route_launch(const RouteArgs& a, cudaStream_t st) {
    // (A warp for several rows, their biases looked up once, was slower: a row in doubt holds up
    // those behind it.)
    const dim3 grid((unsigned)(((long long)a.rows + kRouteWarps - 1) / kRouteWarps)), block(kRouteWarps * 32);
    return a.softmax ? launch_pdl(route_kernel<NPL, true>, grid, block, 0, st, a)
                     : launch_pdl(route_kernel<NPL, false>, grid, block, 0, st, a);
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" int dsa_route(const float* logits, int rows, int n_experts, long long ld, int score,
                         const float* bias, int n_group, int topk_group, int group_top, int topk,
                         int renorm, float scale, int shared, int32_t* ids, float* weights,
                         void* stream) {
    if (rows < 0 || n_experts < 1 || ld < n_experts || topk < 1 || shared < 0)
        return fail(DSA_ERR_INVALID_ARG,
                    "dsa_route: rows %d, n_experts %d, ld %lld, topk %d, shared %d", rows, n_experts,
                    ld, topk, shared);
    if (n_experts > DSA_MAX_EXPERTS || topk > DSA_MAX_TOPK || n_group > 32 || shared > DSA_MAX_TOPK)
        return fail(DSA_ERR_UNSUPPORTED,
                    "dsa_route: at most %d experts, topk and shared %d, 32 groups (got %d, %d, %d, %d)",
                    DSA_MAX_EXPERTS, DSA_MAX_TOPK, n_experts, topk, shared, n_group);
    if (score != DSA_ROUTE_SIGMOID && score != DSA_ROUTE_SOFTMAX)
        return fail(DSA_ERR_INVALID_ARG, "dsa_route: score %d", score);
    if (n_group < 1 || n_experts % n_group != 0 || topk_group < 1 || topk_group > n_group ||
        group_top < 1 || group_top > 2 || (n_group > 1 && group_top > n_experts / n_group))
        return fail(DSA_ERR_INVALID_ARG,
                    "dsa_route: %d groups of %d experts, topk_group %d, group_top %d", n_group,
                    n_experts, topk_group, group_top);
    if (topk > topk_group * (n_experts / n_group))
        return fail(DSA_ERR_INVALID_ARG, "dsa_route: topk %d of %d groups of %d experts", topk,
                    topk_group, n_experts / n_group);
    if (!(scale == scale) || scale > 3.4e38f || scale < -3.4e38f)
        return fail(DSA_ERR_INVALID_ARG, "dsa_route: scale must be finite");
    if (rows == 0) return DSA_OK;
    if (!logits || !ids || !weights) return fail(DSA_ERR_INVALID_ARG, "dsa_route: NULL tensor");
    if ((((uintptr_t)logits) | ((uintptr_t)bias) | ((uintptr_t)ids) | ((uintptr_t)weights)) & 3)
        return fail(DSA_ERR_INVALID_ARG, "dsa_route: misaligned tensor");
    RouteArgs a;
    a.logits = logits;
    a.bias = bias;
    a.ids = ids;
    a.weights = weights;
    a.ld = ld;
    a.rows = rows;
    a.n = n_experts;
    a.groups = n_group;
    a.gsize = n_experts / n_group;
    a.gmagic = a.gsize > 1 ? (uint32_t)(0xffffffffu / (uint32_t)a.gsize + 1) : 0u;
    a.per_log = 5;
    while ((n_group << a.per_log) > 32) --a.per_log;
    a.topk_group = topk_group;
    a.group_top = group_top;
    a.topk = topk;
    a.shared = shared;
    a.softmax = score == DSA_ROUTE_SOFTMAX;
    a.renorm = renorm != 0;
    a.scale = scale;
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e;
    if (n_experts <= 64)
        e = route_launch<2>(a, st);
    else if (n_experts <= 128)
        e = route_launch<4>(a, st);
    else if (n_experts <= 256)
        e = route_launch<8>(a, st);
    else if (n_experts <= 512)
        e = route_launch<16>(a, st);
    else
        e = route_launch<32>(a, st);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "dsa_route launch");
    return DSA_OK;
}

static int check_logits(const char* name, int rows, int hidden, int n) {
    if (rows < 0 || hidden < 1 || n < 1)
        return fail(DSA_ERR_INVALID_ARG, "%s: rows %d, hidden %d, n %d", name, rows, hidden, n);
    if (!project_supported(hidden, n))
        return fail(DSA_ERR_UNSUPPORTED,
                    "%s: hidden must be a multiple of 256 and n of 64 (got %d, %d; pad w with rows of "
                    "zeros)", name, hidden, n);
    return DSA_OK;
}

extern "C" int dsa_router_logits_workspace(int rows, int hidden, int n, size_t* bytes) {
    if (!bytes) return fail(DSA_ERR_INVALID_ARG, "dsa_router_logits_workspace: bytes is NULL");
    int rc = check_logits("dsa_router_logits_workspace", rows, hidden, n);
    if (rc) return rc;
    const int sms = sm_count();
    if (sms <= 0) return fail(DSA_ERR_CUDA, "dsa_router_logits_workspace: no CUDA device");
    *bytes = project_workspace_bytes(rows, hidden, n, sms);
    return DSA_OK;
}

extern "C" int dsa_router_logits(const dsa_bf16* x, int rows, int hidden, const dsa_bf16* w, int n,
                                 float* logits, int32_t* status, void* workspace,
                                 size_t workspace_bytes, void* stream) {
    int rc = check_logits("dsa_router_logits", rows, hidden, n);
    if (rc) return rc;
    if (rows == 0) return DSA_OK;
    if (!x || !w || !logits) return fail(DSA_ERR_INVALID_ARG, "dsa_router_logits: NULL tensor");
    if ((((uintptr_t)x) | ((uintptr_t)w) | ((uintptr_t)logits) | ((uintptr_t)workspace)) & 15)
        return fail(DSA_ERR_INVALID_ARG, "dsa_router_logits: tensors must be 16-byte aligned");
    const int sms = sm_count();
    if (sms <= 0) return fail(DSA_ERR_CUDA, "dsa_router_logits: no CUDA device");
    const size_t need = project_workspace_bytes(rows, hidden, n, sms);
    if (need && (!workspace || workspace_bytes < need))
        return fail(DSA_ERR_INVALID_ARG, "dsa_router_logits: workspace %zu B < %zu B needed",
                    workspace_bytes, need);
    return project_launch(x, false, rows, hidden, w, n, nullptr, status, workspace, workspace_bytes,
                          (cudaStream_t)stream, logits);
}
