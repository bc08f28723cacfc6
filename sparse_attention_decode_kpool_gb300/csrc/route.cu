// dsa_route: a router's scores to the chosen experts and their weights.
// dsa_router_logits: the logits, x . w^T with f32 results (the projection of project.cu).
//
//   s_e = sigmoid(logit_e) or softmax(logits)_e        c_e = s_e + bias_e
//   groups: the topk_group groups whose group_top best c have the largest sum
//   experts: the topk largest c among those groups, ties to the lowest id, written in
//   ascending id; weight = s_e (over the sum of the chosen s when renorm) * scale
//
// One warp per row; expert e is lane e % 32's piece e / 32. Rows are few or short (a
// thousand bytes), so latency and instructions bound it, not memory: the best expert of
// a round is two warp reductions (the largest key, then the lowest id that has it), and
// only the lane that held it looks for its next best.
//
// The choice is the one that 64-bit arithmetic makes. It is first made in f32; every c
// computed so is within err of the exact one (err below), so where the smallest chosen
// and the largest rejected value (of experts, or of groups) are further apart than the
// errors of both, the f32 choice is final. Else, about one row in a thousand for
// unrelated scores, the warp repeats the row in f64. (f64 throughout would take about 30
// times the arithmetic on this part's few FP64 units.)
#include "common.cuh"

namespace dsa {
namespace {

constexpr int kRouteWarps = 4;
constexpr uint32_t kAll = 0xffffffffu;

struct RouteArgs {
    const float* logits;
    const float* bias;  // nullable
    int32_t* ids;
    float* weights;
    long long ld;
    int rows, n, groups, gsize, topk_group, group_top, topk, shared;
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
__device__ __forceinline__ double warp_max_t(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmax(v, __shfl_xor_sync(kAll, v, o));
    return v;
}
template <typename T>
__device__ __forceinline__ T warp_sum_t(T v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// One row in T's arithmetic. logit[] holds the lane's pieces (-inf past the last expert).
// Gives the chosen pieces (bit i of `taken`), their scores s[] and whether the row holds a
// NaN; returns false when T is float and the choice, or the renormalising sum, is not
// certain. buf: the warp's staging area, 33 T per piece.
template <typename T, int NPL>
__device__ bool choose(const RouteArgs& a, const float (&logit)[NPL], int lane, T* buf, T (&s)[NPL],
                       uint32_t& taken, bool& nan) {
    const T NI = neg_inf<T>();
    T c[NPL];
    bool bad = false;
    T top = NI;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        T z = (T)logit[i];
        if (!(z == z) || (a.softmax && z > (T)3.4028235e38)) {
            bad = true;
            z = NI;
        }
        s[i] = z;
        top = z > top ? z : top;
    }
    top = warp_max_t(top);
    T sum = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const T z = s[i];
        c[i] = z;  // the logit, until its score is known
        if (a.softmax) {
            s[i] = z > NI ? exp_t(z - top) : (T)0;
            sum += s[i];
        } else {
            s[i] = z > NI ? (T)1 / ((T)1 + exp_t(-z)) : (T)0;
        }
    }
    if (a.softmax) {
        sum = warp_sum_t(sum);
        const T inv = sum > 0 ? (T)1 / sum : (T)0;
#pragma unroll
        for (int i = 0; i < NPL; ++i) s[i] *= inv;
    }
    T smax = 0, bmax = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = lane + 32 * i;
        T b = 0;
        if (a.bias && e < a.n) b = (T)__ldg(a.bias + e);
        if (!(b == b)) {
            bad = true;
            c[i] = NI;
        }
        const bool cand = e < a.n && c[i] > NI;
        smax = cand && s[i] > smax ? s[i] : smax;
        const T ab = b < 0 ? -b : b;
        bmax = cand && ab > bmax && ab < (T)1e30 ? ab : bmax;
        c[i] = cand ? s[i] + b : NI;
    }
    nan = __any_sync(kAll, bad);
    // |computed c - exact c|: the score's few roundings (2^-19 of the largest leaves room
    // for the softmax's sum) and the bias's addition.
    T err = 0;
    if constexpr (sizeof(T) == 4)
        err = 1.9073486e-6f * warp_max_t(smax) + 1.2e-7f * warp_max_t(bmax) + 1e-37f;
    bool sure = true;

    if (a.groups > 1) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < NPL; ++i) buf[33 * i + lane] = c[i];
        __syncwarp();
        // 32 / groups (rounded down to a power of two) lanes scan one group
        int per = 32;
        while (per * a.groups > 32) per >>= 1;
        const int g = lane / per, j0 = lane % per;
        T b1 = NI, b2 = NI;
        if (g < a.groups) {
            for (int j = j0; j < a.gsize; j += per) {
                const int e = g * a.gsize + j;
                const T v = buf[33 * (e >> 5) + (e & 31)];
                b2 = v > b1 ? b1 : (v > b2 ? v : b2);
                b1 = v > b1 ? v : b1;
            }
        }
        for (int o = per >> 1; o > 0; o >>= 1) {
            const T o1 = __shfl_xor_sync(kAll, b1, o), o2 = __shfl_xor_sync(kAll, b2, o);
            const T lo = o1 > b1 ? b1 : o1;
            b1 = o1 > b1 ? o1 : b1;
            b2 = b2 > o2 ? b2 : o2;
            b2 = lo > b2 ? lo : b2;
        }
        T score = b1;
        if (a.group_top == 2 && b2 > NI) score += b2;
        const bool lead = g < a.groups && j0 == 0;
        if (!lead) score = NI;
        uint32_t kept = 0;
        T low = 0;
        for (int k = 0; k < a.topk_group; ++k) {
            const T m = warp_max_t((kept >> g) & 1u ? NI : score);
            if (!(m > NI)) break;
            const int id = (int)__reduce_min_sync(
                kAll, lead && !((kept >> g) & 1u) && score == m ? (uint32_t)g : 64u);
            kept |= 1u << id;
            low = m;
        }
        if constexpr (sizeof(T) == 4) {
            const T next = warp_max_t((kept >> g) & 1u ? NI : score);
            if (next > NI && !(low - next > 4 * err)) sure = false;
        }
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = lane + 32 * i;
            if (e < a.n && !((kept >> (e / a.gsize)) & 1u)) c[i] = NI;
        }
    }

    // the topk best, one after the other
    taken = 0;
    T best = NI;
    int at = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i)
        if (c[i] > best) {
            best = c[i];
            at = i;
        }
    T low = 0;
    for (int k = 0; k < a.topk; ++k) {
        const T m = warp_max_t(best);
        if (!(m > NI)) break;
        const uint32_t id = __reduce_min_sync(kAll, best == m ? (uint32_t)(lane + 32 * at) : 0xffffffffu);
        low = m;
        if ((id & 31u) == (uint32_t)lane) {
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
    if constexpr (sizeof(T) == 4) {
        const T next = warp_max_t(best);
        if (next > NI && !(low - next > 2 * err)) sure = false;
    }
    return sure;
}

template <int NPL>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(RouteArgs a) {
    __shared__ double stage[kRouteWarps][33 * NPL];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long r = (long long)blockIdx.x * kRouteWarps + warp;
    pdl_wait();
    if (r >= a.rows) return;
    const float* row = a.logits + r * a.ld;
    float logit[NPL], s[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = lane + 32 * i;
        logit[i] = e < a.n ? __ldg(row + e) : neg_inf<float>();
    }
    uint32_t taken;
    bool nan;
    bool sure = choose<float, NPL>(a, logit, lane, reinterpret_cast<float*>(stage[warp]), s, taken, nan);
    float total = 0.f;
    bool tiny = false;  // near f32's smallest: digits are lost that a ratio of scores needs
#pragma unroll
    for (int i = 0; i < NPL; ++i)
        if ((taken >> i) & 1u) {
            total += s[i];
            tiny |= s[i] < 1e-30f;
        }
    total = warp_sum_t(total);
    if (!sure || (a.renorm && __any_sync(kAll, tiny))) {
        double sd[NPL], td = 0;
        choose<double, NPL>(a, logit, lane, stage[warp], sd, taken, nan);
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            if ((taken >> i) & 1u) td += sd[i];
        td = warp_sum_t(td);
        const double inv = a.renorm ? (td > 0 ? 1.0 / td : 0.0) : 1.0;
#pragma unroll
        for (int i = 0; i < NPL; ++i) s[i] = (float)(sd[i] * inv);
        total = 1.f;
    }
    const float f = a.renorm ? (total > 0.f ? a.scale / total : 0.f) : a.scale;
    const int width = a.topk + a.shared;
    int32_t* ids = a.ids + r * width;
    float* weights = a.weights + r * width;
    int n = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const bool mine = (taken >> i) & 1u;
        const uint32_t who = __ballot_sync(kAll, mine);
        if (mine) {
            const int at = n + __popc(who & ((1u << lane) - 1u));
            ids[at] = lane + 32 * i;
            weights[at] = nan ? __uint_as_float(0x7fc00000u) : s[i] * f;
        }
        n += __popc(who);
    }
    for (int k = n + lane; k < width; k += 32) {
        const bool extra = k >= a.topk;
        ids[k] = extra ? a.n + (k - a.topk) : -1;
        weights[k] = extra ? 1.f : 0.f;
    }
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
    a.topk_group = topk_group;
    a.group_top = group_top;
    a.topk = topk;
    a.shared = shared;
    a.softmax = score == DSA_ROUTE_SOFTMAX;
    a.renorm = renorm != 0;
    a.scale = scale;
    const dim3 grid((unsigned)((rows + kRouteWarps - 1) / kRouteWarps)), block(kRouteWarps * 32);
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e;
    if (n_experts <= 64)
        e = launch_pdl(route_kernel<2>, grid, block, 0, st, a);
    else if (n_experts <= 128)
        e = launch_pdl(route_kernel<4>, grid, block, 0, st, a);
    else if (n_experts <= 256)
        e = launch_pdl(route_kernel<8>, grid, block, 0, st, a);
    else if (n_experts <= 512)
        e = launch_pdl(route_kernel<16>, grid, block, 0, st, a);
    else
        e = launch_pdl(route_kernel<32>, grid, block, 0, st, a);
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
