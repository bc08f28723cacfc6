// dsa_rmsnorm: the residual stream's addition and the RMS norm behind it, in one pass.
//
//   v = x + residual (f32)            residual_out = bf16(v)
//   out = bf16(v / sqrt(mean(v^2) + eps) * weight)
//   codes, scales = the FP8 rows of out (the codec of fp8.cuh, on the bf16 values)
//
// Bound by memory for many rows and by latency for few. Each row is read once: a thread
// keeps its eight-channel pieces in registers between the sum of squares and the
// output (rms_vec_kernel); rows whose width is no multiple of 8, or too wide for that, are
// read twice (rms_any_kernel). The mean is of the unrounded sum v, so the residual's
// rounding to bf16 does not enter the norm. An FP8 group is 16 lanes of one warp.
//
// The sum of squares, the root and the products carry their rounding errors along in a second
// f32 (the standard error-free transformations by fused multiply-add), so that out is the
// formula's value rounded to f32 and then to bf16: in plain f32 one value in some 100,000 comes
// out one bf16 step off, and its FP8 code with it one step of 2^-3. It costs 4,096 rows of 4,096
// with residual and FP8 rows 31 us instead of 27 (their 151 MB: 23 us at the copy rate). Measured
// there: 8 warps a row and two pieces a thread 31.8 us, 4 and four 33.0, 16 and one 35 (with the
// plain sums); the weights requested with the row 33.5 (registers, so fewer blocks an SM), though
// 8 rows take 3.2 us with that instead of 3.5.
#include "fp8.cuh"

namespace dsa {
namespace {

struct RmsArgs {
    const uint16_t* x;
    const uint16_t* residual;  // nullable
    const uint16_t* weight;
    uint16_t* residual_out;  // nullable
    uint16_t* out;           // nullable
    uint8_t* codes;          // nullable, with scales
    float* scales;
    long long rows;
    int width;
    float inv_width;  // 1 / width
    float eps;
};

// A sum of squares and its rounding errors.
struct Squares {
    float s, c;
};
__device__ __forceinline__ void add_square(Squares& a, float v) {
    const float t = fmaf(v, v, a.s);
    a.c += fmaf(v, v, a.s - t);
    a.s = t;
}
__device__ __forceinline__ Squares add_squares(const Squares& a, const Squares& b) {
    const float t = a.s + b.s, u = t - a.s;
    return {t, a.c + b.c + ((a.s - (t - u)) + (b.s - u))};
}
__device__ __forceinline__ Squares warp_squares(Squares a) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        a = add_squares(a, {__shfl_xor_sync(0xffffffffu, a.s, o), __shfl_xor_sync(0xffffffffu, a.c, o)});
    return a;
}
// 1 / sqrt(mean + eps) as hi + lo: one Newton step on the root of the leading part.
struct Root {
    float hi, lo;
};
__device__ __forceinline__ Root root_of(const Squares& a, float n, float inv_n, float eps) {
    const float q = a.s * inv_n;  // near a.s / n; the rest of it is in `low`
    const float m = q + eps, u = m - q;
    const float low = fmaf(fmaf(-q, n, a.s) + a.c, inv_n, (q - (m - u)) + (eps - u));
    const float r = rsqrtf(m), t = r * r;
    const float e = fmaf(low, t, fmaf(m, fmaf(r, r, -t), fmaf(m, t, -1.f)));
    return {r, m > 0.f && m < __uint_as_float(0x7f800000u) ? -0.5f * r * e : 0.f};
}
// v * root * w, rounded once.
__device__ __forceinline__ float normed(float v, const Root& r, float w) {
    const float h = v * r.hi, l = fmaf(v, r.lo, fmaf(v, r.hi, -h));
    const float p = h * w;
    return fabsf(p) < __uint_as_float(0x7f800000u) ? p + fmaf(l, w, fmaf(h, w, -p)) : p;
}

__device__ __forceinline__ void team_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(threads) : "memory");
}

// Below this mean of squares (eps included) f32 runs out of digits and then of range for the squares
// and the root: such a row, every value below 2^-36 (width <= 2^24), is multiplied by 2^96 and its eps by
// 2^192, which leaves the result as it is. (The root of a mean above 2^-96 squared is below 2^96.)
constexpr float kSmallMean = 1.262177448e-29f;  // 2^-96
constexpr float kRaise = 7.922816251e28f;       // 2^96
__device__ __forceinline__ bool small_row(const Squares& a, float inv_n, float eps) {
    return fmaf(a.s, inv_n, eps) < kSmallMean;
}

// WPR warps per row, 8 / WPR rows per 256-thread block (WPR <= 8), or one row per block of
// WPR warps; V pieces of eight channels per thread.
template <int WPR, int V>
__global__ void __launch_bounds__(WPR >= 8 ? WPR * 32 : 256) rms_vec_kernel(RmsArgs a) {
    constexpr int ROWS = WPR >= 8 ? 1 : 8 / WPR;
    __shared__ Squares red[WPR * ROWS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int team = warp / WPR;
    const long long r = (long long)blockIdx.x * ROWS + team;
    const int t = threadIdx.x - team * WPR * 32;
    const int nvec = a.width >> 3;
    const bool row_ok = r < a.rows;
    const long long base = r * a.width;
    pdl_wait();
    float v[V][8];
    Squares ss = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int p = t + k * WPR * 32;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[k][j] = 0.f;
        if (row_ok && p < nvec) {
            const uint4 q = *reinterpret_cast<const uint4*>(a.x + base + p * 8);
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[k][2 * j] = bf16_lo(w[j]);
                v[k][2 * j + 1] = bf16_hi(w[j]);
            }
        }
    }
    if (a.residual) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int p = t + k * WPR * 32;
            if (row_ok && p < nvec) {
                const uint4 q = *reinterpret_cast<const uint4*>(a.residual + base + p * 8);
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[k][2 * j] += bf16_lo(w[j]);
                    v[k][2 * j + 1] += bf16_hi(w[j]);
                }
            }
        }
    }
#pragma unroll
    for (int k = 0; k < V; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) add_square(ss, v[k][j]);
    ss = warp_squares(ss);
    if constexpr (WPR > 1) {
        if (lane == 0) red[warp] = ss;
        __syncthreads();
        ss = red[team * WPR];
#pragma unroll 4
        for (int i = 1; i < WPR; ++i) ss = add_squares(ss, red[team * WPR + i]);
    }
    if (!row_ok) return;
    if (a.residual_out) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int p = t + k * WPR * 32;
            if (p >= nvec) continue;
            uint4 q;
            q.x = pack_bf16x2(v[k][0], v[k][1]);
            q.y = pack_bf16x2(v[k][2], v[k][3]);
            q.z = pack_bf16x2(v[k][4], v[k][5]);
            q.w = pack_bf16x2(v[k][6], v[k][7]);
            *reinterpret_cast<uint4*>(a.residual_out + base + p * 8) = q;
        }
    }
    float eps = a.eps;
    if (small_row(ss, a.inv_width, eps)) {  // (the whole row's warps alike)
        ss = {0.f, 0.f};
        eps = eps * kRaise * kRaise;
#pragma unroll
        for (int k = 0; k < V; ++k) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[k][j] *= kRaise;
                add_square(ss, v[k][j]);
            }
        }
        ss = warp_squares(ss);
        if constexpr (WPR > 1) {
            team_sync(1 + team, WPR * 32);  // the first sums are read
            if (lane == 0) red[warp] = ss;
            team_sync(1 + team, WPR * 32);
            ss = red[team * WPR];
            for (int i = 1; i < WPR; ++i) ss = add_squares(ss, red[team * WPR + i]);
        }
    }
    const Root rs = root_of(ss, (float)a.width, a.inv_width, eps);
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int p = t + k * WPR * 32;
        // With codes the width is a multiple of 128, so the 16 lanes of a group are all
        // inside the row or all outside.
        if (p >= nvec) continue;
        const uint4 wq = ldg16(a.weight + p * 8);
        const uint32_t w[4] = {wq.x, wq.y, wq.z, wq.w};
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            o[j] = pack_bf16x2(normed(v[k][2 * j], rs, bf16_lo(w[j])), normed(v[k][2 * j + 1], rs, bf16_hi(w[j])));
        if (a.out) *reinterpret_cast<uint4*>(a.out + base + p * 8) = make_uint4(o[0], o[1], o[2], o[3]);
        if (a.codes) {
            float f[8], m = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f[2 * j] = bf16_lo(o[j]);
                f[2 * j + 1] = bf16_hi(o[j]);
                m = fmaxf(m, fmaxf(fabsf(f[2 * j]), fabsf(f[2 * j + 1])));
            }
            const uint32_t half = 0xffffu << (lane & 16);
#pragma unroll
            for (int s = 8; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(half, m, s));
            const int e = fp8_scale_exp(m);
            const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
            uint2 c;
            c.x = e4m3x2(f[0] * inv, f[1] * inv) | (e4m3x2(f[2] * inv, f[3] * inv) << 16);
            c.y = e4m3x2(f[4] * inv, f[5] * inv) | (e4m3x2(f[6] * inv, f[7] * inv) << 16);
            *reinterpret_cast<uint2*>(a.codes + base + p * 8) = c;
            if ((lane & 15) == 0)
                a.scales[r * (a.width >> 7) + (p >> 4)] = __uint_as_float((uint32_t)(e + 127) << 23);
        }
    }
}

// Any width: one block per row, the row read twice (the second time from L1 or L2; a small row thrice). The
// element a thread reads is the element it writes, so outputs may be the inputs.
constexpr int kAnyThreads = 512;
__global__ void __launch_bounds__(kAnyThreads) rms_any_kernel(RmsArgs a) {
    __shared__ Squares red[kAnyThreads / 32];
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long r = blockIdx.x, base = r * a.width;
    float up = 1.f, eps = a.eps;
    Squares ss;
    for (int turn = 0; turn < 2; ++turn) {
        ss = {0.f, 0.f};
        for (int c = threadIdx.x; c < a.width; c += kAnyThreads) {
            float v = bf16_lo(a.x[base + c]);
            if (a.residual) v += bf16_lo(a.residual[base + c]);
            add_square(ss, v * up);
        }
        ss = warp_squares(ss);
        if (turn) __syncthreads();  // the first sums are read
        if (lane == 0) red[warp] = ss;
        __syncthreads();
        ss = red[0];
        for (int i = 1; i < kAnyThreads / 32; ++i) ss = add_squares(ss, red[i]);
        if (turn || !small_row(ss, a.inv_width, eps)) break;
        up = kRaise;
        eps = eps * kRaise * kRaise;
    }
    const Root rs = root_of(ss, (float)a.width, a.inv_width, eps);
    // a group of 128 channels is a warp's turn of four channels a lane
    for (int c0 = warp * 128; c0 < a.width; c0 += kAnyThreads * 4) {
        float f[4], m = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = c0 + j * 32 + lane;
            f[j] = 0.f;
            if (c < a.width) {
                float v = bf16_lo(a.x[base + c]);
                if (a.residual) v += bf16_lo(a.residual[base + c]);
                f[j] = round_bf16(normed(v * up, rs, bf16_lo(a.weight[c])));
                if (a.residual_out)
                    a.residual_out[base + c] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
                if (a.out) a.out[base + c] = __bfloat16_as_ushort(__float2bfloat16_rn(f[j]));
            }
            m = fmaxf(m, fabsf(f[j]));
        }
        if (a.codes) {
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
            const int e = fp8_scale_exp(m);
            const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                a.codes[base + c0 + j * 32 + lane] = (uint8_t)(e4m3x2(f[j] * inv, 0.f) & 0xffu);
            if (lane == 0)
                a.scales[r * (a.width >> 7) + (c0 >> 7)] = __uint_as_float((uint32_t)(e + 127) << 23);
        }
    }
}

template <int WPR, int V>
cudaError_t rms_launch(const RmsArgs& a, cudaStream_t st) {
    constexpr int ROWS = WPR >= 8 ? 1 : 8 / WPR;
    return launch_pdl(rms_vec_kernel<WPR, V>, dim3((unsigned)((a.rows + ROWS - 1) / ROWS)),
                      dim3(WPR >= 8 ? WPR * 32 : 256), 0, st, a);
}

struct Range {
    const void* p;
    size_t n;
};
bool overlap(const Range& a, const Range& b) {
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return a.p && b.p && x < y + b.n && y < x + a.n;
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" int dsa_rmsnorm(const dsa_bf16* x, const dsa_bf16* residual, const dsa_bf16* weight,
                           long long rows, int width, float eps, dsa_bf16* residual_out,
                           dsa_bf16* out, uint8_t* codes, float* scales, void* stream) {
    if (rows < 0 || width < 1)
        return fail(DSA_ERR_INVALID_ARG, "dsa_rmsnorm: rows %lld, width %d", rows, width);
    if (!(eps >= 0.f)) return fail(DSA_ERR_INVALID_ARG, "dsa_rmsnorm: eps must be >= 0");
    if (codes && width % 128 != 0)
        return fail(DSA_ERR_UNSUPPORTED, "dsa_rmsnorm: FP8 rows need a width of a multiple of 128, not %d",
                    width);
    if (rows > 0x7fffffffLL || width > (1 << 24))
        return fail(DSA_ERR_UNSUPPORTED, "dsa_rmsnorm: at most 2^31 - 1 rows of 2^24 channels");
    if (rows == 0) return DSA_OK;  // (tensors without elements have no address)
    if ((codes != nullptr) != (scales != nullptr))
        return fail(DSA_ERR_INVALID_ARG, "dsa_rmsnorm: codes and scales go together");
    if (!out && !codes) return fail(DSA_ERR_INVALID_ARG, "dsa_rmsnorm: neither out nor codes");
    if (residual_out && !residual)
        return fail(DSA_ERR_INVALID_ARG, "dsa_rmsnorm: residual_out without residual");
    if (!x || !weight) return fail(DSA_ERR_INVALID_ARG, "dsa_rmsnorm: NULL tensor");
    if (((uintptr_t)scales) & 3) return fail(DSA_ERR_INVALID_ARG, "dsa_rmsnorm: scales misaligned");
    const size_t n = (size_t)rows * width;
    const Range in[3] = {{x, 2 * n}, {residual, 2 * n}, {weight, 2 * (size_t)width}};
    const Range to[4] = {{residual_out, 2 * n}, {out, 2 * n}, {codes, n}, {scales, n / 128 * 4}};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 3; ++j)
            if (overlap(to[i], in[j]) && !(i < 2 && j < 2 && to[i].p == in[j].p))
                return fail(DSA_ERR_INVALID_ARG,
                            "dsa_rmsnorm: an output overlaps an input (residual_out and out may each "
                            "be x or residual, exactly)");
        for (int j = 0; j < i; ++j)
            if (overlap(to[i], to[j]))
                return fail(DSA_ERR_INVALID_ARG, "dsa_rmsnorm: two outputs overlap");
    }
    RmsArgs a;
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.residual_out = residual_out;
    a.out = out;
    a.codes = codes;
    a.scales = scales;
    a.rows = rows;
    a.width = width;
    a.inv_width = 1.f / (float)width;
    a.eps = eps;
    const bool aligned = ((((uintptr_t)x) | ((uintptr_t)residual) | ((uintptr_t)weight) |
                           ((uintptr_t)residual_out) | ((uintptr_t)out)) & 15) == 0 &&
                         (((uintptr_t)codes) & 7) == 0;
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e;
    const int nvec = width / 8;
    if (!aligned || width % 8 != 0 || nvec > 4096)
        e = launch_pdl(rms_any_kernel, dim3((unsigned)rows), dim3(kAnyThreads), 0, st, a);
    else if (nvec <= 32)
        e = rms_launch<1, 1>(a, st);
    else if (nvec <= 64)
        e = rms_launch<1, 2>(a, st);
    else if (nvec <= 128)
        e = rms_launch<2, 2>(a, st);
    else if (nvec <= 256)
        e = rms_launch<4, 2>(a, st);
    else if (nvec <= 512)
        e = rms_launch<8, 2>(a, st);
    else if (nvec <= 1024)
        e = rms_launch<16, 2>(a, st);
    else if (nvec <= 2048)
        e = rms_launch<32, 2>(a, st);
    else
        e = rms_launch<32, 4>(a, st);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "dsa_rmsnorm launch");
    return DSA_OK;
}
