// dsa_quantize_latent: the FP8 latent cache's encoder; dsa_dequantize_latent: its rows
// back as bf16.
//
// Format (the layer's stated choice; mod.rs names the FP8 decode kernel,
// glm5next_dsa_mla_decode_fp8, and nothing of its format): OCP E4M3 codes with one
// power-of-two scale 2^k per token and 128-channel group, k the smallest integer with
// amax <= 448 * 2^k (not below -126; 0 for an all-zero group). Dividing by 2^k is
// exact, so the only rounding is the E4M3 conversion (nearest, ties to even), and a
// decoded value (code times 2^k) is exact in bf16.
//
// One warp per latent row; for each 128-channel group every lane takes 4 channels,
// the group's largest magnitude comes from a warp max, and the scale exponent from
// its float bits (fp8.cuh).
#include "fp8.cuh"

namespace dsa {
namespace {

constexpr int kQuantWarps = 8;

__global__ void __launch_bounds__(kQuantWarps * 32) quantize_latent_kernel(
    const uint16_t* __restrict__ x, long long rows, int kvl, uint8_t* __restrict__ codes,
    float* __restrict__ scales) {
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long r = (long long)blockIdx.x * kQuantWarps + (threadIdx.x >> 5);
    if (r >= rows) return;
    const int G = kvl / 128;
    for (int gi = 0; gi < G; ++gi)
        fp8_encode_group(x + r * kvl + gi * 128, codes + r * kvl + gi * 128, scales + r * G + gi, lane);
}

// 16 codes per piece (they lie in one group), PER pieces a thread, a block's pieces
// consecutive so that loads and stores are whole lines. All loads are requested before the
// first is used. Bound by memory: 4,096 rows of 4,096 channels (50 MB) in 10 us. PER is 1, or 4 for
// named rows from 16 x 2,048 pieces an SM on, where the lookups of several rows go at once. Measured
// with a cold L2, rows of 4,096 channels, 1 | 4 a thread: in order 16,384 rows 37 | 41 us, 32,768
// 70 | 72, 131,072 254 | 254; named 16,384 rows 41 | 41, 65,536 143 | 133, 131,072 279 | 258.
constexpr int kDequantThreads = 256;
template <int PER>
__global__ void __launch_bounds__(kDequantThreads) dequantize_latent_kernel(
    const uint4* __restrict__ codes, const float* __restrict__ scales,
    const int32_t* __restrict__ rows, long long pieces, int per_row, long long cache_rows,
    uint4* __restrict__ out, int32_t* status) {
    pdl_wait();
    const long long i0 = (long long)blockIdx.x * (kDequantThreads * PER) + threadIdx.x;
    uint4 c[PER];
    float sc[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const long long i = i0 + k * kDequantThreads;
        c[k] = make_uint4(0, 0, 0, 0);
        sc[k] = 0.f;
        long long src = i;
        if (rows && i < pieces) {
            const long long r = i / per_row;
            const int cr = rows[r];
            src = cr >= 0 && cr < cache_rows ? (long long)cr * per_row + (i - r * per_row) : -1;
            if (src < 0 && i == r * per_row) flag_status(status, DSA_STATUS_BAD_TOKEN);
        }
        if (i < pieces && src >= 0) {
            c[k] = ldg16_stream(codes + src);
            sc[k] = __ldg(scales + (src >> 3));  // per_row is a multiple of 8
        }
    }
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const long long i = i0 + k * kDequantThreads;
        if (i >= pieces) return;
        const uint32_t w[4] = {c[k].x, c[k].y, c[k].z, c[k].w};
        uint32_t o[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            o[2 * j] = e4m3x2_to_bf16x2(w[j] & 0xffffu, sc[k]);
            o[2 * j + 1] = e4m3x2_to_bf16x2(w[j] >> 16, sc[k]);
        }
        out[2 * i] = make_uint4(o[0], o[1], o[2], o[3]);
        out[2 * i + 1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" int dsa_quantize_latent(const dsa_bf16* x, long long rows, int kv_lora_rank,
                                   uint8_t* codes, float* scales, void* stream) {
    if (rows < 0 || kv_lora_rank < 128 || kv_lora_rank % 128 != 0)
        return fail(DSA_ERR_INVALID_ARG, "dsa_quantize_latent: rows %lld, kv_lora_rank %d",
                    rows, kv_lora_rank);
    if (rows == 0) return DSA_OK;
    if (!x || !codes || !scales) return fail(DSA_ERR_INVALID_ARG, "dsa_quantize_latent: NULL tensor");
    if ((((uintptr_t)x) | ((uintptr_t)codes) | ((uintptr_t)scales)) & 15)
        return fail(DSA_ERR_INVALID_ARG, "dsa_quantize_latent: tensors must be 16-byte aligned");
    const long long blocks = (rows + kQuantWarps - 1) / kQuantWarps;
    if (blocks > 0x7fffffffLL) return fail(DSA_ERR_UNSUPPORTED, "dsa_quantize_latent: too many rows");
    cudaError_t e = launch_pdl(quantize_latent_kernel, dim3((unsigned)blocks), dim3(kQuantWarps * 32),
                               0, (cudaStream_t)stream, (const uint16_t*)x, rows, kv_lora_rank,
                               codes, scales);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "dsa_quantize_latent launch");
    return DSA_OK;
}

extern "C" int dsa_dequantize_latent(const uint8_t* codes, const float* scales,
                                     long long cache_rows, const int32_t* row_ids, long long rows,
                                     int kv_lora_rank, dsa_bf16* out, int32_t* status,
                                     void* stream) {
    if (rows < 0 || cache_rows < 0 || kv_lora_rank < 128 || kv_lora_rank % 128 != 0)
        return fail(DSA_ERR_INVALID_ARG,
                    "dsa_dequantize_latent: rows %lld, cache_rows %lld, kv_lora_rank %d", rows,
                    cache_rows, kv_lora_rank);
    if (!row_ids && rows > cache_rows)
        return fail(DSA_ERR_INVALID_ARG, "dsa_dequantize_latent: %lld rows of a cache of %lld", rows,
                    cache_rows);
    if (rows == 0) return DSA_OK;
    if (!codes || !scales || !out)
        return fail(DSA_ERR_INVALID_ARG, "dsa_dequantize_latent: NULL tensor");
    if ((((uintptr_t)codes) | ((uintptr_t)out)) & 15 || ((uintptr_t)scales) & 3 ||
        ((uintptr_t)row_ids) & 3)
        return fail(DSA_ERR_INVALID_ARG, "dsa_dequantize_latent: codes and out must be 16-byte aligned");
    const int per_row = kv_lora_rank / 16;
    if (rows > 0x7fffffffLL || rows * per_row > 0x7fffffffLL * kDequantThreads)
        return fail(DSA_ERR_UNSUPPORTED, "dsa_dequantize_latent: too many rows");
    const long long pieces = rows * per_row;
    const int sms = sm_count();
    const bool many = row_ids && pieces >= 16LL * 2048 * (sms > 0 ? sms : 152);
    const long long per = kDequantThreads * (many ? 4 : 1);
    cudaError_t e = launch_pdl(many ? dequantize_latent_kernel<4> : dequantize_latent_kernel<1>,
                               dim3((unsigned)((pieces + per - 1) / per)), dim3(kDequantThreads), 0,
                               (cudaStream_t)stream, (const uint4*)codes, scales, row_ids, pieces,
                               per_row, cache_rows, (uint4*)out, status);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "dsa_dequantize_latent launch");
    return DSA_OK;
}
