// dsa_quantize_latent_fp4 and dsa_dequantize_latent_fp4: rows into the FP4 latent cache
// and out of it again (format and rounding in fp4.cuh).
//
// Both are streams: a token's rows are independent 16-channel blocks, so a thread takes
// one block (32 bytes of bf16, 8 bytes of codes, one scale byte) and a warp 512
// channels; a block's maximum needs no exchange between threads.
#include "fp4.cuh"

namespace dsa {
namespace {

constexpr int kF4Threads = 256;

// PER blocks per thread, kF4Threads apart: with 4, 128 bytes of loads under way per thread
// (524,283 rows there and back 221 us, with 1 234); with 1, enough thread blocks for the
// GPU where there is little to do (4,096 rows 4.0 us, with 4 4.6).
template <int PER>
__global__ void __launch_bounds__(kF4Threads) quantize_latent_fp4_kernel(
    const uint4* __restrict__ x, long long blocks, int cache_exp, uint2* __restrict__ codes,
    uint8_t* __restrict__ scales) {
    pdl_wait();
    const long long i0 = (long long)blockIdx.x * (kF4Threads * PER) + threadIdx.x;
    uint4 v[PER][2];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const long long i = i0 + k * kF4Threads;
        if (i < blocks) {
            v[k][0] = ldg16_stream(x + 2 * i);
            v[k][1] = ldg16_stream(x + 2 * i + 1);
        }
    }
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const long long i = i0 + k * kF4Threads;
        if (i >= blocks) return;
        uint8_t s;
        codes[i] = fp4_encode16(v[k], cache_exp, &s);
        scales[i] = s;
    }
}

// out row i = cache row rows[i] (rows NULL: row i); a row outside [0, cache_rows) gives
// zeros and flags DSA_STATUS_BAD_TOKEN.
template <int PER>
__global__ void __launch_bounds__(kF4Threads) dequantize_latent_fp4_kernel(
    const uint2* __restrict__ codes, const uint8_t* __restrict__ scales,
    const int32_t* __restrict__ rows, long long blocks, int per_row, long long cache_rows,
    int cache_exp, uint4* __restrict__ out, int32_t* status) {
    pdl_wait();
    const long long i0 = (long long)blockIdx.x * (kF4Threads * PER) + threadIdx.x;
    uint2 c[PER];
    uint32_t sc[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const long long i = i0 + k * kF4Threads;
        long long src = i;
        c[k] = make_uint2(0u, 0u);
        sc[k] = 0;
        if (i < blocks && rows) {
            const long long r = i / per_row;
            const int cr = rows[r];
            src = cr >= 0 && cr < cache_rows ? (long long)cr * per_row + (i - r * per_row) : -1;
            if (src < 0 && i == r * per_row) flag_status(status, DSA_STATUS_BAD_TOKEN);
        }
        if (i < blocks && src >= 0) {
            c[k] = codes[src];
            sc[k] = scales[src];
        }
    }
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const long long i = i0 + k * kF4Threads;
        if (i >= blocks) return;
        const uint32_t sh = e4m3x2_to_f16x2(sc[k]);
        const float s =
            __half2float(__ushort_as_half((unsigned short)(sh & 0xffffu))) * pow2f(cache_exp);
        const uint32_t cw[2] = {c[k].x, c[k].y};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t h[4], o[4];
            e2m1x8_to_f16x8(h, cw[j]);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[p]));
                o[p] = pack_bf16x2(f.x * s, f.y * s);  // exact
            }
            out[2 * i + j] = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

// Whether four blocks per thread still leave every SM its 2,048 threads four times over.
bool many_blocks(long long blocks) {
    const int sms = sm_count();
    return blocks >= 16LL * 2048 * (sms > 0 ? sms : 152);
}

int check_fp4(const char* name, long long rows, int kvl, int cache_exp) {
    if (rows < 0 || kvl < kF4Block || kvl % kF4Block != 0)
        return fail(DSA_ERR_INVALID_ARG, "%s: rows %lld, kv_lora_rank %d (a multiple of %d)", name,
                    rows, kvl, kF4Block);
    if (cache_exp < -kF4MaxExp || cache_exp > kF4MaxExp)
        return fail(DSA_ERR_INVALID_ARG, "%s: cache_exp %d outside [-%d, %d]", name, cache_exp,
                    kF4MaxExp, kF4MaxExp);
    if (rows > 0x7fffffffLL || rows * (kvl / kF4Block) > 0x7fffffffLL * kF4Threads)
        return fail(DSA_ERR_UNSUPPORTED, "%s: too many rows", name);
    return DSA_OK;
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" int dsa_quantize_latent_fp4(const dsa_bf16* x, long long rows, int kv_lora_rank,
                                       int cache_exp, uint8_t* codes, uint8_t* scales,
                                       void* stream) {
    int rc = check_fp4("dsa_quantize_latent_fp4", rows, kv_lora_rank, cache_exp);
    if (rc) return rc;
    if (rows == 0) return DSA_OK;
    if (!x || !codes || !scales)
        return fail(DSA_ERR_INVALID_ARG, "dsa_quantize_latent_fp4: NULL tensor");
    if ((((uintptr_t)x) | ((uintptr_t)codes) | ((uintptr_t)scales)) & 15)
        return fail(DSA_ERR_INVALID_ARG,
                    "dsa_quantize_latent_fp4: tensors must be 16-byte aligned");
    const long long blocks = rows * (kv_lora_rank / kF4Block);
    const bool many = many_blocks(blocks);
    const long long grid = (blocks + kF4Threads * (many ? 4 : 1) - 1) / (kF4Threads * (many ? 4 : 1));
    cudaError_t e = launch_pdl(many ? quantize_latent_fp4_kernel<4> : quantize_latent_fp4_kernel<1>, dim3((unsigned)grid), dim3(kF4Threads),
                               0, (cudaStream_t)stream, (const uint4*)x, blocks, cache_exp,
                               (uint2*)codes, scales);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "dsa_quantize_latent_fp4 launch");
    return DSA_OK;
}

extern "C" int dsa_dequantize_latent_fp4(const uint8_t* codes, const uint8_t* scales,
                                         long long cache_rows, const int32_t* row_ids,
                                         long long rows, int kv_lora_rank, int cache_exp,
                                         dsa_bf16* out, int32_t* status, void* stream) {
    int rc = check_fp4("dsa_dequantize_latent_fp4", rows, kv_lora_rank, cache_exp);
    if (rc) return rc;
    if (cache_rows < 0 || (!row_ids && rows > cache_rows))
        return fail(DSA_ERR_INVALID_ARG, "dsa_dequantize_latent_fp4: %lld rows of a cache of %lld",
                    rows, cache_rows);
    if (rows == 0) return DSA_OK;
    if (!codes || !scales || !out)
        return fail(DSA_ERR_INVALID_ARG, "dsa_dequantize_latent_fp4: NULL tensor");
    if ((((uintptr_t)out) | ((uintptr_t)codes) | ((uintptr_t)scales)) & 15)
        return fail(DSA_ERR_INVALID_ARG,
                    "dsa_dequantize_latent_fp4: tensors must be 16-byte aligned");
    const int per_row = kv_lora_rank / kF4Block;
    const long long blocks = rows * per_row;
    const bool many = many_blocks(blocks);
    const long long grid = (blocks + kF4Threads * (many ? 4 : 1) - 1) / (kF4Threads * (many ? 4 : 1));
    cudaError_t e =
        launch_pdl(many ? dequantize_latent_fp4_kernel<4> : dequantize_latent_fp4_kernel<1>, dim3((unsigned)grid), dim3(kF4Threads), 0,
                   (cudaStream_t)stream, (const uint2*)codes, scales, row_ids, blocks, per_row,
                   cache_rows, cache_exp, (uint4*)out, status);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "dsa_dequantize_latent_fp4 launch");
    return DSA_OK;
}
