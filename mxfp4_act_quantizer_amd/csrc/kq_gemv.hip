// Products of a few bf16 rows with an MXFP4 weight matrix (W4A16):
// out[m, n] = sum_k x[m, k] W[n, k] for 1..64 rows x, W as mx_gemm's second
// operand (codes [N, K/2], element 2i in the low nibble; E8M0 scales
// [N, K/32]).  This is the linear layer of a single-token step, and of the
// AdaLN modulation, whose input is one conditioning row per sample.
//
// A weight is E2M1 value x 2^(s - 127): two significant bits, so it is exact
// in bf16 (the convert instruction applies the scale in the same step), and
// the products run on the bf16 matrix cores with fp32 sums: nothing is
// rounded before the final store.
//
// v_mfma_f32_16x16x32_bf16 with the weights as the row operand: lane l holds
// row l % 16 and eight k of group l / 16.  Which eight is free as long as
// both operands agree, so group g takes the whole MX block 4u + g of a step u
// of 128 k: one 16-byte code load and one scale byte per lane feed four
// matrix instructions, the j-th on the block's elements 8j..8j+7.  The 16
// columns are tokens (kMT column tiles; the columns past M read as zeros).
// The accumulator holds W row 4 (l / 16) + i, token l % 16 in element i.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kq_device.h"
#include "kq_internal.h"

namespace kq {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4; // waves of a workgroup, splitting k

template <int kMT, bool kBF16>
__global__ __launch_bounds__(64 * kWaves) void mx_gemv_kernel(const uint16_t *__restrict__ x,
                                                              const uint8_t *__restrict__ qw,
                                                              const uint8_t *__restrict__ sw, void *__restrict__ out,
                                                              int M, int N, int K)
{
    __shared__ f32x4 red[kWaves - 1][kMT][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = lane & 15, g = lane >> 4;
    const int n0 = (int)blockIdx.x * 16;
    const int rows = N - n0 < 16 ? N - n0 : 16;
    const int blocks = K / 32;
    const __amdgpu_buffer_rsrc_t rq = out_buffer((void *)(qw + (int64_t)n0 * (K / 2)), (int64_t)rows * (K / 2));
    const __amdgpu_buffer_rsrc_t rs = out_buffer((void *)(sw + (int64_t)n0 * blocks), (int64_t)rows * blocks);
    const __amdgpu_buffer_rsrc_t rx = out_buffer((void *)x, (int64_t)M * K * 2);

    f32x4 acc[kMT];
#pragma unroll
    for (int t = 0; t < kMT; ++t)
        acc[t] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
    const int steps = (blocks + 3) / 4;
    for (int u = wave; u < steps; u += kWaves) {
        const int b = 4 * u + g;
        const unsigned drop = (unsigned)(b >= blocks) << 31; // reads zeros
        const u32x4 w = __builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(rq, (int)((unsigned)(c * (K / 2) + b * 16) | drop), 0, 0));
        const unsigned s =
            __builtin_amdgcn_raw_buffer_load_b8(rs, (int)((unsigned)(c * blocks + b) | drop), 0, 0) & 0xFFu;
        const float sc = scale_operand(s);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bf16x8 a = mx_bf16x8(w[j], sc);
#pragma unroll
            for (int t = 0; t < kMT; ++t) {
                const unsigned off = (unsigned)(((16 * t + c) * K + b * 32 + 8 * j) * 2) | drop;
                const bf16x8 v =
                    __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(rx, (int)off, 0, 0));
                acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, v, acc[t], 0, 0, 0);
            }
        }
    }
    if (wave) {
#pragma unroll
        for (int t = 0; t < kMT; ++t)
            red[wave - 1][t][lane] = acc[t];
    }
    __syncthreads();
    if (wave)
        return;
#pragma unroll
    for (int t = 0; t < kMT; ++t) {
#pragma unroll
        for (int w = 0; w < kWaves - 1; ++w)
            acc[t] += red[w][t][lane];
        const int m = 16 * t + c;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = n0 + 4 * g + i;
            if (m < M && n < N) {
                if (kBF16)
                    ((__bf16 *)out)[(int64_t)m * N + n] = (__bf16)acc[t][i];
                else
                    ((float *)out)[(int64_t)m * N + n] = acc[t][i];
            }
        }
    }
}

template <int kMT>
hipError_t launch_gemv(const uint16_t *x, int M, const uint8_t *qw, const uint8_t *sw, int N, int K, void *out,
                       int bf16, hipStream_t stream)
{
    const dim3 grid((unsigned)((N + 15) / 16)), wg(64 * kWaves);
    if (bf16)
        mx_gemv_kernel<kMT, true><<<grid, wg, 0, stream>>>(x, qw, sw, out, M, N, K);
    else
        mx_gemv_kernel<kMT, false><<<grid, wg, 0, stream>>>(x, qw, sw, out, M, N, K);
    return hipGetLastError();
}

} // namespace

hipError_t launch_mx_gemv(const uint16_t *x, int64_t M, const uint8_t *qw, const uint8_t *sw, int64_t N, int64_t K,
                          void *out, int bf16, hipStream_t stream)
{
    const int m = (int)M, n = (int)N, k = (int)K;
    if (m <= 16)
        return launch_gemv<1>(x, m, qw, sw, n, k, out, bf16, stream);
    if (m <= 32)
        return launch_gemv<2>(x, m, qw, sw, n, k, out, bf16, stream);
    return launch_gemv<4>(x, m, qw, sw, n, k, out, bf16, stream);
}

} // namespace kq
