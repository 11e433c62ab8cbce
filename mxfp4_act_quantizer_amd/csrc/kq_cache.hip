// The paged MXFP4 key/value cache: rows quantized as they are written, and
// read back as bf16.  Layout (mx_cache in the public header): codes of one
// head's page are [page_size][dim/2] bytes, its scales [dim/32][page_size],
// so a tile of tokens of a head is one run of codes, and the scales of a
// block over consecutive tokens are consecutive bytes.
//
// A quad of lanes holds one block of 32 channels, eight per lane, as in the
// butterfly quantizer: the same transform stages and the same MX step, so a
// rotated key gets exactly the codes that the butterfly kq_quantize gives it.
// A wave takes 16 blocks at a time of as many whole rows as fill it, which
// makes its bf16 side whole 1-KB runs.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kq_device.h"
#include "kq_internal.h"
#include "kq_paged.h"

namespace kq {
namespace {

constexpr int kWaves = 4;

struct LaneRow {
    int row;      // row of the batch (in range when slot >= 0)
    int64_t slot; // cache slot of the row, or -1
};

// The lane's row (row0 + sub): the wave finds the sequence of row0 together,
// then each lane steps on over the few sequences that start inside the wave.
__device__ __forceinline__ LaneRow lane_row(const mx_cache &c, const mx_batch &b, int64_t row0, int sub, int lane)
{
    LaneRow r;
    const int64_t row = row0 + sub;
    int s = wave_search((int)b.seqs, row0, lane, [&](int i) { return (int64_t)b.row_start[i]; });
    while (s + 1 < b.seqs && (int64_t)b.row_start[s + 1] <= row)
        ++s;
    const SeqRows q = seq_rows(b, s);
    r.row = (int)row;
    r.slot = row < q.first || row >= (int64_t)q.first + q.rows ? -1 : cache_slot(c, b, s, q.pos0 + (row - q.first));
    return r;
}

__device__ __forceinline__ int64_t code_at(const mx_cache &c, int64_t slot, int head)
{
    const int64_t page = slot / c.page_size, off = slot - page * c.page_size;
    return ((page * c.heads + head) * c.page_size + off) * (c.dim / 2);
}

__device__ __forceinline__ int64_t scale_at(const mx_cache &c, int64_t slot, int head, int blk)
{
    const int64_t page = slot / c.page_size, off = slot - page * c.page_size;
    return ((page * c.heads + head) * (c.dim / 32) + blk) * c.page_size + off;
}

// blockIdx.y: 0 keys, 1 values.
template <bool kRotate>
__global__ __launch_bounds__(64 * kWaves) void mx_cache_write_kernel(const uint16_t *__restrict__ k,
                                                                     const uint16_t *__restrict__ v, int64_t k_stride,
                                                                     int64_t v_stride,
                                                                     const float *__restrict__ factors, int64_t nT,
                                                                     mx_cache c, mx_batch b, int rows_per_wave)
{
    const int lane = threadIdx.x & 63;
    const int64_t row0 = ((int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6)) * rows_per_wave;
    if (row0 >= b.rows)
        return;
    const bool value = blockIdx.y != 0;
    const uint16_t *x = value ? v : k;
    const int64_t stride = value ? v_stride : k_stride;
    uint8_t *codes = value ? c.vq : c.kq, *scales = value ? c.vs : c.ks;
    const int dim_blocks = (int)c.dim / 32, blocks = (int)c.heads * dim_blocks; // of a row
    const int qp = lane & 3, quad = lane >> 2;
    const int sub = rows_per_wave > 1 ? quad / blocks : 0;
    const bool lives = sub < rows_per_wave;
    const LaneRow r = lane_row(c, b, row0, lives ? sub : 0, lane);
    // a quad's lanes agree on the row, so whole quads run or skip
    if (!lives || r.slot < 0)
        return;
    for (int blk = quad - sub * blocks; blk < blocks; blk += 16) {
        const int head = blk / dim_blocks, hb = blk - head * dim_blocks;
        const u32x4 w = *(const u32x4 *)(x + (int64_t)r.row * stride + blk * 32 + qp * 8);
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf16lo(w[i]) + 0.0f; // -0 becomes +0: a code's sign means < 0
            f[2 * i + 1] = bf16hi(w[i]) + 0.0f;
        }
        if (kRotate && !value) {
            Bfly B;
            bfly_setup(B, factors + (nT == 1 ? 0 : (int64_t)blk * 20), qp);
            bfly_stages(f, B);
        }
        unsigned byte;
        const unsigned code = mx_encode_quad(f, byte);
        *(unsigned *)(codes + code_at(c, r.slot, head) + hb * 16 + qp * 4) = code;
        if (qp == 0)
            scales[scale_at(c, r.slot, head, hb)] = (uint8_t)byte;
        if (rows_per_wave > 1)
            break;
    }
}

__global__ __launch_bounds__(64 * kWaves) void mx_cache_read_kernel(mx_cache c, mx_batch b, uint16_t *__restrict__ k,
                                                                    uint16_t *__restrict__ v, int rows_per_wave)
{
    const int lane = threadIdx.x & 63;
    const int64_t row0 = ((int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6)) * rows_per_wave;
    if (row0 >= b.rows)
        return;
    const bool value = blockIdx.y != 0;
    uint16_t *x = value ? v : k;
    const uint8_t *codes = value ? c.vq : c.kq, *scales = value ? c.vs : c.ks;
    const int dim_blocks = (int)c.dim / 32, blocks = (int)c.heads * dim_blocks;
    const int qp = lane & 3, quad = lane >> 2;
    const int sub = rows_per_wave > 1 ? quad / blocks : 0;
    const bool lives = sub < rows_per_wave;
    const LaneRow r = lane_row(c, b, row0, lives ? sub : 0, lane);
    if (!lives || r.slot < 0)
        return;
    for (int blk = quad - sub * blocks; blk < blocks; blk += 16) {
        const int head = blk / dim_blocks, hb = blk - head * dim_blocks;
        const unsigned w = *(const unsigned *)(codes + code_at(c, r.slot, head) + hb * 16 + qp * 4);
        const unsigned s = scales[scale_at(c, r.slot, head, hb)];
        *(u32x4 *)(x + ((int64_t)r.row * blocks + blk) * 32 + qp * 8) =
            __builtin_bit_cast(u32x4, mx_bf16x8(w, scale_operand(s)));
        if (rows_per_wave > 1)
            break;
    }
}

// Rows of one wave: enough to give its 16 quads a block each.
int rows_per_wave(const mx_cache &c)
{
    const int64_t blocks = c.heads * (c.dim / 32);
    return blocks >= 16 ? 1 : (int)(16 / blocks);
}

dim3 grid_of(const mx_batch &b, int rpw)
{
    const int64_t per = (int64_t)kWaves * rpw;
    return dim3((unsigned)((b.rows + per - 1) / per), 2);
}

} // namespace

hipError_t launch_cache_write(const uint16_t *k, const uint16_t *v, int64_t k_stride, int64_t v_stride,
                              const float *factors, int64_t nT, const mx_cache &c, const mx_batch &b,
                              hipStream_t stream)
{
    const int rpw = rows_per_wave(c);
    const dim3 grid = grid_of(b, rpw);
    if (factors)
        mx_cache_write_kernel<true><<<grid, 64 * kWaves, 0, stream>>>(k, v, k_stride, v_stride, factors, nT, c, b, rpw);
    else
        mx_cache_write_kernel<false><<<grid, 64 * kWaves, 0, stream>>>(k, v, k_stride, v_stride, factors, nT, c, b,
                                                                       rpw);
    return hipGetLastError();
}

hipError_t launch_cache_read(const mx_cache &c, const mx_batch &b, uint16_t *k, uint16_t *v, hipStream_t stream)
{
    const int rpw = rows_per_wave(c);
    mx_cache_read_kernel<<<grid_of(b, rpw), 64 * kWaves, 0, stream>>>(c, b, k, v, rpw);
    return hipGetLastError();
}

} // namespace kq
