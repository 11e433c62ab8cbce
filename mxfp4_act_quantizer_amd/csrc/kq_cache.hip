// The paged MXFP4 key/value cache: rows quantized as they are written, and
// read back as bf16.  Layout (mx_cache in the public header): codes of one
// head's page are [page_size][dim/2] bytes, its scales [dim/32][page_size],
// so a tile of tokens of a head is one run of codes, and the scales of a
// block over consecutive tokens are consecutive bytes.
//
// A quad of lanes holds one block of 32 channels, eight per lane, as in the
// butterfly quantizer: the same transform stages and the same MX step, so a
// rotated key gets exactly the codes that the butterfly kq_quantize gives it.
//
// A wave keeps its 16 blocks of a row (or all blocks of 16 / blocks rows, where
// a row has fewer) and goes through up to four steps of rows with them: the
// factors of a block are read once, the bf16 side is whole runs of 1 KB, and
// the loads of all steps are in flight together.  The rows' slots are found by
// the lanes side by side, before the steps.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kq_device.h"
#include "kq_internal.h"
#include "kq_paged.h"

namespace kq {
namespace {

constexpr int kWaves = 4;

constexpr int kSteps = 4; // 1, 2, 4, 8, 12: 25.6, 20.2, 19.4, 19.0, 20.9 us (9224 rotated rows), 3.8 .. 4.5 us (61)
constexpr unsigned kXcds = 8;

// How a wave's quads lie over rows and blocks.
struct Tiling {
    int blocks;  // of a row
    int abreast; // rows of a step
    int steps;   // of a wave; abreast * steps <= 64
    int groups;  // waves along the blocks of a row
};

// Slot of row0 + lane for the first `rows` lanes of the wave (-1: none).  The
// wave finds the sequence of row0 together and reads the next 64 starts at
// once; each lane then looks its row up among them.
__device__ __forceinline__ int64_t lane_slot(const mx_cache &c, const mx_batch &b, int64_t row0, int rows, int lane)
{
    const int S = (int)b.seqs;
    const int s0 = wave_search(S, row0, lane, [&](int i) { return (int64_t)b.row_start[i]; });
    const int at = s0 + 1 + lane < S ? s0 + 1 + lane : S;
    const int start = b.row_start[at];
    const int64_t row = row0 + (lane < rows ? lane : 0);
    int n = 0; // starts among the 64 at or before the row (those of index S end the last sequence)
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) {
        const int v = __shfl(start, n + m - 1, 64);
        n += s0 + n + m < S && v <= row ? m : 0;
    }
    const int last = __shfl(start, 63, 64);
    int s = s0 + n;
    if (n == 63 && s0 + 64 < S && last <= row)
        ++s;
    while (n == 63 && s + 1 < S && b.row_start[s + 1] <= row)
        ++s;
    if (lane >= rows)
        return -1;
    const SeqRows q = seq_rows(b, s);
    return row < q.first || row >= (int64_t)q.first + q.rows ? -1 : cache_slot(c, b, s, q.pos0 + (row - q.first));
}

__device__ __forceinline__ int64_t shfl64(int64_t v, int lane)
{
    return (int64_t)((uint64_t)(unsigned)__shfl((int)v, lane, 64) | (uint64_t)(unsigned)__shfl((int)(v >> 32), lane, 64) << 32);
}

// This lane's place: its block, and for each step its row and slot.
struct LanePlace {
    int blk, head, hb; // block of the row, its head and place in the head
    int sub, rows;     // its row of a step, and the wave's rows
    int64_t row0;      // first of them
    int64_t slot[kSteps]; // slot < 0: nothing to do
    bool lives;        // the lane has a block at all

    __device__ __forceinline__ LanePlace(const mx_cache &c, const mx_batch &b, const Tiling &t, int lane, int wave)
    {
        // workgroups go to the eight XCDs in turn: each takes a run of rows, so
        // that the bytes of a cache line meet in one L2
        const unsigned run = gridDim.x / kXcds;
        const int64_t unit = (int64_t)(blockIdx.x % kXcds * run + blockIdx.x / kXcds) * kWaves + wave;
        const int group = (int)(unit % t.groups), quad = lane >> 2;
        row0 = unit / t.groups * (t.abreast * t.steps);
        sub = t.abreast > 1 ? quad / t.blocks : 0;
        blk = t.abreast > 1 ? quad - sub * t.blocks : 16 * group + quad;
        lives = sub < t.abreast && blk < t.blocks;
        const int dim_blocks = (int)c.dim / 32;
        head = blk / dim_blocks;
        hb = blk - head * dim_blocks;
        const int64_t left = b.rows - row0;
        rows = left <= 0 ? 0 : left < t.abreast * t.steps ? (int)left : t.abreast * t.steps;
    }

    __device__ __forceinline__ int64_t row(const Tiling &t, int i) const { return row0 + i * t.abreast + sub; }

    // Is there a row of the batch in step i?
    __device__ __forceinline__ bool in(const Tiling &t, int i) const
    {
        return lives && i < t.steps && i * t.abreast + sub < rows;
    }

    __device__ __forceinline__ void find_slots(const mx_cache &c, const mx_batch &b, const Tiling &t, int lane)
    {
        const int64_t mine = lane_slot(c, b, row0, rows, lane);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int64_t v = shfl64(mine, (i * t.abreast + (lives ? sub : 0)) & 63);
            slot[i] = in(t, i) ? v : -1;
        }
    }

    __device__ __forceinline__ void address(const mx_cache &c, int i, int64_t &codes, int64_t &scale) const
    {
        const int size = (int)c.page_size;
        const unsigned page = (unsigned)((uint64_t)slot[i] / (unsigned)size);
        const unsigned off = (unsigned)(slot[i] - (int64_t)page * size);
        const int64_t block = (int64_t)page * c.heads + head;
        codes = (block * size + off) * (c.dim / 2) + hb * 16;
        scale = (block * (c.dim / 32) + hb) * size + off;
    }
};

// blockIdx.y: 0 keys, 1 values.
template <bool kRotate>
__global__ __launch_bounds__(64 * kWaves) void mx_cache_write_kernel(const uint16_t *__restrict__ k,
                                                                     const uint16_t *__restrict__ v, int64_t k_stride,
                                                                     int64_t v_stride,
                                                                     const float *__restrict__ factors, int64_t nT,
                                                                     mx_cache c, mx_batch b, Tiling t)
{
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), qp = lane & 3;
    const bool value = blockIdx.y != 0;
    const uint16_t *x = value ? v : k;
    const int64_t stride = value ? v_stride : k_stride;
    uint8_t *codes = value ? c.vq : c.kq, *scales = value ? c.vs : c.ks;
    LanePlace p(c, b, t, lane, wave);
    // the rows themselves, while their slots are looked up; a quad's lanes
    // agree on block and rows, so whole quads run or skip
    u32x4 w[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
        if (p.in(t, i))
            w[i] = *(const u32x4 *)(x + p.row(t, i) * stride + p.blk * 32 + qp * 8);
    p.find_slots(c, b, t, lane);
    Bfly B{};
    if (kRotate && !value && p.lives)
        bfly_setup(B, factors + (nT == 1 ? 0 : (int64_t)p.blk * 20), qp);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        if (p.slot[i] < 0)
            continue;
        float f[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f[2 * e] = bf16lo(w[i][e]) + 0.0f; // -0 becomes +0: a code's sign means < 0
            f[2 * e + 1] = bf16hi(w[i][e]) + 0.0f;
        }
        if (kRotate && !value)
            bfly_stages(f, B);
        unsigned byte;
        const unsigned code = mx_encode_quad(f, byte);
        int64_t at, sat;
        p.address(c, i, at, sat);
        *(unsigned *)(codes + at + qp * 4) = code;
        if (qp == 0)
            scales[sat] = (uint8_t)byte;
    }
}

__global__ __launch_bounds__(64 * kWaves) void mx_cache_read_kernel(mx_cache c, mx_batch b, uint16_t *__restrict__ k,
                                                                    uint16_t *__restrict__ v, Tiling t)
{
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), qp = lane & 3;
    const bool value = blockIdx.y != 0;
    uint16_t *x = value ? v : k;
    const uint8_t *codes = value ? c.vq : c.kq, *scales = value ? c.vs : c.ks;
    LanePlace p(c, b, t, lane, wave);
    p.find_slots(c, b, t, lane);
    unsigned w[kSteps], s[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
        if (p.slot[i] >= 0) {
            int64_t at, sat;
            p.address(c, i, at, sat);
            w[i] = *(const unsigned *)(codes + at + qp * 4);
            s[i] = scales[sat];
        }
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
        if (p.slot[i] >= 0)
            *(u32x4 *)(x + (p.row(t, i) * t.blocks + p.blk) * 32 + qp * 8) =
                __builtin_bit_cast(u32x4, mx_bf16x8(w[i], scale_operand(s[i])));
}

// Four steps a wave where that leaves four waves a CU; fewer rows are spread
// over more waves.
Tiling tiling(const mx_cache &c, const mx_batch &b)
{
    Tiling t{};
    t.blocks = (int)(c.heads * (c.dim / 32));
    t.abreast = t.blocks >= 16 ? 1 : 16 / t.blocks;
    t.groups = t.abreast > 1 ? 1 : (t.blocks + 15) / 16;
    const int64_t waves = (b.rows + t.abreast - 1) / t.abreast * t.groups; // of one step, keys or values alone
    const int64_t want = waves * 2 / (4 * (int64_t)device_cus());
    const int most = 64 / t.abreast < kSteps ? 64 / t.abreast : kSteps;
    t.steps = (int)(want < 1 ? 1 : want > most ? most : want);
    return t;
}

dim3 grid_of(const mx_batch &b, const Tiling &t)
{
    const int64_t rows = (int64_t)t.abreast * t.steps, waves = (b.rows + rows - 1) / rows * t.groups;
    const int64_t wgs = (waves + kWaves - 1) / kWaves;
    return dim3((unsigned)((wgs + kXcds - 1) / kXcds * kXcds), 2); // whole runs; those past the rows have none
}

} // namespace

hipError_t launch_cache_write(const uint16_t *k, const uint16_t *v, int64_t k_stride, int64_t v_stride,
                              const float *factors, int64_t nT, const mx_cache &c, const mx_batch &b,
                              hipStream_t stream)
{
    const Tiling t = tiling(c, b);
    const dim3 grid = grid_of(b, t);
    if (factors)
        mx_cache_write_kernel<true><<<grid, 64 * kWaves, 0, stream>>>(k, v, k_stride, v_stride, factors, nT, c, b, t);
    else
        mx_cache_write_kernel<false><<<grid, 64 * kWaves, 0, stream>>>(k, v, k_stride, v_stride, factors, nT, c, b,
                                                                       t);
    return hipGetLastError();
}

hipError_t launch_cache_read(const mx_cache &c, const mx_batch &b, uint16_t *k, uint16_t *v, hipStream_t stream)
{
    const Tiling t = tiling(c, b);
    mx_cache_read_kernel<<<grid_of(b, t), 64 * kWaves, 0, stream>>>(c, b, k, v, t);
    return hipGetLastError();
}

} // namespace kq
