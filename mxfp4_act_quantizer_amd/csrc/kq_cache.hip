// The paged MXFP4 key/value cache: rows quantized as they are written, and
// read back as bf16.  Layout (mx_cache in the public header): codes of one
// head's page are [page_size][dim/2] bytes, its scales [dim/32][page_size],
// so a tile of tokens of a head is one run of codes, and the scales of a
// block over consecutive tokens are consecutive bytes.
//
// A quad of lanes holds one block of 32 channels, eight per lane, as in the
// butterfly quantizer: the same transform stages and the same MX step.  A
// rotated key gets the codes of the exact transform: where fp32 leaves a code
// in doubt, the block is done again in double.
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

// ---- rotated keys: codes of the exact transform ----------------------------
// The butterfly's five stages run in fp32, ten roundings on the way of each
// sum, so a value may be off by gamma_10 z, z = sum_k |x_k| |K_kj| <= max|x|
// times the product of the factors' largest column sums.  12 * 2^-24 of that
// bound covers it, the rounding of value + bound and the bound's own.  Where a
// code or the scale byte would be another one within that distance (about one
// step of a wave in twenty), the wave does the step again in double, rounded to
// fp32 so that the conversion to codes rounds as if from the double itself.
// (Put off until after a wave's steps, which then need 88 registers instead of
// 117, the second loads cost more: 39.6 us instead of 35.)  A cached key is read as often
// as there are tokens after it, so its codes are the nearest ones: 9224 rows of
// 8 x 128, written and read, take 34.5 us, and 31.7 without the check.
struct Doubt {
    float reach; // of the bound above, relative to max|x|

    // f: the block's values, x: what they were computed from, of a quad.
    __device__ __forceinline__ bool operator()(const float (&f)[8], const float (&x)[8]) const
    {
        float ax = 0.0f, af = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            ax = amax_step(ax, x[i]);
            af = amax_step(af, f[i]);
        }
        ax = vmax(ax, dpp_xor1(ax));
        ax = vmax(ax, dpp_xor2(ax));
        af = vmax(af, dpp_xor1(af));
        af = vmax(af, dpp_xor2(af));
        const float off = reach * ax;
        const unsigned b = e8m0_byte(af - off);
        float lo[8], hi[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo[i] = f[i] - off;
            hi[i] = f[i] + off;
        }
        const float sc = scale_operand(b);
        const bool same = b == e8m0_byte(af + off) && cvt8(lo[0], lo[1], lo[2], lo[3], lo[4], lo[5], lo[6], lo[7], sc) ==
                                                          cvt8(hi[0], hi[1], hi[2], hi[3], hi[4], hi[5], hi[6], hi[7], sc);
        // blocks with a NaN or an infinity are settled; where subnormals may
        // have been rounded, or fp32 was left on the way, nothing is
        if (!(ax < __builtin_inff()) || ax == 0.0f)
            return false;
        return !same || ax < 0x1p-90f || !(af + off < __builtin_inff());
    }
};

__device__ __forceinline__ Doubt doubt_of(const float *__restrict__ F)
{
    float reach = 0x1.8p-21f; // 12 * 2^-24
#pragma unroll
    for (int k = 0; k < 5; ++k) {
        const float c0 = __builtin_fabsf(F[4 * k]) + __builtin_fabsf(F[4 * k + 2]);
        const float c1 = __builtin_fabsf(F[4 * k + 1]) + __builtin_fabsf(F[4 * k + 3]);
        reach *= vmax(c0, c1);
    }
    return {reach};
}

__device__ __forceinline__ double dpp_double(double v, bool two)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const float lo = __uint_as_float((unsigned)b), hi = __uint_as_float((unsigned)(b >> 32));
    const unsigned l = __float_as_uint(two ? dpp_xor2(lo) : dpp_xor1(lo));
    const unsigned h = __float_as_uint(two ? dpp_xor2(hi) : dpp_xor1(hi));
    return __builtin_bit_cast(double, (uint64_t)h << 32 | l);
}

// fp32 with the last bit set where y lies between two of them (never to
// even), so that a second rounding to fewer bits is right; not -0.
__device__ __forceinline__ float round_to_odd(double y)
{
    const float r = (float)y;
    unsigned b = __float_as_uint(r);
    const bool finite = (b & 0x7F800000u) != 0x7F800000u;
    if (finite && (double)r != y && !(b & 1u))
        b += (y > (double)r) != ((b >> 31) != 0) ? 1u : 0xFFFFFFFFu;
    return __uint_as_float(b) + 0.0f;
}

__device__ __forceinline__ void bfly_exact(float (&f)[8], const Bfly &B)
{
    double v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = (double)f[i];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = fma_f64((double)B.o1, dpp_double(v[i], true), (double)B.s1 * v[i]);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = fma_f64((double)B.o2, dpp_double(v[i], false), (double)B.s2 * v[i]);
    auto stage = [&](int st, const float(&A)[4]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i & st)
                continue;
            const double u = v[i], w = v[i + st];
            v[i] = fma_f64((double)A[0], u, (double)A[2] * w);
            v[i + st] = fma_f64((double)A[1], u, (double)A[3] * w);
        }
    };
    stage(4, B.a3);
    stage(2, B.a4);
    stage(1, B.a5);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        f[i] = round_to_odd(v[i]);
}

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
    Doubt doubt{0.0f};
    if (kRotate && !value && p.lives) {
        const float *F = factors + (nT == 1 ? 0 : (int64_t)p.blk * 20);
        bfly_setup(B, F, qp);
        doubt = doubt_of(F);
    }
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
        if (kRotate && !value) {
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[e] = f[e];
            bfly_stages(f, B);
            if (__builtin_amdgcn_ballot_w64(doubt(f, x))) {
                bfly_exact(x, B);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    f[e] = x[e];
            }
        }
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
