// Attention of a step's new tokens over the paged MXFP4 cache.  For a row of
// sequence i at position p, query head h and its key/value head:
//   o = sum_j softmax_j(scale q . K_j) V_j over the positions j it sees,
//   j <= p, and with a window w only p - j < w or j < sinks;
// a row that sees nothing (or whose visible scores are all -infinity) is 0.
//
// Everything runs on the bf16 matrix cores: a cached value is exact in bf16
// (kq_device.h, mx_bf16x8), scores and sums are fp32, and the only roundings
// before the output are those of the softmax weights to bf16.
//
// Work: the query heads that share a key/value head are stacked, so the rows
// of one sequence and head are rows x group columns, cut into tiles of R.  A
// wave holds kNQ tiles of 16 columns and walks the cache in tiles of 32
// positions:
//  - scores S^T = K Q^T, v_mfma_f32_16x16x32_bf16 with 16 positions as rows.
//    Lane (c, g) = (l % 16, l / 16) takes position c's channels [8 NB g, 8 NB
//    (g + 1)) (NB = dim / 32): one code load a position and group, the same
//    channels of Q in the column operand;
//  - the accumulator's rows are positions 4g + i, and those are the k slots
//    that the lane gives the next product, so the weights go straight from
//    the softmax registers into its operand: k slot 8g + i is position 4g +
//    i of the tile's first half, 8g + 4 + i of its second;
//  - O^T = V^T P^T with 16 channels as rows.  Lane (c, g) reads channels [2
//    NB c, 2 NB (c + 1)) of the positions of its k slots, converts them and
//    regroups pairs of positions; the j-th product covers channels 2 NB c + j.
//    A lane then holds 8 NB consecutive channels of its column's output.
// No shared memory and no barrier in the loop: the cache is read as 4-bit
// codes (17 bytes per 32 values), small enough to be fetched and converted by
// every wave that needs it.
//
// Softmax: one pass, running maximum and sum.  The maximum used for scaling is
// raised only when a score exceeds it by 2^8 (weights then stay below 2^8,
// sums far below fp32's range), so most tiles need no reduction across lanes
// and no rescaling; the sum is kept per lane and reduced once at the end.
//
// Few columns: the waves of a workgroup take every kWK-th tile and join
// through LDS; long sequences are also split over workgroups, whose partial
// results a second kernel joins.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kq_device.h"
#include "kq_internal.h"
#include "kq_paged.h"

namespace kq {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

constexpr int kTile = 32;  // cache positions of a step
constexpr int kWaves = 4;  // of a workgroup
constexpr float kRaise = 8.0f; // log2 of how far a score may exceed the scaling maximum
constexpr int kMaxSplits = 128;
constexpr int kSplitSeqs = 256; // with more sequences there is work enough without splitting

struct AttnArgs {
    const uint16_t *q;
    uint16_t *out;
    float *part_o; // [splits][rows][q_heads][dim] unnormalised outputs
    float *part_ml; // [splits][rows][q_heads][2] maximum (log2) and sum
    int64_t q_stride, out_stride;
    mx_cache c;
    mx_batch b;
    int q_heads, group;
    int window, sinks;
    float scale2; // scale * log2(e)
    int splits;   // most splits of a sequence
    int wanted;   // workgroups that fill the chip
    unsigned size16, size_magic; // page_size / 16, and floor(2^32 / size16) + 1
    int tiles;    // column tiles: an upper bound over the batch
};

// Column tile `local` (R columns) of a sequence: its rows and positions, and
// the cache tiles that some column sees: `sink_tiles` first ones, then
// [first_tile, ...), n in all, in `splits` parts.
struct TilePlan {
    SeqRows seq;
    int cols;         // columns of the sequence
    int pmin, pmax;   // positions of the tile's first and last row
    int span;         // positions that can have a slot
    int sink_tiles, first_tile, n;
    int splits, per_split;
};

// Tiles of one sequence, roughly: for sharing out the splits.
__device__ __forceinline__ int rough_tiles(const AttnArgs &a, int s)
{
    int64_t len = a.b.lengths[s];
    const int64_t span = a.b.width * a.c.page_size;
    len = len < 0 ? 0 : len > span ? span : len;
    if (a.window) {
        const int64_t seen = (int64_t)a.window + a.sinks + (a.b.row_start[s + 1] - a.b.row_start[s]);
        len = seen < len && seen >= 0 ? seen : len;
    }
    return (int)((len + kTile - 1) / kTile);
}

// Cache tiles of one split: the batch's tiles over the workgroups wanted, at
// least two per wave.  Every wave gets the same answer.
__device__ __forceinline__ int split_tiles(const AttnArgs &a, int lane)
{
    float sum = 0.0f;
    for (int s = lane; s < a.b.seqs; s += 64)
        sum += (float)rough_tiles(a, s);
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1)
        sum += __shfl_xor(sum, m, 64);
    // each sequence has about tiles / seqs column tiles for every head
    const float units = sum * (float)a.tiles / (float)a.b.seqs * (float)a.c.heads;
    const int per = (int)(units / (float)a.wanted) + 1;
    return __builtin_amdgcn_readfirstlane(per < 2 * kWaves ? 2 * kWaves : per);
}

__device__ __forceinline__ void plan_tile(const AttnArgs &a, int s, int local, int R, int lane, TilePlan &t)
{
    t.seq = seq_rows(a.b, s);
    t.cols = t.seq.rows * a.group;
    const int64_t c0 = (int64_t)local * R;
    const int64_t c1 = c0 + R < t.cols ? c0 + R : t.cols; // one past the last
    t.span = (int)(a.b.width * a.c.page_size);
    t.pmin = (int)(t.seq.pos0 + c0 / a.group);
    t.pmax = (int)(t.seq.pos0 + (c1 - 1) / a.group);
    const int64_t end = (int64_t)t.pmax + 1;
    const int hi = end < 0 ? 0 : end > t.span ? t.span : (int)end;
    const int hi_tile = (hi + kTile - 1) / kTile;
    t.sink_tiles = t.first_tile = 0;
    if (a.window) {
        const int64_t lo = (int64_t)t.pmin - a.window + 1;
        t.first_tile = lo <= 0 ? 0 : (int)((lo < hi ? lo : hi) / kTile);
        t.sink_tiles = ((a.sinks < hi ? a.sinks : hi) + kTile - 1) / kTile;
        if (t.first_tile <= t.sink_tiles)
            t.sink_tiles = t.first_tile = 0;
    }
    t.n = t.sink_tiles + hi_tile - t.first_tile;
    t.splits = 1;
    t.per_split = t.n;
    if (a.splits > 1 && t.n > 0) {
        const int per = split_tiles(a, lane);
        const int want = (t.n + per - 1) / per;
        t.splits = want < a.splits ? want : a.splits;
        t.per_split = (t.n + t.splits - 1) / t.splits;
        t.splits = (t.n + t.per_split - 1) / t.per_split;
    }
}

// Largest of the four lane groups, in all of them.
__device__ __forceinline__ float max_groups(float v)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __builtin_fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
    const auto t = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __builtin_fmaxf(__uint_as_float(t[0]), __uint_as_float(t[1]));
}

__device__ __forceinline__ float sum_groups(float v)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    const auto t = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(t[0]) + __uint_as_float(t[1]);
}

__device__ __forceinline__ unsigned pack_bf16(float a, float b)
{
    return __builtin_bit_cast(unsigned, __builtin_convertvector((f32x2){a, b}, bf16x2));
}

// Raw codes and scales of one tile, as one lane reads them.
template <int NB>
struct RawTile {
    static constexpr int kVW = NB == 8 ? 2 : 1; // dwords of a V piece
    unsigned k[2][NB];
    unsigned ks[2][NB == 8 ? 2 : 1];
    unsigned v[8][kVW]; // k slots: positions 4g + i, 16 + 4g + i
    unsigned vs[2];
};

// Where half a tile (16 positions, always inside one page) lies.
struct Half {
    int64_t codes; // byte offset of its codes
    int64_t scales;
};

template <int NB>
__device__ __forceinline__ void load_half(const AttnArgs &a, const Half &at, int h, int c, int g, RawTile<NB> &r)
{
    const int size = (int)a.c.page_size;
    const uint8_t *kq = a.c.kq + at.codes, *vq = a.c.vq + at.codes;
    const uint8_t *ks = a.c.ks + at.scales, *vs = a.c.vs + at.scales;
    const unsigned kc = (unsigned)(c * (NB * 16) + g * (NB * 4));
    if constexpr (NB == 2) {
        const u32x2 w = *(const u32x2 *)(kq + kc);
        r.k[h][0] = w[0];
        r.k[h][1] = w[1];
    } else {
#pragma unroll
        for (int i = 0; i < NB / 4; ++i) {
            const u32x4 w = *(const u32x4 *)(kq + kc + 16 * i);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                r.k[h][4 * i + j] = w[j];
        }
    }
    const int kb = NB == 8 ? 2 * g : NB == 4 ? g : g >> 1;
    r.ks[h][0] = ks[(unsigned)(kb * size + c)];
    if constexpr (NB == 8)
        r.ks[h][1] = ks[(unsigned)((kb + 1) * size + c)];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const unsigned vc = (unsigned)((4 * g + i) * (NB * 16) + c * NB);
        if constexpr (NB == 2) {
            r.v[4 * h + i][0] = *(const uint16_t *)(vq + vc);
        } else if constexpr (NB == 4) {
            r.v[4 * h + i][0] = *(const unsigned *)(vq + vc);
        } else {
            const u32x2 w = *(const u32x2 *)(vq + vc);
            r.v[4 * h + i][0] = w[0];
            r.v[4 * h + i][RawTile<NB>::kVW - 1] = w[1];
        }
    }
    r.vs[h] = *(const unsigned *)(vs + (unsigned)((NB * c / 16) * size + 4 * g));
}

// NB = dim / 32; kNQ tiles of 16 columns per wave; kWQ waves of a workgroup
// along the columns, kWaves / kWQ along the cache.
template <int NB, int kNQ, int kWQ>
__global__ __launch_bounds__(64 * kWaves, 2) void attention_kernel(AttnArgs a)
{
    constexpr int kWK = kWaves / kWQ;
    constexpr int R = 16 * kNQ * kWQ; // columns of a workgroup
    constexpr int dim = 32 * NB;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int wq = wave / kWK, wk = wave % kWK;

    // workgroup -> (split, column tile, head), the head fastest: the eight
    // XCDs take workgroups in turn, so a head's cache stays in few L2s
    const int heads = (int)a.c.heads;
    int id = (int)blockIdx.x;
    const int head = id % heads;
    id /= heads;
    const int split = id % a.splits;
    const int tile = a.tiles - 1 - id / a.splits; // the last rows see most: they start first
    // the tiles of sequence s start at row_start[s] group / R + s, which leaves
    // it at least ceil(columns / R)
    auto first_of = [&](int s) {
        const int64_t r = a.b.row_start[s];
        return (r < 0 ? 0 : r) * a.group / R + s;
    };
    const int s = wave_search((int)a.b.seqs, tile, lane, first_of);
    const int64_t local64 = tile - first_of(s);
    if (local64 < 0 || local64 > ((int64_t)1 << 31) / R)
        return;
    const int local = (int)local64;
    TilePlan t;
    t.seq = seq_rows(a.b, s);
    if ((int64_t)local * R >= (int64_t)t.seq.rows * a.group)
        return;
    plan_tile(a, s, local, R, lane, t);
    if (split >= t.splits)
        return;
    const int begin = split * t.per_split;
    const int stop = begin + t.per_split < t.n ? begin + t.per_split : t.n;

    // queries, and what each column sees: [low, p] and the first `sinks`
    bf16x8 Q[kNQ][NB];
    int pos[kNQ], low[kNQ], row[kNQ], qhead[kNQ];
    bool live[kNQ];
#pragma unroll
    for (int n = 0; n < kNQ; ++n) {
        const int col = local * R + (wq * kNQ + n) * 16 + c;
        live[n] = col < t.cols;
        const int i = (live[n] ? col : 0) / a.group;
        row[n] = t.seq.first + i;
        qhead[n] = head * a.group + (live[n] ? col : 0) - i * a.group;
        pos[n] = live[n] ? (int)(t.seq.pos0 + i) : -1;
        low[n] = a.window && live[n] ? pos[n] - a.window + 1 : -0x7FFFFFFF;
        const uint16_t *q = a.q + (int64_t)row[n] * a.q_stride + qhead[n] * dim + g * (8 * NB);
#pragma unroll
        for (int i4 = 0; i4 < NB; ++i4) {
            u32x4 w = *(const u32x4 *)(q + 8 * i4);
            if (!live[n])
                w = (u32x4){0, 0, 0, 0};
            Q[n][i4] = __builtin_bit_cast(bf16x8, w);
        }
    }
    // positions of the wave's own columns, for tiles that need no mask
    const int wcol0 = local * R + wq * kNQ * 16;
    const int wcol1 = (wcol0 + kNQ * 16 < t.cols ? wcol0 + kNQ * 16 : t.cols) - 1;
    const bool idle = wcol0 >= t.cols; // a wave of padding columns only
    const int wmin = (int)(t.seq.pos0 + wcol0 / a.group);
    const int wmax = (int)(t.seq.pos0 + wcol1 / a.group);
    const int whi = idle || wmax < 0 ? 0 : wmax + 1 < t.span ? wmax + 1 : t.span;

    f32x4 acc[kNQ][2 * NB];
    float m[kNQ], l[kNQ];
#pragma unroll
    for (int n = 0; n < kNQ; ++n) {
        m[n] = -__builtin_inff();
        l[n] = 0.0f;
#pragma unroll
        for (int j = 0; j < 2 * NB; ++j)
            acc[n][j] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
    }

    const int size = (int)a.c.page_size;
    const int64_t page_codes = (int64_t)heads * size * (dim / 2), page_scales = (int64_t)heads * size * NB;
    const int32_t *table = a.b.page_table + (int64_t)s * a.b.width;
    auto tile_at = [&](int i) { return i < t.sink_tiles ? i : t.first_tile + i - t.sink_tiles; };
    // both halves of tile index i: their places, and whether they have one
    auto place = [&](int i, Half (&at)[2], bool (&there)[2]) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            // u / size16 by multiplication: u < 2^26 and size16 <= 64, so the
            // product's excess over u / size16 2^32 stays below 2^32
            const unsigned u = (unsigned)(2 * tile_at(i) + h);
            const unsigned pg = a.size16 == 1 ? u : __umulhi(u, a.size_magic);
            const unsigned off = 16 * (u - pg * a.size16);
            int page = (int)(16 * u) < t.span ? table[pg] : -1;
            there[h] = page >= 0 && page < (int)a.c.pages;
            page = there[h] ? page : 0;
            at[h].codes = page * page_codes + (unsigned)(head * size + off) * (dim / 2);
            at[h].scales = page * page_scales + (unsigned)(head * NB * size + off);
        }
    };
    auto load = [&](int i, RawTile<NB> &r, bool (&there)[2]) {
        Half at[2];
        place(i, at, there);
        load_half<NB>(a, at[0], 0, c, g, r);
        load_half<NB>(a, at[1], 1, c, g, r);
    };

    int i = begin + wk;
    RawTile<NB> next;
    bool there_next[2];
    if (i < stop)
        load(i, next, there_next);
    for (; i < stop; i += kWK) {
        RawTile<NB> r = next;
        const bool there[2] = {there_next[0], there_next[1]};
        load(i + kWK < stop ? i + kWK : i, next, there_next);
        const int j0 = tile_at(i) * kTile;
        if (kWQ > 1 && j0 >= whi)
            continue; // past this wave's columns (another wave's still see it)

        const bool full = j0 + kTile <= wmin + 1 && j0 + kTile <= t.span && there[0] && there[1] && !idle &&
                          (!a.window || j0 >= wmax - a.window + 1 || j0 + kTile <= a.sinks);

        f32x4 S[kNQ][2];
#pragma unroll
        for (int n = 0; n < kNQ; ++n)
            S[n][0] = S[n][1] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int p = 0; p < NB; ++p) {
                const bf16x8 kf = mx_bf16x8(r.k[h][p], scale_operand(r.ks[h][NB == 8 ? p / 4 : 0]));
#pragma unroll
                for (int n = 0; n < kNQ; ++n)
                    S[n][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, Q[n][p], S[n][h], 0, 0, 0);
            }
        }

        // scale bytes of the lane's eight positions of V
        unsigned vsb[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            vsb[k] = (r.vs[k >> 2] >> (8 * (k & 3))) & 0xFFu;

        unsigned nan_slots = 0; // positions of this lane whose V block is NaN, masked tiles only
        unsigned seen[kNQ];     // positions (bit 4h + i) that the column sees
        if (!full) {
#pragma unroll
            for (int n = 0; n < kNQ; ++n) {
                seen[n] = 0;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int h = k >> 2, j = j0 + 16 * h + 4 * g + (k & 3);
                    const bool see = j <= pos[n] && j < t.span && (j >= low[n] || j < a.sinks) && there[h];
                    seen[n] |= (unsigned)see << k;
                    S[n][h][k & 3] = see ? S[n][h][k & 3] : -__builtin_inff();
                }
            }
            // A weight of zero does not hide a NaN or an infinity of V: what
            // lies behind the wave's last position (another length, or never
            // written) is cleared, and a NaN block counts only for columns
            // that see it (below).
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int h = k >> 2, j = j0 + 16 * h + 4 * g + (k & 3);
                const bool dead = j >= whi || !there[h];
                const bool nan = vsb[k] == 0xFFu && !dead;
                nan_slots |= (unsigned)nan << k;
                if (dead || nan) {
                    vsb[k] = 127;
#pragma unroll
                    for (int w = 0; w < RawTile<NB>::kVW; ++w)
                        r.v[k][w] = 0;
                }
            }
        }

        // scores -> weights
        bool raise = false;
        float top[kNQ];
#pragma unroll
        for (int n = 0; n < kNQ; ++n) {
            float x = __builtin_fmaxf(S[n][0][0], S[n][0][1]);
            x = __builtin_fmaxf(x, __builtin_fmaxf(S[n][0][2], S[n][0][3]));
            x = __builtin_fmaxf(x, __builtin_fmaxf(S[n][1][0], S[n][1][1]));
            x = __builtin_fmaxf(x, __builtin_fmaxf(S[n][1][2], S[n][1][3]));
            top[n] = x * a.scale2;
            raise |= top[n] > m[n] + kRaise;
        }
        if (__builtin_amdgcn_ballot_w64(raise)) {
#pragma unroll
            for (int n = 0; n < kNQ; ++n) {
                const float up = __builtin_fmaxf(m[n], max_groups(top[n]));
                const float f = up == m[n] ? 1.0f : __builtin_amdgcn_exp2f(m[n] - up);
                m[n] = up;
                l[n] *= f;
#pragma unroll
                for (int j = 0; j < 2 * NB; ++j)
                    acc[n][j] *= f;
            }
        }
        bf16x8 P[kNQ];
#pragma unroll
        for (int n = 0; n < kNQ; ++n) {
            const float base = m[n] == -__builtin_inff() ? 0.0f : m[n];
            float w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                w[k] = __builtin_amdgcn_exp2f(__builtin_fmaf(S[n][k >> 2][k & 3], a.scale2, -base));
                l[n] += w[k];
            }
            const u32x4 pk = {pack_bf16(w[0], w[1]), pack_bf16(w[2], w[3]), pack_bf16(w[4], w[5]),
                              pack_bf16(w[6], w[7])};
            P[n] = __builtin_bit_cast(bf16x8, pk);
        }

#pragma unroll
        for (int b = 0; b < NB; ++b) {
            unsigned w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const unsigned raw = r.v[k][NB == 8 ? b / 4 : 0];
                const float sc = scale_operand(vsb[k]);
                bf16x2 v;
                switch (b & 3) { // the byte is part of the instruction
                case 0: v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(raw, sc, 0); break;
                case 1: v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(raw, sc, 1); break;
                case 2: v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(raw, sc, 2); break;
                default: v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(raw, sc, 3); break;
                }
                w[k] = __builtin_bit_cast(unsigned, v);
            }
            u32x4 even, odd; // channels 2b and 2b + 1 of the lane's eight positions
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                even[k] = __builtin_amdgcn_perm(w[2 * k + 1], w[2 * k], 0x05040100u);
                odd[k] = __builtin_amdgcn_perm(w[2 * k + 1], w[2 * k], 0x07060302u);
            }
#pragma unroll
            for (int n = 0; n < kNQ; ++n) {
                acc[n][2 * b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, even), P[n],
                                                                        acc[n][2 * b], 0, 0, 0);
                acc[n][2 * b + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, odd), P[n],
                                                                            acc[n][2 * b + 1], 0, 0, 0);
            }
        }

        // NaN blocks of V that some column of a masked tile may see: count
        // them per column with one more product (the rows of a lane share
        // their block), and spoil the channels where the count is not zero.
        if (!full && __builtin_amdgcn_ballot_w64(nan_slots != 0)) {
            u32x4 ind;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                ind[k] = ((nan_slots >> (2 * k) & 1u) * 0x3F80u) | ((nan_slots >> (2 * k + 1) & 1u) * 0x3F800000u);
#pragma unroll
            for (int n = 0; n < kNQ; ++n) {
                u32x4 see;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    see[k] = ((seen[n] >> (2 * k) & 1u) * 0x3F80u) | ((seen[n] >> (2 * k + 1) & 1u) * 0x3F800000u);
                const f32x4 count = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    __builtin_bit_cast(bf16x8, ind), __builtin_bit_cast(bf16x8, see),
                    (f32x4){0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
#pragma unroll
                for (int j = 0; j < 2 * NB; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[n][j][e] = count[e] > 0.0f ? __builtin_nanf("") : acc[n][j][e];
            }
        }
    }

    // sums over the lane groups, then over the waves that shared the tiles
#pragma unroll
    for (int n = 0; n < kNQ; ++n)
        l[n] = sum_groups(l[n]);
    if constexpr (kWK > 1) {
        __shared__ float sm[kWaves][kNQ][16], sl[kWaves][kNQ][16];
        __shared__ f32x4 so[kWaves - 1][kNQ][2 * NB][64];
        if (g == 0) {
#pragma unroll
            for (int n = 0; n < kNQ; ++n) {
                sm[wave][n][c] = m[n];
                sl[wave][n][c] = l[n];
            }
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < kNQ; ++n) {
            float up = sm[0][n][c];
#pragma unroll
            for (int w = 1; w < kWK; ++w)
                up = __builtin_fmaxf(up, sm[w][n][c]);
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kWK; ++w) {
                const float mw = sm[w][n][c];
                sum += sl[w][n][c] * (mw == up ? 1.0f : __builtin_amdgcn_exp2f(mw - up));
            }
            const float f = m[n] == up ? 1.0f : __builtin_amdgcn_exp2f(m[n] - up);
            m[n] = up;
            l[n] = sum;
#pragma unroll
            for (int j = 0; j < 2 * NB; ++j) {
                acc[n][j] *= f;
                if (wave)
                    so[wave - 1][n][j][lane] = acc[n][j];
            }
        }
        __syncthreads();
        if (wave)
            return;
#pragma unroll
        for (int n = 0; n < kNQ; ++n)
#pragma unroll
            for (int j = 0; j < 2 * NB; ++j)
#pragma unroll
                for (int w = 0; w < kWK - 1; ++w)
                    acc[n][j] += so[w][n][j][lane];
    }

    // the lane's channels [8 NB g, 8 NB (g + 1)) of column c: channel 2 NB e + j is acc[j][e]
#pragma unroll
    for (int n = 0; n < kNQ; ++n) {
        if (!live[n])
            continue;
        if (t.splits > 1) {
            const int64_t at = ((int64_t)split * a.b.rows + row[n]) * a.q_heads + qhead[n];
            if (g == 0)
                *(f32x2 *)(a.part_ml + at * 2) = (f32x2){m[n], l[n]};
            float *o = a.part_o + at * dim + g * (8 * NB);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int j = 0; j < 2 * NB; j += 4)
                    *(f32x4 *)(o + e * 2 * NB + j) =
                        (f32x4){acc[n][j][e], acc[n][j + 1][e], acc[n][j + 2][e], acc[n][j + 3][e]};
        } else {
            const float inv = l[n] == 0.0f ? 0.0f : 1.0f / l[n];
            uint16_t *o = a.out + (int64_t)row[n] * a.out_stride + qhead[n] * dim + g * (8 * NB);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int j = 0; j < 2 * NB; j += 4)
                    *(u32x2 *)(o + e * 2 * NB + j) = (u32x2){pack_bf16(acc[n][j][e] * inv, acc[n][j + 1][e] * inv),
                                                             pack_bf16(acc[n][j + 2][e] * inv, acc[n][j + 3][e] * inv)};
        }
    }
}

// Joins the splits of one row and head: a workgroup of 256 threads, dim / 4
// of them along the channels and the rest along the splits.
template <int NB>
__global__ __launch_bounds__(256) void attention_join_kernel(AttnArgs a, int R)
{
    constexpr int dim = 32 * NB, along = dim / 4, ways = 256 / along;
    const int lane = threadIdx.x & 63;
    const int head = (int)(blockIdx.x % (unsigned)a.q_heads);
    const int row = (int)(blockIdx.x / (unsigned)a.q_heads);
    const int s = wave_search((int)a.b.seqs, row, lane, [&](int i) { return (int64_t)a.b.row_start[i]; });
    const SeqRows q = seq_rows(a.b, s);
    if (row < q.first || row >= q.first + q.rows)
        return;
    const int col = (row - q.first) * a.group + head % a.group;
    TilePlan t;
    plan_tile(a, s, col / R, R, lane, t);
    if (t.splits == 1)
        return;
    const int64_t at0 = (int64_t)row * a.q_heads + head, step = a.b.rows * a.q_heads;
    float m = -__builtin_inff();
    for (int i = lane; i < t.splits; i += 64)
        m = __builtin_fmaxf(m, a.part_ml[(at0 + i * step) * 2]);
#pragma unroll
    for (int x = 32; x >= 1; x >>= 1)
        m = __builtin_fmaxf(m, __shfl_xor(m, x, 64));
    const int d4 = threadIdx.x % along, way = threadIdx.x / along;
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
    float l = 0.0f;
    for (int i = way; i < t.splits; i += ways) {
        const f32x2 ml = *(const f32x2 *)(a.part_ml + (at0 + i * step) * 2);
        const float f = ml[0] == m ? 1.0f : __builtin_amdgcn_exp2f(ml[0] - m);
        o += f * *(const f32x4 *)(a.part_o + (at0 + i * step) * dim + d4 * 4);
        l += f * ml[1];
    }
    __shared__ f32x4 so[256];
    __shared__ float sl[256];
    so[threadIdx.x] = o;
    sl[threadIdx.x] = l;
    __syncthreads();
    if (way)
        return;
#pragma unroll
    for (int w = 1; w < ways; ++w) {
        o += so[w * along + d4];
        l += sl[w * along + d4];
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    *(u32x2 *)(a.out + (int64_t)row * a.out_stride + head * dim + d4 * 4) =
        (u32x2){pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv)};
}

// Columns of a workgroup, and how its waves share them.
struct Shape {
    int nq, wq, R;
    int tiles, splits, wanted;
};

Shape shape_of(int64_t q_heads, const mx_cache &c, const mx_batch &b, int64_t window, int64_t sinks)
{
    Shape s{};
    const int64_t group = q_heads / c.heads, cols = b.rows * group;
    const int64_t mean = (cols + b.seqs - 1) / b.seqs; // columns of a sequence
    s.wq = mean <= 64 ? 1 : kWaves;
    s.nq = mean <= 16 || c.dim == 256 ? 1 : 2;
    s.R = 16 * s.nq * s.wq;
    s.tiles = (int)(cols / s.R + b.seqs);
    s.wanted = (s.wq == 1 ? 4 : 2) * device_cus();
    s.splits = 1;
    const int64_t groups = (int64_t)s.tiles * c.heads;
    if (b.seqs <= kSplitSeqs && 2 * groups <= s.wanted) {
        // tiles of the longest sequence the table can hold
        int64_t span = b.width * c.page_size;
        if (window && window + sinks + b.rows < span)
            span = window + sinks + b.rows;
        const int64_t most = (span / kTile + 2 * kWaves) / (2 * kWaves);
        // twice the mean: the longer sequences of a mixed batch take more
        int64_t n = 2 * (s.wanted / groups);
        n = n < most ? n : most;
        s.splits = (int)(n < 1 ? 1 : n > kMaxSplits ? kMaxSplits : n);
    }
    return s;
}

template <int NB>
hipError_t launch(const AttnArgs &a, const Shape &s, hipStream_t stream)
{
    const int64_t grid = (int64_t)s.tiles * s.splits * a.c.heads;
    if (grid > 0x7FFFFFFF || a.b.rows * a.q_heads > 0x7FFFFFFF)
        return hipErrorInvalidConfiguration;
    const dim3 g((unsigned)grid), w(64 * kWaves);
    constexpr int kMost = NB == 8 ? 1 : 2; // column tiles a wave has registers for
    if (s.wq > 1)
        attention_kernel<NB, kMost, kWaves><<<g, w, 0, stream>>>(a);
    else if (s.nq > 1)
        attention_kernel<NB, kMost, 1><<<g, w, 0, stream>>>(a);
    else
        attention_kernel<NB, 1, 1><<<g, w, 0, stream>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || s.splits == 1)
        return e;
    attention_join_kernel<NB><<<dim3((unsigned)(a.b.rows * a.q_heads)), dim3(256), 0, stream>>>(a, s.R);
    return hipGetLastError();
}

} // namespace

int64_t attention_workspace(int64_t q_heads, const mx_cache &c, const mx_batch &b, int64_t window, int64_t sinks)
{
    const Shape s = shape_of(q_heads, c, b, window, sinks);
    return s.splits == 1 ? 0 : (int64_t)s.splits * b.rows * q_heads * (c.dim + 2) * 4;
}

hipError_t launch_cache_attention(const uint16_t *q, int64_t q_stride, int64_t q_heads, const mx_cache &c,
                                  const mx_batch &b, float scale, int64_t window, int64_t sinks, uint16_t *out,
                                  int64_t out_stride, void *workspace, hipStream_t stream)
{
    const Shape s = shape_of(q_heads, c, b, window, sinks);
    AttnArgs a{};
    a.q = q;
    a.out = out;
    a.part_o = (float *)workspace;
    a.part_ml = a.part_o + (int64_t)s.splits * b.rows * q_heads * c.dim;
    a.q_stride = q_stride;
    a.out_stride = out_stride;
    a.c = c;
    a.b = b;
    a.q_heads = (int)q_heads;
    a.group = (int)(q_heads / c.heads);
    a.window = (int)window;
    a.sinks = (int)sinks;
    a.scale2 = (float)((double)scale * 1.4426950408889634);
    a.splits = s.splits;
    a.wanted = s.wanted;
    a.size16 = (unsigned)(c.page_size / 16);
    a.size_magic = (unsigned)(((uint64_t)1 << 32) / a.size16) + 1;
    a.tiles = s.tiles;
    switch (c.dim) {
    case 64: return launch<2>(a, s, stream);
    case 128: return launch<4>(a, s, stream);
    default: return launch<8>(a, s, stream);
    }
}

} // namespace kq
