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
//
// Softmax: one pass, running maximum and sum.  The maximum used for scaling is
// raised only when a score exceeds it by 2^8 (weights then stay below 2^8,
// sums far below fp32's range), so most tiles need no reduction across lanes
// and no rescaling; the sum is kept per lane and reduced once at the end.
//
// Few columns (attention_few_kernel): the waves of a workgroup take every
// fourth tile and join through LDS.  Many (attention_many_kernel): every wave
// has its own columns, and the converted tiles are shared through LDS.  Where
// workgroups are few, long sequences are also split over them, and a second
// kernel joins the parts.
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

struct AttnArgs {
    const uint16_t *q;
    uint16_t *out;
    float *part_o;  // [parts][dim] unnormalised outputs of columns
    float *part_ml; // [parts][2] their maxima (log2) and sums
    int64_t q_stride, out_stride;
    mx_cache c;
    mx_batch b;
    int q_heads, group;
    int window, sinks;
    float scale2; // scale * log2(e)
    int splits;   // many columns: most splits of a sequence
    int wanted;   // workgroups that fill the chip
    int line;     // few columns: workgroups of a head's line (0: one for each column tile)
    unsigned size16, magic, magic_hi; // page_size / 16; the words of floor(2^32 / size16) + 1
    int tiles;    // column tiles: an upper bound over the batch
};

// Column tile `local` (R columns) of a sequence: its rows and positions, and
// the cache tiles that some column sees: `sink_tiles` first ones, then
// [first_tile, ...), n in all.
struct TilePlan {
    SeqRows seq;
    int cols;         // columns of the sequence
    int pmin, pmax;   // positions of the tile's first and last row
    int span;         // positions that can have a slot
    int sink_tiles, first_tile, n;
};

__device__ __forceinline__ TilePlan plan_tile(const AttnArgs &a, const SeqRows &seq, int local, int R)
{
    TilePlan t;
    t.seq = seq;
    t.cols = seq.rows * a.group;
    const int64_t c0 = (int64_t)local * R;
    const int64_t c1 = c0 + R < t.cols ? c0 + R : t.cols; // one past the last
    t.span = (int)(a.b.width * a.c.page_size);
    t.pmin = (int)(seq.pos0 + c0 / a.group);
    t.pmax = (int)(seq.pos0 + (c1 - 1) / a.group);
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
    return t;
}

// No column tile of a sequence of this length has more cache tiles.
__device__ __forceinline__ int most_tiles(const AttnArgs &a, int64_t len, int R)
{
    const int64_t span = a.b.width * a.c.page_size;
    len = len < 0 ? 0 : len > span ? span : len;
    int64_t n = (len + kTile - 1) / kTile;
    if (a.window) {
        // the window of R / group + 1 rows ends inside a tile on either side
        const int64_t w = ((int64_t)a.window + R / a.group + 1 + kTile - 1) / kTile + 1 + (a.sinks + kTile - 1) / kTile;
        n = w < n ? w : n;
    }
    return (int)n;
}

// The work of one workgroup: cache tiles [begin, stop) of a column tile's
// plan, and where its columns go: to the output (part < 0), or as rows part,
// part + 1, ... of the partial results.
struct Place {
    int head, s, local;
    TilePlan t;
    int begin, stop;
    int64_t part;
};

// The partial results of a column tile: part i starts at row base + i stride,
// part 0 `extra` rows later.
struct Parts {
    int count;
    int64_t base, stride, extra;
};

// Column tile -> sequence and its local number: the tiles of sequence s start
// at row_start[s] group / R + s, which leaves it at least ceil(columns / R).
// False: the sequence has no such tile.
__device__ __forceinline__ bool find_tile(const AttnArgs &a, int R, int tile, int lane, Place &w)
{
    auto first_of = [&](int s) {
        const int64_t r = a.b.row_start[s];
        return (r < 0 ? 0 : r) * a.group / R + s;
    };
    w.s = wave_search((int)a.b.seqs, tile, lane, first_of);
    const int64_t local = tile - first_of(w.s);
    const SeqRows q = seq_rows(a.b, w.s);
    if (local < 0 || local * R >= (int64_t)q.rows * a.group)
        return false;
    w.local = (int)local;
    w.t = plan_tile(a, q, w.local, R);
    return true;
}

// ---- many columns: a workgroup for each column tile, head and split -------
// Cache tiles of one split: the batch's tiles over the workgroups wanted, at
// least two per wave.  Every wave of both kernels gets the same answer.
__device__ __forceinline__ int split_tiles(const AttnArgs &a, int R, int lane)
{
    float sum = 0.0f;
    for (int s = lane; s < a.b.seqs; s += 64)
        sum += (float)most_tiles(a, a.b.lengths[s], R);
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1)
        sum += __shfl_xor(sum, m, 64);
    // each sequence has about tiles / seqs column tiles for every head
    const float units = sum * (float)a.tiles / (float)a.b.seqs * (float)a.c.heads;
    const int per = (int)(units / (float)a.wanted) + 1;
    return __builtin_amdgcn_readfirstlane(per < 2 * kWaves ? 2 * kWaves : per);
}

__device__ __forceinline__ Parts split_parts(const AttnArgs &a, int R, int tile, int head, int n, int lane,
                                             int &per_split)
{
    Parts p{1, 0, 0, 0};
    per_split = n;
    if (a.splits > 1 && n > 0) {
        const int per = split_tiles(a, R, lane);
        const int want = (n + per - 1) / per;
        p.count = want < a.splits ? want : a.splits;
        per_split = (n + p.count - 1) / p.count;
        p.count = (n + per_split - 1) / per_split;
    }
    p.base = ((int64_t)tile * a.c.heads + head) * R;
    p.stride = (int64_t)a.tiles * a.c.heads * R;
    return p;
}

// Workgroup -> (split, column tile, head), the head fastest: the eight XCDs
// take workgroups in turn, so a head's cache stays in few L2s.  The last
// column tiles, whose rows see most, start first.  False: nothing to do.
__device__ __forceinline__ bool find_many(const AttnArgs &a, int R, int lane, Place &w)
{
    const int heads = (int)a.c.heads;
    int id = (int)blockIdx.x;
    w.head = id % heads;
    id /= heads;
    const int split = id % a.splits, tile = a.tiles - 1 - id / a.splits;
    if (!find_tile(a, R, tile, lane, w))
        return false;
    int per = 0;
    const Parts p = split_parts(a, R, tile, w.head, w.t.n, lane, per);
    if (split >= p.count)
        return false;
    w.begin = split * per;
    w.stop = w.begin + per < w.t.n ? w.begin + per : w.t.n;
    w.part = p.count > 1 ? p.base + split * p.stride : -1;
    return true;
}

// ---- few columns: equal shares of a line ----------------------------------
// The cache tiles of all column tiles of all sequences, one after the other,
// are cut into equal shares, one for each of a head's workgroups: a share ends
// inside a column tile wherever it does, so lengths do not have to match for
// the chip to be filled evenly.  A workgroup has at most one column tile that
// began before its share and one that goes on after it, so it needs two
// places for partial results: 2 p and 2 p + 1.  Where no sequence has more than
// kWhole tiles, a column tile counts as one and is not cut.
//
// The arrays of the batch are read once, together, and kept in LDS.
constexpr int kLineSeqs = 256;
constexpr int kWhole = 12 * kWaves; // a join costs about as much as 12 tiles of a wave

struct LineSeq {
    int64_t at;            // where the sequence starts in the line
    int first, rows, len;  // its rows
    int per;               // tiles of one of its column tiles
};

struct Line {
    const LineSeq *seq;
    int64_t share, end;
    int seqs, lane;
    bool whole;

    // Every wave of the workgroup takes part; each writes the same to `to`
    // (whole groups of 64 sequences), which is read after the barrier here.
    __device__ __forceinline__ void build(const AttnArgs &a, int R, int lane_, LineSeq *to)
    {
        seq = to;
        seqs = (int)a.b.seqs;
        lane = lane_;
        LineSeq v[kLineSeqs / 64];
        int most = 0;
#pragma unroll
        for (int k = 0; k < kLineSeqs / 64; ++k) {
            const int s = 64 * k + lane;
            v[k] = {0, 0, 0, 0, 0};
            if (s < seqs) {
                const int64_t b = a.b.row_start[s], e = a.b.row_start[s + 1];
                v[k].len = a.b.lengths[s] < 0 ? 0 : a.b.lengths[s];
                const bool ok = b >= 0 && b < e && e <= a.b.rows;
                v[k].first = ok ? (int)b : 0;
                v[k].rows = ok ? (int)(e - b) : 0;
                const int n = most_tiles(a, v[k].len, R);
                v[k].per = n < 1 ? 1 : n;
                most = ok && v[k].per > most ? v[k].per : most;
            }
        }
        whole = __builtin_amdgcn_ballot_w64(most > kWhole) == 0;
        end = 0;
#pragma unroll
        for (int k = 0; k < kLineSeqs / 64; ++k) {
            if (64 * k >= seqs)
                continue;
            if (whole)
                v[k].per = 1;
            const int64_t all = (((int64_t)v[k].rows * a.group + R - 1) / R) * v[k].per;
            int64_t sum = all;
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) {
                const int64_t up = __shfl_up(sum, m, 64);
                sum += lane >= m ? up : 0;
            }
            v[k].at = end + sum - all;
            end += __shfl(sum, 63, 64);
            to[64 * k + lane] = v[k];
        }
        end = lane64(end);
        share = (end + a.line - 1) / a.line;
        const int64_t least = whole ? 1 : 2 * kWaves;
        share = share < least ? least : share;
        __syncthreads();
    }

    static __device__ __forceinline__ int64_t lane64(int64_t v)
    {
        return (int64_t)((uint64_t)(unsigned)__builtin_amdgcn_readfirstlane((int)v) |
                         (uint64_t)(unsigned)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32);
    }

    // A sequence's entry, the same in all lanes.
    __device__ __forceinline__ LineSeq of(int s) const
    {
        const LineSeq v = seq[s];
        return {lane64(v.at), __builtin_amdgcn_readfirstlane(v.first), __builtin_amdgcn_readfirstlane(v.rows),
                __builtin_amdgcn_readfirstlane(v.len), __builtin_amdgcn_readfirstlane(v.per)};
    }

    // The sequence that place x of the line belongs to: the last that starts
    // there or before (an empty one starts where the next one does).
    __device__ __forceinline__ int find(int64_t x) const
    {
        int n = 0;
        for (int k = 0; 64 * k < seqs; ++k)
            n += __popcll(__builtin_amdgcn_ballot_w64(64 * k + lane < seqs && seq[64 * k + lane].at <= x));
        return n - 1;
    }
};

// Largest of the four lane groups, in all of them.
__device__ __forceinline__ float max_groups(float v)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = vmax(__uint_as_float(r[0]), __uint_as_float(r[1]));
    const auto t = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return vmax(__uint_as_float(t[0]), __uint_as_float(t[1]));
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

// A wave's columns: queries, what each column sees, running sums.
template <int NB, int kNQ>
struct Columns {
    bf16x8 Q[kNQ][NB];
    f32x4 acc[kNQ][2 * NB];
    float m[kNQ], l[kNQ];     // scaling maximum (log2), and the lane's part of the sum
    int pos[kNQ], low[kNQ];   // the column sees [low, pos] and the first `sinks`
    int row[kNQ], qhead[kNQ];
    bool live[kNQ];           // not a padding column
    // positions of the wave's first and last column, and one past what it sees
    int wmin, wmax, whi;
    bool idle;                // padding columns only
};

template <int NB, int kNQ>
__device__ __forceinline__ void load_columns(const AttnArgs &a, const Place &w, int col0, int c, int g,
                                             Columns<NB, kNQ> &q)
{
    const TilePlan &t = w.t;
#pragma unroll
    for (int n = 0; n < kNQ; ++n) {
        const int col = col0 + n * 16 + c;
        q.live[n] = col < t.cols;
        const int at = q.live[n] ? col : 0, i = at / a.group;
        q.row[n] = t.seq.first + i;
        q.qhead[n] = w.head * a.group + at - i * a.group;
        q.pos[n] = q.live[n] ? (int)(t.seq.pos0 + i) : -1;
        q.low[n] = a.window && q.live[n] ? q.pos[n] - a.window + 1 : -0x7FFFFFFF;
        const uint16_t *src = a.q + (int64_t)q.row[n] * a.q_stride + q.qhead[n] * (32 * NB) + g * (8 * NB);
#pragma unroll
        for (int p = 0; p < NB; ++p) {
            u32x4 v = *(const u32x4 *)(src + 8 * p);
            if (!q.live[n])
                v = (u32x4){0, 0, 0, 0};
            q.Q[n][p] = __builtin_bit_cast(bf16x8, v);
        }
        q.m[n] = -__builtin_inff();
        q.l[n] = 0.0f;
#pragma unroll
        for (int j = 0; j < 2 * NB; ++j)
            q.acc[n][j] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
    }
    const int last = (col0 + kNQ * 16 < t.cols ? col0 + kNQ * 16 : t.cols) - 1;
    q.idle = col0 >= t.cols;
    q.wmin = (int)(t.seq.pos0 + col0 / a.group);
    q.wmax = (int)(t.seq.pos0 + last / a.group);
    q.whi = q.idle || q.wmax < 0 ? 0 : q.wmax + 1 < t.span ? q.wmax + 1 : t.span;
}

// Does every column of the wave see all of [j0, j0 + 32)?
template <int NB, int kNQ>
__device__ __forceinline__ bool sees_all(const AttnArgs &a, const Columns<NB, kNQ> &q, int j0, int span)
{
    return j0 + kTile <= q.wmin + 1 && j0 + kTile <= span && !q.idle &&
           (!a.window || j0 >= q.wmax - a.window + 1 || j0 + kTile <= a.sinks);
}

// Scores of what a column does not see become -infinity; `seen` gets the
// positions (k slot 4h + i: position 16h + 4g + i of the tile) that it sees.
template <int NB, int kNQ>
__device__ __forceinline__ void mask_scores(const AttnArgs &a, const Columns<NB, kNQ> &q, int j0, int span,
                                            const bool (&there)[2], int g, f32x4 (&S)[kNQ][2], unsigned (&seen)[kNQ])
{
#pragma unroll
    for (int n = 0; n < kNQ; ++n) {
        seen[n] = 0;
        const int hi = q.pos[n] < span ? q.pos[n] + 1 : span;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int h = k >> 2, j = j0 + 16 * h + 4 * g + (k & 3);
            const bool see = (int)(j < hi) & ((int)(j >= q.low[n]) | (int)(j < a.sinks)) & (int)there[h];
            seen[n] |= (unsigned)see << k;
            S[n][h][k & 3] = see ? S[n][h][k & 3] : -__builtin_inff();
        }
    }
}

// Scores -> bf16 weights as the next product's column operand; raises the
// running maximum (and rescales) only where a score passes it by 2^kRaise.
template <int NB, int kNQ>
__device__ __forceinline__ void weigh(const AttnArgs &a, Columns<NB, kNQ> &q, const f32x4 (&S)[kNQ][2],
                                      bf16x8 (&P)[kNQ])
{
    bool raise = false;
    float top[kNQ];
#pragma unroll
    for (int n = 0; n < kNQ; ++n) {
        float x = vmax(vmax(S[n][0][0], S[n][0][1]), S[n][0][2]);
        x = vmax(vmax(x, S[n][0][3]), S[n][1][0]);
        x = vmax(vmax(x, S[n][1][1]), vmax(S[n][1][2], S[n][1][3]));
        top[n] = x * a.scale2; // a NaN raises nothing, and reaches the sums as a weight
        raise |= top[n] > q.m[n] + kRaise;
    }
    if (__builtin_amdgcn_ballot_w64(raise)) {
#pragma unroll
        for (int n = 0; n < kNQ; ++n) {
            const float up = vmax(q.m[n], max_groups(top[n]));
            const float f = up == q.m[n] ? 1.0f : __builtin_amdgcn_exp2f(q.m[n] - up);
            q.m[n] = up;
            q.l[n] *= f;
#pragma unroll
            for (int j = 0; j < 2 * NB; ++j)
                q.acc[n][j] *= f;
        }
    }
#pragma unroll
    for (int n = 0; n < kNQ; ++n) {
        const float base = q.m[n] == -__builtin_inff() ? 0.0f : q.m[n];
        float w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            w[k] = __builtin_amdgcn_exp2f(__builtin_fmaf(S[n][k >> 2][k & 3], a.scale2, -base));
        q.l[n] += ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
        const u32x4 pk = {pack_bf16(w[0], w[1]), pack_bf16(w[2], w[3]), pack_bf16(w[4], w[5]), pack_bf16(w[6], w[7])};
        P[n] = __builtin_bit_cast(bf16x8, pk);
    }
}

// Two bits of a slot mask -> bf16 1.0 / 0.0, for the NaN counts.
__device__ __forceinline__ bf16x8 ones(unsigned bits)
{
    u32x4 v;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        v[k] = ((bits >> (2 * k) & 1u) * 0x3F80u) | ((bits >> (2 * k + 1) & 1u) * 0x3F800000u);
    return __builtin_bit_cast(bf16x8, v);
}

// A weight of zero does not hide a NaN of V, so a NaN that only some columns
// see is taken out of the product, and counted per channel row (ind) and
// column (seen) by one of its own: where the count is not zero the channel
// becomes NaN.
__device__ __forceinline__ void spoil(f32x4 &acc, const f32x4 &count)
{
#pragma unroll
    for (int e = 0; e < 4; ++e)
        acc[e] = count[e] > 0.0f ? __builtin_nanf("") : acc[e];
}

// Writes the columns' results, or their parts; col0: the wave's first column in the workgroup's tile.  The lane's channels are [8 NB
// g, 8 NB (g + 1)): channel 2 NB e + j of them is acc[j][e].
template <int NB, int kNQ>
__device__ __forceinline__ void store_columns(const AttnArgs &a, const Place &w, const Columns<NB, kNQ> &q, int col0,
                                              int c, int g)
{
    constexpr int dim = 32 * NB;
#pragma unroll
    for (int n = 0; n < kNQ; ++n) {
        if (!q.live[n])
            continue;
        if (w.part >= 0) {
            const int64_t at = w.part + col0 + n * 16 + c;
            if (g == 0)
                *(f32x2 *)(a.part_ml + at * 2) = (f32x2){q.m[n], q.l[n]};
            float *o = a.part_o + at * dim + g * (8 * NB);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int j = 0; j < 2 * NB; j += 4)
                    *(f32x4 *)(o + e * 2 * NB + j) =
                        (f32x4){q.acc[n][j][e], q.acc[n][j + 1][e], q.acc[n][j + 2][e], q.acc[n][j + 3][e]};
        } else {
            const float inv = q.l[n] == 0.0f ? 0.0f : 1.0f / q.l[n];
            uint16_t *o = a.out + (int64_t)q.row[n] * a.out_stride + q.qhead[n] * dim + g * (8 * NB);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int j = 0; j < 2 * NB; j += 4)
                    *(u32x2 *)(o + e * 2 * NB + j) =
                        (u32x2){pack_bf16(q.acc[n][j][e] * inv, q.acc[n][j + 1][e] * inv),
                                pack_bf16(q.acc[n][j + 2][e] * inv, q.acc[n][j + 3][e] * inv)};
        }
    }
}

// Walks a sequence's pages in tiles of 32 positions, as one wave takes them:
// tile indices first, first + step, ... below stop, both halves of a tile
// (kHalves = 2) or only half `part`.  A half (16 positions) lies in one page.
// Page numbers are fetched 64 halves at a time, one to a lane, one such window
// ahead, and handed out by lane: a fetch per tile would have to be waited for
// in the middle of the loop, and with it everything that is in flight.
template <int kHalves>
struct Pages {
    static constexpr int kWindow = 64 / kHalves; // tiles
    const int32_t *table;
    int span, pages, size, lane;
    unsigned size16, magic, magic_hi;
    unsigned page_codes, page_scales;         // bytes of a page
    const uint8_t *kq, *ks, *vq, *vs;         // of this head in page 0
    int sink_tiles, skip;                     // tile index -> tile
    int first, step, stop, part;
    int now, next;                            // this lane's page numbers of two windows
    int at_tile;                              // tiles taken so far

    __device__ __forceinline__ Pages(const AttnArgs &a, const Place &w, int lane_, int first_, int step_, int part_)
        : table(a.b.page_table + (int64_t)w.s * a.b.width), span(w.t.span), pages((int)a.c.pages),
          size((int)a.c.page_size), lane(lane_), size16(a.size16), magic(a.magic), magic_hi(a.magic_hi),
          sink_tiles(w.t.sink_tiles), skip(w.t.first_tile - w.t.sink_tiles), first(first_), step(step_), stop(w.stop),
          part(part_)
    {
        const unsigned head_codes = (unsigned)size * (unsigned)(a.c.dim / 2); // below 2^18; a page below 2^28
        const unsigned head_scales = (unsigned)size * (unsigned)(a.c.dim / 32);
        page_codes = (unsigned)a.c.heads * head_codes;
        page_scales = (unsigned)a.c.heads * head_scales;
        kq = a.c.kq + w.head * head_codes;
        vq = a.c.vq + w.head * head_codes;
        ks = a.c.ks + w.head * head_scales;
        vs = a.c.vs + w.head * head_scales;
        at_tile = 0;
        now = fetch(0);
        next = fetch(kWindow);
    }

    __device__ __forceinline__ int tile(int i) const { return i < sink_tiles ? i : i + skip; }

    // u / size16 by multiplication: u < 2^26 and size16 <= 64, so the
    // product's excess over u / size16 2^32 stays below 2^32
    __device__ __forceinline__ unsigned page_of(unsigned u) const { return __umulhi(u, magic) + u * magic_hi; }

    // Page number of the lane's half in the window of the walk that starts at tile `from`
    // (the last tile's past its end), -1 past the table.
    __device__ __forceinline__ int fetch(int from) const
    {
        const int64_t i = first + (int64_t)step * (from + lane / kHalves);
        const unsigned u = (unsigned)(2 * tile(i < stop ? (int)i : stop - 1) + (kHalves == 2 ? lane & 1 : part));
        return stop > 0 && (int)(16 * u) < span ? table[page_of(u)] : -1;
    }

    // The page numbers of the next tile of the walk.
    __device__ __forceinline__ void take(int (&page)[kHalves])
    {
        if (at_tile == kWindow) {
            now = next;
            first += kWindow * step;
            next = fetch(kWindow);
            at_tile = 0;
        }
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
            page[h] = __builtin_amdgcn_readlane(now, kHalves * at_tile + h);
        ++at_tile;
    }

    // Byte offsets of a half's codes and scales in the head's arrays (those of
    // page 0 where it has no page).
    __device__ __forceinline__ bool at(int i, int h, int page, unsigned half_row, uint64_t &codes,
                                       uint64_t &scales) const
    {
        const unsigned u = (unsigned)(2 * tile(i) + h);
        const unsigned off = 16 * (u - page_of(u) * size16);
        const bool there = page >= 0 && page < pages;
        const unsigned pg = there ? (unsigned)page : 0u;
        codes = (uint64_t)pg * page_codes + off * half_row;
        scales = (uint64_t)pg * page_scales + off;
        return there;
    }
};

// Raw codes and scales of one tile, as one lane reads them.
template <int NB>
struct RawTile {
    static constexpr int kVW = NB == 8 ? 2 : 1; // dwords of a V piece
    unsigned k[2][NB];
    unsigned ks[2][NB == 8 ? 2 : 1];
    unsigned v[8][kVW]; // k slots: positions 4g + i, 16 + 4g + i
    unsigned vs[2];
};

// Codes of position c's channels [8 NB g, 8 NB (g + 1)) and their scales.
template <int NB, class P>
__device__ __forceinline__ void load_keys(const P &pages, uint64_t codes, uint64_t scales, int c, int g,
                                          unsigned (&k)[NB], unsigned (&ks)[NB == 8 ? 2 : 1])
{
    const int size = pages.size;
    const uint8_t *src = pages.kq + codes + (unsigned)(c * (NB * 16) + g * (NB * 4));
    if constexpr (NB == 2) {
        const u32x2 w = *(const u32x2 *)src;
        k[0] = w[0];
        k[1] = w[1];
    } else {
#pragma unroll
        for (int i = 0; i < NB / 4; ++i) {
            const u32x4 w = *(const u32x4 *)(src + 16 * i);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                k[4 * i + j] = w[j];
        }
    }
    const int blk = NB == 8 ? 2 * g : NB == 4 ? g : g >> 1;
    const uint8_t *sc = pages.ks + scales + (unsigned)(blk * size + c);
    ks[0] = sc[0];
    if constexpr (NB == 8)
        ks[1] = sc[size];
}

// Codes of channels [2 NB c, 2 NB (c + 1)) of one position.
template <int NB>
__device__ __forceinline__ void load_value(const uint8_t *src, unsigned (&v)[NB == 8 ? 2 : 1])
{
    if constexpr (NB == 2) {
        v[0] = *(const uint16_t *)src;
    } else if constexpr (NB == 4) {
        v[0] = *(const unsigned *)src;
    } else {
        const u32x2 w = *(const u32x2 *)src;
        v[0] = w[0];
        v[1] = w[1];
    }
}

// Byte b of a dword of codes -> the two channels as packed bf16.
__device__ __forceinline__ unsigned cvt_byte(unsigned raw, float sc, int b)
{
    bf16x2 v;
    switch (b) { // the byte is part of the instruction
    case 0: v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(raw, sc, 0); break;
    case 1: v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(raw, sc, 1); break;
    case 2: v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(raw, sc, 2); break;
    default: v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(raw, sc, 3); break;
    }
    return __builtin_bit_cast(unsigned, v);
}

// (channel 2b, channel 2b + 1) of two positions -> each channel's two positions.
__device__ __forceinline__ unsigned even_of(unsigned w0, unsigned w1) { return __builtin_amdgcn_perm(w1, w0, 0x05040100u); }
__device__ __forceinline__ unsigned odd_of(unsigned w0, unsigned w1) { return __builtin_amdgcn_perm(w1, w0, 0x07060302u); }

// Few columns (NB = dim / 32; kNQ tiles of 16): every wave has the same
// columns and takes every kW-th cache tile.  What bounds it is reading the
// cache, so each wave keeps kD - 1 tiles in flight, loaded straight into LDS
// (no registers, whole 16-byte pieces, 17 NB / 16 KB a tile) in the order in
// which its lanes read them: the k-th 16-byte piece of a load goes to the
// k-th place, so the order is chosen by the address that each lane loads
// from.  A wave reads only what it loaded: no barrier.
//
// A stage: K pieces (half h, piece pc of a position, position c), V pieces
// (h, i, g, piece) of position 4g + i, then dwords of scale bytes (K or V, h,
// block, four positions).
template <int NB>
struct FewStage {
    static constexpr int kPieces = 32 * NB;         // of K, and of V
    static constexpr int kDwords = 16 * NB;         // of scales
    static constexpr int kScalePad = kDwords < 64 ? 64 : kDwords;
    static constexpr int kVAt = kPieces * 16, kSAt = 2 * kPieces * 16;
    static constexpr int kBytes = kSAt + kScalePad * 4;
    static constexpr int kLoads = 2 * kPieces / 64 + kScalePad / 64; // instructions of a tile
};

typedef __attribute__((address_space(3))) void lds_void;
typedef const __attribute__((address_space(1))) void global_void;

template <int NB>
__device__ __forceinline__ void load_stage(const Pages<2> &pages, int i, const int (&page)[2], int lane,
                                           unsigned char *st, bool (&there)[2])
{
    using L = FewStage<NB>;
    uint64_t codes[2], scales[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
        there[h] = pages.at(i, h, page[h], 16 * NB, codes[h], scales[h]);
#pragma unroll
    for (int k = 0; k < L::kPieces / 64; ++k) {
        const int u = 64 * k + lane, c = u % 16, pc = u / 16 % NB, h = u / (16 * NB);
        __builtin_amdgcn_global_load_lds((global_void *)(pages.kq + (h ? codes[1] : codes[0]) + c * (16 * NB) + pc * 16),
                                         (lds_void *)(st + k * 1024), 16, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < L::kPieces / 64; ++k) {
        const int u = 64 * k + lane, pc = u % NB, g = u / NB % 4, x = u / (4 * NB) % 4, h = u / (16 * NB);
        __builtin_amdgcn_global_load_lds(
            (global_void *)(pages.vq + (h ? codes[1] : codes[0]) + (4 * g + x) * (16 * NB) + pc * 16),
            (lds_void *)(st + L::kVAt + k * 1024), 16, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < L::kScalePad / 64; ++k) {
        const int u = (64 * k + lane) % L::kDwords, t4 = u % 4, blk = u / 4 % NB, h = u / (4 * NB) % 2, v = u / (8 * NB);
        __builtin_amdgcn_global_load_lds(
            (global_void *)((v ? pages.vs : pages.ks) + (h ? scales[1] : scales[0]) + blk * pages.size + 4 * t4),
            (lds_void *)(st + L::kSAt + k * 256), 4, 0, 0);
    }
}

// A stage into the lane's registers.
template <int NB>
__device__ __forceinline__ void read_stage(const unsigned char *st, int c, int g, RawTile<NB> &r)
{
    using L = FewStage<NB>;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if constexpr (NB == 2) {
            const u32x2 w = *(const u32x2 *)(st + ((h * NB + g / 2) * 16 + c) * 16 + 8 * (g & 1));
            r.k[h][0] = w[0];
            r.k[h][1] = w[1];
        } else {
#pragma unroll
            for (int e = 0; e < NB / 4; ++e) {
                const u32x4 w = *(const u32x4 *)(st + ((h * NB + g * (NB / 4) + e) * 16 + c) * 16);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    r.k[h][4 * e + j] = w[j];
            }
        }
        const int blk = NB == 8 ? 2 * g : NB == 4 ? g : g >> 1;
        r.ks[h][0] = st[L::kSAt + (h * NB + blk) * 16 + c];
        if constexpr (NB == 8)
            r.ks[h][1] = st[L::kSAt + (h * NB + blk + 1) * 16 + c];
#pragma unroll
        for (int x = 0; x < 4; ++x)
            load_value<NB>(st + L::kVAt + (((h * 4 + x) * 4 + g) * (16 * NB) + c * NB), r.v[4 * h + x]);
        r.vs[h] = *(const unsigned *)(st + L::kSAt + ((2 + h) * NB + NB * c / 16) * 16 + 4 * g);
    }
}

// Bytes of LDS for the rings, or the join of the waves in the same place.
template <int NB, int kNQ, int kW, int kD>
__host__ __device__ constexpr int few_lds()
{
    constexpr int ring = kW * kD * FewStage<NB>::kBytes, join = kW * kNQ * (2 * NB * 64 * 16 + 2 * 16 * 4);
    return ring > join ? ring : join;
}

// One workgroup's cache tiles of a column tile.
template <int NB, int kNQ, int kW, int kD>
__device__ __forceinline__ void attention_few(const AttnArgs &a, const Place &w, int lane, int wave,
                                              unsigned char *lds)
{
    using L = FewStage<NB>;
    constexpr int R = 16 * kNQ;
    const int c = lane & 15, g = lane >> 4;
    int i = w.begin + wave;
    Pages<2> pages(a, w, lane, i, kW, 0);
    unsigned char *ring = lds + wave * (kD * L::kBytes);
    bool there[kD][2];
    auto load = [&](int at, int z) {
        int page[2];
        pages.take(page);
        load_stage<NB>(pages, at < w.stop ? at : w.stop - 1, page, lane, ring + z * L::kBytes, there[z]);
    };
    if (i < w.stop) {
#pragma unroll
        for (int z = 0; z < kD - 1; ++z)
            load(i + z * kW, z);
    }
    Columns<NB, kNQ> q;
    load_columns<NB, kNQ>(a, w, w.local * R, c, g, q);

    auto tile = [&](int at, const bool (&has)[2], const unsigned char *st) {
        RawTile<NB> r;
        read_stage<NB>(st, c, g, r);
        const int j0 = pages.tile(at) * kTile;
        const bool full = has[0] && has[1] && sees_all<NB, kNQ>(a, q, j0, w.t.span);

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
                    S[n][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, q.Q[n][p], S[n][h], 0, 0, 0);
            }
        }

        // scale bytes of the lane's eight positions of V
        unsigned vsb[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            vsb[k] = (r.vs[k >> 2] >> (8 * (k & 3))) & 0xFFu;
        unsigned nan_slots = 0, seen[kNQ];
        if (!full) {
            mask_scores<NB, kNQ>(a, q, j0, w.t.span, has, g, S, seen);
            // positions that no column sees (past the last one, or never
            // written) are cleared: a weight of zero would not hide what they
            // hold.  NaN blocks are cleared too and counted below.
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int h = k >> 2, j = j0 + 16 * h + 4 * g + (k & 3);
                const bool dead = j >= q.whi || !has[h];
                const bool nan = vsb[k] == 0xFFu && !dead;
                nan_slots |= (unsigned)nan << k;
                if (dead || nan) {
                    vsb[k] = 127;
#pragma unroll
                    for (int x = 0; x < RawTile<NB>::kVW; ++x)
                        r.v[k][x] = 0;
                }
            }
        }
        bf16x8 P[kNQ];
        weigh<NB, kNQ>(a, q, S, P);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            unsigned v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[k] = cvt_byte(r.v[k][NB == 8 ? b / 4 : 0], scale_operand(vsb[k]), b & 3);
            u32x4 even, odd;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                even[k] = even_of(v[2 * k], v[2 * k + 1]);
                odd[k] = odd_of(v[2 * k], v[2 * k + 1]);
            }
#pragma unroll
            for (int n = 0; n < kNQ; ++n) {
                q.acc[n][2 * b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, even), P[n],
                                                                          q.acc[n][2 * b], 0, 0, 0);
                q.acc[n][2 * b + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, odd), P[n],
                                                                              q.acc[n][2 * b + 1], 0, 0, 0);
            }
        }
        // the channels of a lane share a block, so one count serves them all
        if (!full && __builtin_amdgcn_ballot_w64(nan_slots != 0)) {
#pragma unroll
            for (int n = 0; n < kNQ; ++n) {
                const f32x4 count = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    ones(nan_slots), ones(seen[n]), (f32x4){0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
#pragma unroll
                for (int j = 0; j < 2 * NB; ++j)
                    spoil(q.acc[n][j], count);
            }
        }
    };

    // s_waitcnt vmcnt: the loads of the kD - 1 younger tiles may be in flight
    // (page numbers fetched in between only make it wait for more)
    constexpr int kYounger = (kD - 1) * L::kLoads;
    static_assert(kYounger < 64, "vmcnt has six bits");
    constexpr unsigned kWait = 0x0F70u | (kYounger & 15) | ((kYounger >> 4) << 14);
    while (i < w.stop) {
#pragma unroll
        for (int z = 0; z < kD; ++z) {
            if (i >= w.stop)
                break;
            // the stage that was read last is loaded again, once its reads have
            // arrived; nothing moves across the empty asm
            __builtin_amdgcn_s_waitcnt(0xC07Fu); // lgkmcnt(0) alone
            asm volatile("" ::: "memory");
            load(i + (kD - 1) * kW, (z + kD - 1) % kD);
            __builtin_amdgcn_s_waitcnt(kWait);
            asm volatile("" ::: "memory");
            tile(i, there[z], ring + z * L::kBytes);
            i += kW;
        }
    }

    // sums over the lane groups, then over the waves, through the ring (after
    // what is still in flight into it)
    __builtin_amdgcn_s_waitcnt(0x0F70u);
    f32x4 *so = (f32x4 *)lds;                               // [kW][kNQ][2 NB][64]
    float *sm = (float *)(so + kW * kNQ * 2 * NB * 64);     // [kW][kNQ][16], and the sums after it
    float *sl = sm + kW * kNQ * 16;
#pragma unroll
    for (int n = 0; n < kNQ; ++n)
        q.l[n] = sum_groups(q.l[n]);
    __syncthreads();
    if (g == 0) {
#pragma unroll
        for (int n = 0; n < kNQ; ++n) {
            sm[(wave * kNQ + n) * 16 + c] = q.m[n];
            sl[(wave * kNQ + n) * 16 + c] = q.l[n];
        }
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < kNQ; ++n) {
        float up = sm[n * 16 + c];
#pragma unroll
        for (int x = 1; x < kW; ++x)
            up = vmax(up, sm[(x * kNQ + n) * 16 + c]);
        float sum = 0.0f;
#pragma unroll
        for (int x = 0; x < kW; ++x) {
            const float mx = sm[(x * kNQ + n) * 16 + c];
            sum += sl[(x * kNQ + n) * 16 + c] * (mx == up ? 1.0f : __builtin_amdgcn_exp2f(mx - up));
        }
        const float f = q.m[n] == up ? 1.0f : __builtin_amdgcn_exp2f(q.m[n] - up);
        q.m[n] = up;
        q.l[n] = sum;
#pragma unroll
        for (int j = 0; j < 2 * NB; ++j) {
            q.acc[n][j] *= f;
            if (wave)
                so[((wave * kNQ + n) * 2 * NB + j) * 64 + lane] = q.acc[n][j];
        }
    }
    __syncthreads();
    if (wave)
        return; // to the caller's barrier
#pragma unroll
    for (int n = 0; n < kNQ; ++n)
#pragma unroll
        for (int j = 0; j < 2 * NB; ++j)
#pragma unroll
            for (int x = 1; x < kW; ++x)
                q.acc[n][j] += so[((x * kNQ + n) * 2 * NB + j) * 64 + lane];
    store_columns<NB, kNQ>(a, w, q, 0, c, g);
}

template <int NB, int kNQ, int kW, int kD>
__global__ __launch_bounds__(64 * kW, 2) void attention_few_kernel(AttnArgs a)
{
    constexpr int R = 16 * kNQ;
    extern __shared__ __align__(16) unsigned char lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int heads = (int)a.c.heads, p = (int)blockIdx.x / heads;
    Place w;
    w.head = (int)blockIdx.x % heads;
    if (a.line == 0) { // more sequences than a line holds: a column tile each
        if (!find_tile(a, R, a.tiles - 1 - p, lane, w))
            return;
        w.begin = 0;
        w.stop = w.t.n;
        w.part = -1;
    }
    Line line;
    int64_t begin = 0, end = 1;
    if (a.line) {
        line.build(a, R, lane, (LineSeq *)(lds + few_lds<NB, kNQ, kW, kD>()));
        begin = p * line.share;
        end = begin + line.share < line.end ? begin + line.share : line.end;
    }
    for (int64_t x = begin; x < end;) {
        int64_t next = end;
        if (a.line) {
            w.s = line.find(x);
            const LineSeq q = line.of(w.s);
            w.local = (int)((x - q.at) / q.per);
            const int64_t tile = q.at + (int64_t)w.local * q.per; // the column tile's first place in the line
            next = tile + q.per < end ? tile + q.per : end;
            w.t = plan_tile(a, {q.first, q.rows, (int64_t)q.len - q.rows}, w.local, R);
            w.begin = line.whole ? 0 : (int)(x - tile) < w.t.n ? (int)(x - tile) : w.t.n;
            w.stop = line.whole ? w.t.n : (int)(next - tile) < w.t.n ? (int)(next - tile) : w.t.n;
            const bool all = x == tile && next == tile + q.per;
            w.part = all ? -1 : ((int64_t)(2 * p + (tile >= begin ? 1 : 0)) * heads + w.head) * R;
        }
        attention_few<NB, kNQ, kW, kD>(a, w, lane, wave, lds);
        x = next;
        __syncthreads(); // the join is done with the ring
    }
}

// Many columns: the waves have columns of their own and share the cache tiles
// through LDS, 64 positions at a time in two stages, already converted: each
// wave converts a quarter, in the order in which the products read it (one
// 16-byte piece per lane and operand).  Per wave and 32 positions that
// leaves a quarter of the conversions (24 of 96 vector instructions at dim
// 128) next to its own softmax.
template <int NB>
struct __align__(16) WideStage {
    u32x4 k[kWaves][NB][64];        // 16 positions each
    u32x2 v[2][2 * NB][64][2];      // 32 positions each, a half in 8 bytes
    unsigned flags[kWaves];         // of the wave that wrote: 1 some of nan is set, 2 its half has a page
    unsigned char nan[kWaves][64];  // per lane: the slots whose V block was NaN (stored as zeros)
};

template <int NB, int kNQ>
__global__ __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(2, 2))) void attention_many_kernel(AttnArgs a)
{
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    constexpr int R = 16 * kNQ * kWaves;
    extern __shared__ __align__(16) unsigned char lds[];
    WideStage<NB> *stage = (WideStage<NB> *)lds;
    Place w;
    if (!find_many(a, R, lane, w))
        return;
    Columns<NB, kNQ> q;
    load_columns<NB, kNQ>(a, w, w.local * R + wave * kNQ * 16, c, g, q);
    const int end = w.t.pmax < 0 ? 0 : w.t.pmax + 1 < w.t.span ? w.t.pmax + 1 : w.t.span; // of all columns

    // This wave's quarter of a stage: half `part` of tile `mine` of the two.
    const int mine = wave >> 1, part = wave & 1;
    unsigned k[NB], ks[NB == 8 ? 2 : 1], v[4][NB == 8 ? 2 : 1], vs;
    bool there;
    Pages<1> pages(a, w, lane, w.begin + mine, 2, part);
    auto clamp = [&](int i) { return i < w.stop ? i : w.stop - 1; };
    auto load = [&](int i) {
        int page[1];
        pages.take(page);
        uint64_t codes, scales;
        there = pages.at(i, part, page[0], 16 * NB, codes, scales);
        load_keys<NB>(pages, codes, scales, c, g, k, ks);
#pragma unroll
        for (int x = 0; x < 4; ++x)
            load_value<NB>(pages.vq + codes + (unsigned)((4 * g + x) * (NB * 16) + c * NB), v[x]);
        vs = *(const unsigned *)(pages.vs + scales + (unsigned)((NB * c / 16) * pages.size + 4 * g));
    };
    auto convert = [&](int i, WideStage<NB> &st) {
#pragma unroll
        for (int p = 0; p < NB; ++p)
            st.k[wave][p][lane] =
                __builtin_bit_cast(u32x4, mx_bf16x8(k[p], scale_operand(ks[NB == 8 ? p / 4 : 0])));
        const int j0 = pages.tile(i) * kTile + 16 * part;
        unsigned vsb[4], slots = 0;
#pragma unroll
        for (int x = 0; x < 4; ++x)
            vsb[x] = (vs >> (8 * x)) & 0xFFu;
        // a scale byte 0xFF: its low seven bits carry into the eighth, which is set
        const bool nans = __builtin_amdgcn_ballot_w64(((vs & 0x7F7F7F7Fu) + 0x01010101u) & vs & 0x80808080u) != 0;
        if (j0 + 16 > end || !there || nans) {
            // cleared: positions that no column sees, as in
            // attention_few_kernel, and NaN blocks, which are noted
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const bool dead = j0 + 4 * g + x >= end || !there, nan = vsb[x] == 0xFFu;
                slots |= (unsigned)(nan && !dead) << x;
                vsb[x] = dead || nan ? 127 : vsb[x];
#pragma unroll
                for (int y = 0; y < (NB == 8 ? 2 : 1); ++y)
                    v[x][y] = dead || nan ? 0 : v[x][y];
            }
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            unsigned x[4];
#pragma unroll
            for (int y = 0; y < 4; ++y)
                x[y] = cvt_byte(v[y][NB == 8 ? b / 4 : 0], scale_operand(vsb[y]), b & 3);
            st.v[mine][2 * b][lane][part] = (u32x2){even_of(x[0], x[1]), even_of(x[2], x[3])};
            st.v[mine][2 * b + 1][lane][part] = (u32x2){odd_of(x[0], x[1]), odd_of(x[2], x[3])};
        }
        const bool any = __builtin_amdgcn_ballot_w64(slots != 0) != 0;
        st.nan[wave][lane] = (unsigned char)slots;
        if (lane == 0)
            st.flags[wave] = (unsigned)any | (unsigned)there << 1;
    };

    int i = w.begin;
    if (i < w.stop) {
        load(clamp(i + mine));
        convert(clamp(i + mine), stage[0]);
        load(clamp(i + 2 + mine));
    }
    for (int buf = 0; i < w.stop; i += 2, buf ^= 1) {
        // stage[buf] is written, and every wave is done with the other one
        __syncthreads();
        if (i + 2 < w.stop) {
            convert(clamp(i + 2 + mine), stage[buf ^ 1]);
            load(clamp(i + 4 + mine));
        }
        const WideStage<NB> &st = stage[buf];
#pragma unroll 1
        for (int u = 0; u < 2; ++u) {
            const int j0 = pages.tile(i + u) * kTile;
            if (i + u >= w.stop || j0 >= q.whi)
                continue;
            const unsigned f0 = (unsigned)__builtin_amdgcn_readfirstlane((int)st.flags[2 * u]);
            const unsigned f1 = (unsigned)__builtin_amdgcn_readfirstlane((int)st.flags[2 * u + 1]);
            const bool has[2] = {(f0 & 2u) != 0, (f1 & 2u) != 0};
            const bool full = has[0] && has[1] && sees_all<NB, kNQ>(a, q, j0, w.t.span);
            f32x4 S[kNQ][2];
#pragma unroll
            for (int n = 0; n < kNQ; ++n)
                S[n][0] = S[n][1] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int p = 0; p < NB; ++p) {
                    const bf16x8 kf = __builtin_bit_cast(bf16x8, st.k[2 * u + h][p][lane]);
#pragma unroll
                    for (int n = 0; n < kNQ; ++n)
                        S[n][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, q.Q[n][p], S[n][h], 0, 0, 0);
                }
            }
            // LDS reads four operands ahead of the products
            __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
#pragma unroll
            for (int x = 0; x < 2 * NB; ++x) {
                __builtin_amdgcn_sched_group_barrier(0x008, kNQ, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
            unsigned seen[kNQ];
            if (!full)
                mask_scores<NB, kNQ>(a, q, j0, w.t.span, has, g, S, seen);
            // the softmax gives way to the products of the other waves of its
            // SIMD (2048-token chunk: 590 -> 569 us); the first operands of
            // the second product are read under it
            __builtin_amdgcn_s_setprio(0);
            bf16x8 P[kNQ], early[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                early[j] = __builtin_bit_cast(bf16x8, *(const u32x4 *)st.v[u][j][lane]);
            weigh<NB, kNQ>(a, q, S, P);
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int j = 0; j < 2 * NB; ++j) {
                const bf16x8 vf = j < 4 ? early[j] : __builtin_bit_cast(bf16x8, *(const u32x4 *)st.v[u][j][lane]);
#pragma unroll
                for (int n = 0; n < kNQ; ++n)
                    q.acc[n][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, P[n], q.acc[n][j], 0, 0, 0);
            }
            if constexpr (NB > 2)
                __builtin_amdgcn_sched_group_barrier(0x100, 2 * NB - 4, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, 2 * NB * kNQ, 0);
            if ((f0 | f1) & 1u) {
                const unsigned slots = st.nan[2 * u][lane] | (unsigned)st.nan[2 * u + 1][lane] << 4;
#pragma unroll
                for (int n = 0; n < kNQ; ++n) {
                    const f32x4 count = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        ones(slots), ones(full ? 0xFFu : seen[n]), (f32x4){0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
#pragma unroll
                    for (int j = 0; j < 2 * NB; ++j)
                        spoil(q.acc[n][j], count);
                }
            }
        }
    }
#pragma unroll
    for (int n = 0; n < kNQ; ++n)
        q.l[n] = sum_groups(q.l[n]);
    store_columns<NB, kNQ>(a, w, q, wave * kNQ * 16, c, g);
}

// Joins the splits of the column tiles that have several: `per_tile`
// workgroups of 256 threads for each column tile and head, `cols` columns at a
// time; of the threads of a column dim / 4 lie along its channels and the rest
// along the splits.
template <int NB>
__global__ __launch_bounds__(256) void attention_join_kernel(AttnArgs a, int R, int per_tile, int cols)
{
    constexpr int dim = 32 * NB, along = dim / 4;
    __shared__ f32x4 so[256];
    __shared__ float sl[256];
    __shared__ LineSeq seqs[kLineSeqs];
    const int lane = threadIdx.x & 63;
    const int part = (int)(blockIdx.x % (unsigned)per_tile);
    const int id = (int)(blockIdx.x / (unsigned)per_tile), tile = id / (int)a.c.heads;
    Place w;
    w.head = id % (int)a.c.heads;
    if (!find_tile(a, R, tile, lane, w))
        return;
    Parts parts;
    if (a.line) {
        Line line;
        line.build(a, R, lane, seqs);
        const LineSeq q = line.of(w.s);
        const int64_t start = q.at + (int64_t)w.local * q.per;
        const int64_t p0 = start / line.share, p1 = (start + q.per - 1) / line.share;
        parts.count = (int)(p1 - p0) + 1;
        parts.stride = 2 * a.c.heads * R;
        parts.extra = a.c.heads * R;
        parts.base = (2 * p0 * a.c.heads + w.head) * R;
    } else {
        int per = 0;
        parts = split_parts(a, R, tile, w.head, w.t.n, lane, per);
    }
    if (parts.count == 1)
        return;
    auto part_at = [&](int i) { return parts.base + i * parts.stride + (i == 0 ? parts.extra : 0); };
    const int ways = 256 / along / cols; // threads along the splits
    const int d4 = threadIdx.x % along, way = threadIdx.x / along % ways, sub = threadIdx.x / along / ways;
    const int stop = (w.local + 1) * R < w.t.cols ? (w.local + 1) * R : w.t.cols;
    for (int col0 = w.local * R + part * cols; col0 < stop; col0 += per_tile * cols) {
        const int col = col0 + sub < stop ? col0 + sub : stop - 1;
        const int i = col / a.group, row = w.t.seq.first + i, head = w.head * a.group + col - i * a.group;
        const int at = col - w.local * R;
        f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
        float l = 0.0f, m = -__builtin_inff();
        for (int x = way; x < parts.count; x += ways)
            m = vmax(m, a.part_ml[(part_at(x) + at) * 2]);
        sl[threadIdx.x] = m;
        __syncthreads();
        for (int x = 0; x < ways; ++x)
            m = vmax(m, sl[(sub * ways + x) * along + d4]);
        __syncthreads();
        for (int x = way; x < parts.count; x += ways) {
            const int64_t r = part_at(x) + at;
            const f32x2 ml = *(const f32x2 *)(a.part_ml + r * 2);
            const float f = ml[0] == m ? 1.0f : __builtin_amdgcn_exp2f(ml[0] - m);
            o += f * *(const f32x4 *)(a.part_o + r * dim + d4 * 4);
            l += f * ml[1];
        }
        so[threadIdx.x] = o;
        sl[threadIdx.x] = l;
        __syncthreads();
        if (way == 0 && col0 + sub < stop) {
            for (int x = 1; x < ways; ++x) {
                o += so[threadIdx.x + x * along];
                l += sl[threadIdx.x + x * along];
            }
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            *(u32x2 *)(a.out + (int64_t)row * a.out_stride + head * dim + d4 * 4) =
                (u32x2){pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv)};
        }
        __syncthreads();
    }
}

// Stages of a wave's ring, few columns.
constexpr int few_depth(int64_t dim) { return dim == 256 ? 2 : dim == 128 ? 3 : 4; }

// Bytes of the line's table in LDS.
constexpr int line_lds(int64_t seqs) { return (int)((seqs + 63) / 64 * 64) * (int)sizeof(LineSeq); }

// Workgroups of attention_few_kernel that a CU holds: by registers three with
// one column tile (dim 64, 128), else two; by LDS as computed.
int few_resident(int64_t dim, int nq, int64_t seqs)
{
    const int ring = dim == 64    ? few_lds<2, 1, kWaves, few_depth(64)>()
                     : dim == 128 ? few_lds<4, 1, kWaves, few_depth(128)>()
                                  : few_lds<8, 1, kWaves, few_depth(256)>();
    const int lds = 160 * 1024 / (ring + line_lds(seqs)), regs = nq == 1 && dim < 256 ? 3 : 2;
    return lds < regs ? lds : regs;
}

// Columns of a workgroup, and how the work is cut.
struct Shape {
    bool many;
    int nq, R;
    int tiles, wanted;
    int splits; // many columns
    int line;   // few columns
    int64_t parts; // rows of partial results (0: none, and no join)
};

Shape shape_of(int64_t q_heads, const mx_cache &c, const mx_batch &b, int64_t window, int64_t sinks)
{
    Shape s{};
    const int64_t group = q_heads / c.heads, cols = b.rows * group;
    const int64_t mean = (cols + b.seqs - 1) / b.seqs; // columns of a sequence
    s.many = mean > 64;
    s.nq = mean <= 16 || c.dim == 256 ? 1 : 2;
    s.R = 16 * s.nq * (s.many ? kWaves : 1);
    s.tiles = (int)(cols / s.R + b.seqs);
    s.splits = 1;
    const int64_t groups = (int64_t)s.tiles * c.heads;
    // cache tiles of the longest sequence the table can hold
    int64_t span = b.width * c.page_size;
    if (window && window + sinks + b.rows + 2 * kTile < span)
        span = window + sinks + b.rows + 2 * kTile;
    const int64_t most = (span + kTile - 1) / kTile;
    if (s.many) {
        // resident workgroups, by LDS
        s.wanted = (c.dim == 64 ? 4 : c.dim == 128 ? 2 : 1) * device_cus();
        if (b.seqs <= kLineSeqs && 2 * groups <= s.wanted) {
            const int64_t cut = (most + 2 * kWaves - 1) / (2 * kWaves);
            // twice the mean: the longer sequences of a mixed batch take more
            int64_t n = 2 * (s.wanted / groups);
            n = n < cut ? n : cut;
            s.splits = (int)(n < 1 ? 1 : n > kMaxSplits ? kMaxSplits : n);
        }
        s.parts = s.splits > 1 ? (int64_t)s.splits * groups * s.R : 0;
    } else {
        s.wanted = (b.seqs <= kLineSeqs ? few_resident(c.dim, s.nq, b.seqs) : 2) * device_cus();
        // with many column tiles the chip evens out by itself
        if (b.seqs <= kLineSeqs && groups <= 4 * s.wanted && most > kWhole) {
            s.line = (int)((s.wanted + c.heads - 1) / c.heads);
            s.parts = 2 * (int64_t)s.line * c.heads * s.R;
        }
    }
    return s;
}

template <int NB, int kNQ, int kW, int kD>
hipError_t launch_few(const AttnArgs &a, int64_t grid, hipStream_t stream)
{
    constexpr int most = few_lds<NB, kNQ, kW, kD>() + kLineSeqs * (int)sizeof(LineSeq);
    static_assert(most <= 160 * 1024, "LDS of a CU");
    const hipError_t e = allow_dynamic_lds((const void *)attention_few_kernel<NB, kNQ, kW, kD>, most);
    if (e != hipSuccess)
        return e;
    const int bytes = few_lds<NB, kNQ, kW, kD>() + line_lds(a.line ? a.b.seqs : 0);
    attention_few_kernel<NB, kNQ, kW, kD><<<dim3((unsigned)grid), dim3(64 * kW), bytes, stream>>>(a);
    return hipGetLastError();
}

template <int NB>
hipError_t launch(const AttnArgs &a, const Shape &s, hipStream_t stream)
{
    const int64_t grid = (s.line ? (int64_t)s.line : (int64_t)s.tiles * s.splits) * a.c.heads;
    if (grid > 0x7FFFFFFF)
        return hipErrorInvalidConfiguration;
    const dim3 g((unsigned)grid), w(64 * kWaves);
    constexpr int kMost = NB == 8 ? 1 : 2; // column tiles a wave has registers for
    if (s.many) {
        constexpr int bytes = 2 * (int)sizeof(WideStage<NB>);
        const void *fn = (const void *)attention_many_kernel<NB, kMost>;
        const hipError_t e = allow_dynamic_lds(fn, bytes);
        if (e != hipSuccess)
            return e;
        attention_many_kernel<NB, kMost><<<g, w, bytes, stream>>>(a);
    } else {
        hipError_t e;
        constexpr int kD = few_depth(32 * NB);
        e = s.nq > 1 ? launch_few<NB, kMost, kWaves, kD>(a, grid, stream)
                     : launch_few<NB, 1, kWaves, kD>(a, grid, stream);
        if (e != hipSuccess)
            return e;
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || s.parts == 0)
        return e;
    // about 2048 workgroups (8 a CU), each with the columns abreast that leave
    // threads for four parts or more
    const int parts = s.line ? s.line : s.splits;
    int cols = 256 / (8 * NB);
    while (cols > 1 && 256 / (8 * NB) / cols < (parts < 4 ? parts : 4))
        cols /= 2;
    const int64_t groups = (int64_t)s.tiles * a.c.heads, chunks = (s.R + cols - 1) / cols;
    int64_t per = 2048 / groups;
    per = per < 1 ? 1 : per > chunks ? chunks : per;
    attention_join_kernel<NB><<<dim3((unsigned)(groups * per)), dim3(256), 0, stream>>>(a, s.R, (int)per, cols);
    return hipGetLastError();
}

} // namespace

int64_t attention_workspace(int64_t q_heads, const mx_cache &c, const mx_batch &b, int64_t window, int64_t sinks)
{
    return shape_of(q_heads, c, b, window, sinks).parts * (c.dim + 2) * 4;
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
    a.part_ml = a.part_o + s.parts * c.dim;
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
    a.line = s.line;
    a.wanted = s.wanted;
    a.size16 = (unsigned)(c.page_size / 16);
    const uint64_t magic = ((uint64_t)1 << 32) / a.size16 + 1;
    a.magic = (unsigned)magic;
    a.magic_hi = (unsigned)(magic >> 32);
    a.tiles = s.tiles;
    switch (c.dim) {
    case 64: return launch<2>(a, s, stream);
    case 128: return launch<4>(a, s, stream);
    default: return launch<8>(a, s, stream);
    }
}

} // namespace kq
