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
// fourth tile, loaded straight into LDS, and join through LDS.  Many
// (attention_many_kernel): every wave has its own columns, and the converted
// tiles are shared through LDS.  Both take equal shares (or pieces) of the
// batch's work; a second kernel joins the parts of what was cut.
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
    int line;     // workgroups of a head's line (0: one for each column tile)
    int join;     // cache tiles of a workgroup that take as long as a join
    unsigned size16, magic, magic_hi; // page_size / 16; the words of floor(2^32 / size16) + 1
    int tiles;    // column tiles: an upper bound over the batch
};

// The kernel's arguments, read again from where they lie: there are more of
// them than fit the scalar registers next to a walk through the cache, and the
// compiler would keep what it has read.
typedef const __attribute__((address_space(4))) AttnArgs KArgs;

__device__ __forceinline__ KArgs &kernel_args()
{
    auto p = __builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return *(KArgs *)p;
}

// The lane as a value that nothing computed before depends on: what follows
// from it is not carried in registers from one place of the work to the next.
__device__ __forceinline__ int fresh(int lane)
{
    asm volatile("" : "+v"(lane));
    return lane;
}

template <class A>
__device__ __forceinline__ mx_batch batch_of(A &a)
{
    return {a.b.page_table, a.b.row_start, a.b.lengths, a.b.seqs, a.b.width, a.b.rows};
}

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

template <class A>
__device__ __forceinline__ TilePlan plan_tile(A &a, const SeqRows &seq, int local, int R)
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
template <class A>
__device__ __forceinline__ int most_tiles(A &a, int64_t len, int R)
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

// Column tiles are numbered so that those of sequence s start here, which
// leaves it at least ceil(columns / R).
__device__ __forceinline__ int64_t tiles_before(int64_t row_start, int group, int R, int s)
{
    return (row_start < 0 ? 0 : row_start) * group / R + s;
}

// Column tile -> sequence and its local number.  False: the sequence has no
// such tile.
template <class A>
__device__ __forceinline__ bool find_tile(A &a, int R, int tile, int lane, Place &w)
{
    auto first_of = [&](int s) { return tiles_before(a.b.row_start[s], a.group, R, s); };
    w.s = wave_search((int)a.b.seqs, tile, lane, first_of);
    const int64_t local = tile - first_of(w.s);
    const SeqRows q = seq_rows(batch_of(a), w.s);
    if (local < 0 || local * R >= (int64_t)q.rows * a.group)
        return false;
    w.local = (int)local;
    w.t = plan_tile(a, q, w.local, R);
    return true;
}

// ---- equal shares of a line ------------------------------------------------
// The cache tiles of all column tiles of all sequences, one after the other,
// are cut into equal shares, one for each of a head's workgroups: a share ends
// inside a column tile wherever it does, so lengths do not have to match for
// the chip to be filled evenly.  A workgroup has at most one column tile that
// began before its share and one that goes on after it, so it needs two
// places for partial results: 2 p and 2 p + 1.  (12 ragged chunks of 16 heads:
// 87 us, 151 with a workgroup for each column tile; 48 single tokens 117, 142;
// eight sequences seen through a window 28, 48.)
//
// A workgroup that works on two column tiles starts twice, though, which costs
// it about kSecond tiles.  Where cutting every column tile into pieces of its
// own makes the longest piece no longer than that, the places of the line are
// these pieces, one a workgroup (the window: 27.7 us, 33.3 with shares; ragged
// chunks, whose pieces would be longer, 95.8 with pieces).  And where whole
// column tiles take no longer than equal shares and a join, they are the pieces.
//
// The arrays of the batch are read once, together, and kept in LDS.
constexpr int kLineSeqs = 256;
constexpr int kLineMost = 1 << 30; // places of a line: what follows is 32-bit
constexpr unsigned kSecond = 8;

struct LineSeq {
    int at;                // where the sequence starts in the line
    int first, rows, len;  // its rows (none: where they would start)
    int per;               // places of one of its column tiles
};

// Where a workgroup is in the line.
struct LineState {
    int share, end; // places of a workgroup, and of the line
    int x;          // the next place
    int pieces;     // a place is a piece of a column tile, not one cache tile
};

// Sums (or maxima) of v over the lanes up to each one, v >= 0: the steps of a
// scan along rows of 16 lanes, then across the rows.
template <class Op>
__device__ __forceinline__ int wave_scan(int v, Op op)
{
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false)); // row_shr 1, 2, 4, 8
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false));
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false));
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false));
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false)); // row_bcast 15, 31
    return op(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false));
}

// The line's sequences, in LDS after a state for each wave.
struct Line {
    LineState *state;
    LineSeq *seq;
    int lane;

    __device__ __forceinline__ Line(void *lds, int lane_)
        : state((LineState *)lds), seq((LineSeq *)(state + kWaves)), lane(lane_)
    {
    }

    // Every wave of the workgroup takes part; each writes the same (whole
    // groups of 64 sequences), which is read after a barrier.
    template <class A>
    __device__ __forceinline__ LineState build(A &a, int R, int p) const
    {
        const auto add = [](int x, int y) { return x + y; };
        const auto larger = [](int x, int y) { return x > y ? x : y; };
        const int seqs = (int)a.b.seqs;
        LineSeq v[kLineSeqs / 64];
        int mine[kLineSeqs / 64];            // column tiles of the lane's sequence
        int most = 0, places = 0, tiles = 0; // of the longest column tile, and of all; all column tiles
        int load = 0; // at least places / 1024
#pragma unroll
        for (int k = 0; k < kLineSeqs / 64; ++k) {
            const int s = 64 * k + lane;
            v[k] = {0, 0, 0, 0, 0};
            if (s < seqs) {
                const int64_t b = a.b.row_start[s], e = a.b.row_start[s + 1];
                v[k].len = a.b.lengths[s] < 0 ? 0 : a.b.lengths[s];
                const bool ok = b >= 0 && b < e && e <= a.b.rows;
                v[k].first = b < 0 ? 0 : (int)b;
                v[k].rows = ok ? (int)(e - b) : 0;
                const int n = most_tiles(a, v[k].len, R);
                v[k].per = n < 1 ? 1 : n;
            }
        }
#pragma unroll
        for (int k = 0; k < kLineSeqs / 64; ++k) {
            if (64 * k >= seqs)
                continue;
            mine[k] = (v[k].rows * a.group + R - 1) / R;
            const float all = (float)mine[k] * (float)v[k].per / 1024.0f;
            load += __builtin_amdgcn_readlane(wave_scan((int)(all < 1 << 22 ? all : 1 << 22) + 1, add), 63);
            most = larger(most, __builtin_amdgcn_readlane(wave_scan(mine[k] ? v[k].per : 0, larger), 63));
            const int upto = places + wave_scan(mine[k] * v[k].per, add);
            v[k].at = upto - mine[k] * v[k].per;
            places = __builtin_amdgcn_readlane(upto, 63);
            tiles += __builtin_amdgcn_readlane(wave_scan(mine[k], add), 63);
        }
        // a share of the line, and the least of one: two tiles a wave
        const unsigned line = (unsigned)a.line, least = 2 * kWaves;
        unsigned share = ((unsigned)places + line - 1) / line;
        share = share < least ? least : share;
        // tiles of a piece: all of a column tile, or so many that there are no
        // more pieces than workgroups (ceil(n / each) <= n / each + 1 of each)
        unsigned each = (unsigned)most;
        const unsigned rounds = ((unsigned)tiles + line - 1) / line;
        bool pieces = (float)rounds * (float)most <= (float)((unsigned)places / line + (unsigned)a.join);
        if (!pieces && (unsigned)tiles < line) {
            each = ((unsigned)places + line - (unsigned)tiles - 1) / (line - (unsigned)tiles);
            each = each < least ? least : each;
            pieces = each <= share + kSecond;
        }
        if (pieces) {
            each = each < 1 ? 1 : each;
            places = 0;
#pragma unroll
            for (int k = 0; k < kLineSeqs / 64; ++k) {
                if (64 * k >= seqs)
                    continue;
                v[k].per = (int)(((unsigned)v[k].per + each - 1) / each);
                const int upto = places + wave_scan(mine[k] * v[k].per, add);
                v[k].at = upto - mine[k] * v[k].per;
                places = __builtin_amdgcn_readlane(upto, 63);
            }
            share = ((unsigned)places + line - 1) / line;
            share = share < 1 ? 1 : share;
        }
#pragma unroll
        for (int k = 0; k < kLineSeqs / 64; ++k)
            if (64 * k < seqs)
                seq[64 * k + lane] = v[k];
        // only sequences that overlap (a row_start that decreases) have more
        // places than a line: none of them is worked on
        const unsigned end = load > kLineMost / 1024 ? 0u : (unsigned)places;
        return {(int)share, (int)end, (int)(p * share), pieces};
    }

    // A sequence's entry, the same in all lanes.
    __device__ __forceinline__ LineSeq of(int s) const
    {
        const LineSeq v = seq[s];
        return {__builtin_amdgcn_readfirstlane(v.at), __builtin_amdgcn_readfirstlane(v.first), __builtin_amdgcn_readfirstlane(v.rows),
                __builtin_amdgcn_readfirstlane(v.len), __builtin_amdgcn_readfirstlane(v.per)};
    }

    // The last sequence whose key is at most x.
    template <class Key>
    __device__ __forceinline__ int last(int x, int seqs, Key key) const
    {
        int n = 0;
        for (int k = 0; 64 * k < seqs; ++k) {
            const int s = 64 * k + lane;
            n += __popcll(__builtin_amdgcn_ballot_w64(s < seqs && key(s) <= x));
        }
        return n > 0 ? n - 1 : 0;
    }

    // The sequence that place x of the line belongs to (an empty one starts
    // where the next one does).
    __device__ __forceinline__ int find(int x, int seqs) const
    {
        return last(x, seqs, [&](int s) { return seq[s].at; });
    }

    // The sequence that has column tile `tile`, as find_tile numbers them.
    __device__ __forceinline__ int find_tile(int R, int group, int tile, int seqs) const
    {
        return last(tile, seqs, [&](int s) { return tiles_before(seq[s].first, group, R, s); });
    }
};

// Bytes of the line in LDS.
__host__ __device__ constexpr int line_lds(int64_t seqs)
{
    return kWaves * (int)sizeof(LineState) + (int)((seqs + 63) / 64 * 64) * (int)sizeof(LineSeq);
}

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
    // positions of the wave's first and last column, and one past what it sees
    int wmin, wmax, whi;
    bool idle;                // padding columns only
};

template <int NB, int kNQ, class A>
__device__ __forceinline__ void load_columns(A &a, const Place &w, int col0, int c, int g,
                                             Columns<NB, kNQ> &q)
{
    const TilePlan &t = w.t;
#pragma unroll
    for (int n = 0; n < kNQ; ++n) {
        const int col = col0 + n * 16 + c;
        const bool live = col < t.cols; // not a padding column
        const int at = live ? col : 0, i = at / a.group, head = w.head * a.group + at - i * a.group;
        q.pos[n] = live ? (int)(t.seq.pos0 + i) : -1;
        q.low[n] = a.window && live ? q.pos[n] - a.window + 1 : -0x7FFFFFFF;
        const uint16_t *src = a.q + (int64_t)(t.seq.first + i) * a.q_stride + head * (32 * NB) + g * (8 * NB);
#pragma unroll
        for (int p = 0; p < NB; ++p) {
            u32x4 v = *(const u32x4 *)(src + 8 * p);
            if (!live)
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
template <int NB, int kNQ, class A>
__device__ __forceinline__ bool sees_all(A &a, const Columns<NB, kNQ> &q, int j0, int span)
{
    return j0 + kTile <= q.wmin + 1 && j0 + kTile <= span && !q.idle &&
           (!a.window || j0 >= q.wmax - a.window + 1 || j0 + kTile <= a.sinks);
}

// Scores of what a column does not see become -infinity; `seen` gets the
// positions (k slot 4h + i: position 16h + 4g + i of the tile) that it sees.
template <int NB, int kNQ, class A>
__device__ __forceinline__ void mask_scores(A &a, const Columns<NB, kNQ> &q, int j0, int span,
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
template <int NB, int kNQ, class A>
__device__ __forceinline__ void weigh(A &a, Columns<NB, kNQ> &q, const f32x4 (&S)[kNQ][2],
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
template <int NB, int kNQ, class A>
__device__ __forceinline__ void store_columns(A &a, const Place &w, const Columns<NB, kNQ> &q, int R,
                                              int col0, int lane)
{
    constexpr int dim = 32 * NB;
    const int c = lane & 15, g = lane >> 4;
#pragma unroll
    for (int n = 0; n < kNQ; ++n) {
        const int col = w.local * R + col0 + n * 16 + c;
        if (col >= w.t.cols)
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
            const int i = col / a.group, head = w.head * a.group + col - i * a.group;
            uint16_t *o = a.out + (int64_t)(w.t.seq.first + i) * a.out_stride + head * dim + g * (8 * NB);
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

    template <class A>
    __device__ __forceinline__ Pages(A &a, const Place &w, int lane_, int first_, int step_, int part_)
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
template <int NB, int kNQ, int kW, int kD, class A>
__device__ __forceinline__ void attention_few(A &a, const Place &w, int lane, int wave,
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
    lane = fresh(lane);
    const int col = lane & 15;
    f32x4 *so = (f32x4 *)lds;                               // [kW][kNQ][2 NB][64]
    float *sm = (float *)(so + kW * kNQ * 2 * NB * 64);     // [kW][kNQ][16], and the sums after it
    float *sl = sm + kW * kNQ * 16;
#pragma unroll
    for (int n = 0; n < kNQ; ++n)
        q.l[n] = sum_groups(q.l[n]);
    __syncthreads();
    if (lane < 16) {
#pragma unroll
        for (int n = 0; n < kNQ; ++n) {
            sm[(wave * kNQ + n) * 16 + col] = q.m[n];
            sl[(wave * kNQ + n) * 16 + col] = q.l[n];
        }
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < kNQ; ++n) {
        float up = sm[n * 16 + col];
#pragma unroll
        for (int x = 1; x < kW; ++x)
            up = vmax(up, sm[(x * kNQ + n) * 16 + col]);
        float sum = 0.0f;
#pragma unroll
        for (int x = 0; x < kW; ++x) {
            const float mx = sm[(x * kNQ + n) * 16 + col];
            sum += sl[(x * kNQ + n) * 16 + col] * (mx == up ? 1.0f : __builtin_amdgcn_exp2f(mx - up));
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
    store_columns<NB, kNQ>(a, w, q, R, 0, lane);
}

// Walks the places of this workgroup: `work(place)` for each, with a barrier
// after it.  Workgroup -> (share or column tile, head), the head fastest: the
// eight XCDs take workgroups in turn, so a head's cache stays in few L2s, and
// the last first, whose rows see most (2048-token chunk: 598 -> 580 us).
// `args()`: the arguments; `lds`: for the line.  kLean: nothing is kept in
// registers while a place is worked on.  The many-column kernel has none to
// spare (12 ragged chunks: 101 -> 90 us); few columns only lose by it (48 single
// tokens: 119 -> 129 us).
template <bool kLean, class Args, class Work>
__device__ __forceinline__ void for_places(Args args, int R, int lane, int wave, void *lds, Work work)
{
    const Line line(lds, lane);
    LineState at{};
    {
        auto &a = args();
        if (a.line) {
            at = line.build(a, R, a.line - 1 - (int)blockIdx.x / (int)a.c.heads);
            __syncthreads();
        }
    }
    for (;;) {
        auto &a = args();
        const int heads = (int)a.c.heads, p = (a.line ? a.line : a.tiles) - 1 - (int)blockIdx.x / heads;
        Place w;
        w.head = (int)blockIdx.x % heads;
        if (a.line) {
            const int begin = p * at.share, end = begin + at.share < at.end ? begin + at.share : at.end;
            if (at.x >= end)
                return;
            w.s = line.find(at.x, (int)a.b.seqs);
            const LineSeq q = line.of(w.s);
            w.local = (int)((unsigned)(at.x - q.at) / (unsigned)q.per);
            const int tile = q.at + w.local * q.per; // the column tile's first place in the line
            const int next = at.pieces ? at.x + 1 : tile + q.per < end ? tile + q.per : end;
            w.t = plan_tile(a, {q.first, q.rows, (int64_t)q.len - q.rows}, w.local, R);
            const int of = at.pieces ? (int)((unsigned)(w.t.n + q.per - 1) / (unsigned)q.per) : 1; // a place's tiles
            w.begin = (at.x - tile) * of < w.t.n ? (at.x - tile) * of : w.t.n;
            w.stop = (next - tile) * of < w.t.n ? (next - tile) * of : w.t.n;
            const bool all = at.x == tile && next == tile + q.per;
            w.part = all ? -1 : ((int64_t)(2 * p + (tile >= begin ? 1 : 0)) * heads + w.head) * R;
            at.x = next;
            if (kLean)
                line.state[wave] = at;
        } else {
            if (!find_tile(a, R, p, lane, w))
                return;
            w.begin = 0;
            w.stop = w.t.n;
            w.part = -1;
        }
        work(w);
        if (args().line == 0)
            return;
        __syncthreads(); // LDS is free again
        if (kLean) {
            at = line.state[wave];
            at = {__builtin_amdgcn_readfirstlane(at.share), __builtin_amdgcn_readfirstlane(at.end),
                  __builtin_amdgcn_readfirstlane(at.x), __builtin_amdgcn_readfirstlane(at.pieces)};
        }
    }
}

template <int NB, int kNQ, int kW, int kD>
__global__ __launch_bounds__(64 * kW, 2) void attention_few_kernel(AttnArgs a)
{
    extern __shared__ __align__(16) unsigned char lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    for_places<false>([&]() -> const AttnArgs & { return a; }, 16 * kNQ, lane, wave,
                      lds + few_lds<NB, kNQ, kW, kD>(),
                      [&](const Place &w) { attention_few<NB, kNQ, kW, kD>(a, w, lane, wave, lds); });
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

// One workgroup's cache tiles of a column tile.
template <int NB, int kNQ>
__device__ __forceinline__ void attention_many(KArgs &a, const Place &w, int lane, int wave,
                                               WideStage<NB> *stage)
{
    constexpr int R = 16 * kNQ * kWaves;
    const int c = lane & 15, g = lane >> 4;
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
    store_columns<NB, kNQ>(kernel_args(), w, q, R, wave * kNQ * 16, fresh(lane));
}

// dim 64: registers for four waves a SIMD, as many as LDS holds (12 ragged
// chunks of 16 heads: 134 -> 108 us); wider heads have LDS for two or one.
template <int NB, int kNQ>
__global__ __launch_bounds__(64 * kWaves)
    __attribute__((amdgpu_waves_per_eu(NB == 2 ? 4 : 2, NB == 2 ? 4 : 2))) void attention_many_kernel(AttnArgs)
{
    extern __shared__ __align__(16) unsigned char lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    WideStage<NB> *stage = (WideStage<NB> *)lds;
    for_places<true>(kernel_args, 16 * kNQ * kWaves, lane, wave, stage + 2,
                     [&](const Place &w) { attention_many<NB, kNQ>(kernel_args(), w, fresh(lane), wave, stage); });
}

// Joins the parts of the column tiles that have several: `per_tile` workgroups
// of 256 threads for each column tile and head.  dim / 4 threads lie along the
// channels of a column; the rest are columns, or, where there are many parts,
// ways along them.  A thread loads four parts at a time, with their maxima and
// sums, before it adds them, in order.
template <int NB>
__global__ __launch_bounds__(256) void attention_join_kernel(AttnArgs a, int R, int per_tile)
{
    constexpr int dim = 32 * NB, along = dim / 4, slots = 256 / along;
    __shared__ f32x4 so[256];
    __shared__ f32x2 sml[256];
    __shared__ __align__(16) unsigned char lds[line_lds(kLineSeqs)];
    const int lane = threadIdx.x & 63;
    const int chunk = (int)(blockIdx.x % (unsigned)per_tile);
    const int id = (int)(blockIdx.x / (unsigned)per_tile), heads = (int)a.c.heads, tile = id / heads, kv = id % heads;
    const Line line(lds, lane);
    const LineState whole_line = line.build(a, R, 0);
    __syncthreads();
    const int sq = line.find_tile(R, a.group, tile, (int)a.b.seqs);
    const LineSeq q = line.of(sq);
    const int64_t local = tile - tiles_before(q.first, a.group, R, sq);
    const int columns = q.rows * a.group;
    if (whole_line.end == 0 || local < 0 || local * R >= columns)
        return;
    const int first = (int)local * R, stop = first + R < columns ? first + R : columns;
    const unsigned share = (unsigned)whole_line.share, start = (unsigned)(q.at + (int)local * q.per), p0 = start / share;
    const int count = (int)((start + (unsigned)q.per - 1) / share - p0) + 1;
    if (count == 1)
        return;
    // part i starts at row base + i stride, part 0 `stride / 2` rows later
    const int64_t stride = (int64_t)2 * heads * R, base = ((int64_t)2 * p0 * heads + kv) * R;
    int ways = 1;
    while (ways < slots && 4 * ways < count)
        ways *= 2;
    const int cols = slots / ways;
    const int d4 = threadIdx.x % along, way = threadIdx.x / along % ways, sub = threadIdx.x / along / ways;
    for (int col0 = first + chunk * cols; col0 < stop; col0 += per_tile * cols) {
        const int col = col0 + sub < stop ? col0 + sub : stop - 1;
        const int64_t at = base + col - first;
        f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
        float l = 0.0f, m = -__builtin_inff();
        auto add = [&](const f32x2 &ml, const f32x4 &v) {
            const float up = vmax(m, ml[0]);
            const float f0 = m == up ? 1.0f : __builtin_amdgcn_exp2f(m - up);
            const float f1 = ml[0] == up ? 1.0f : __builtin_amdgcn_exp2f(ml[0] - up);
            m = up;
            o = o * f0 + v * f1;
            l = l * f0 + ml[1] * f1;
        };
        for (int x = way; x < count; x += 4 * ways) {
            f32x2 ml[4];
            f32x4 v[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int i = x + y * ways < count ? x + y * ways : x;
                const int64_t r = at + i * stride + (i == 0 ? stride / 2 : 0);
                ml[y] = *(const f32x2 *)(a.part_ml + r * 2);
                v[y] = *(const f32x4 *)(a.part_o + r * dim + d4 * 4);
            }
#pragma unroll
            for (int y = 0; y < 4; ++y)
                if (x + y * ways < count)
                    add(ml[y], v[y]);
        }
        if (ways > 1) {
            __syncthreads(); // the last columns' are read
            so[threadIdx.x] = o;
            sml[threadIdx.x] = (f32x2){m, l};
            __syncthreads();
            if (way == 0)
                for (int x = 1; x < ways; ++x)
                    add(sml[threadIdx.x + x * along], so[threadIdx.x + x * along]);
        }
        if (way == 0 && col0 + sub < stop) {
            const int i = col / a.group, row = q.first + i, head = kv * a.group + col - i * a.group;
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            *(u32x2 *)(a.out + (int64_t)row * a.out_stride + head * dim + d4 * 4) =
                (u32x2){pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv)};
        }
    }
}

// Stages of a wave's ring, few columns.
constexpr int few_depth(int64_t dim) { return dim == 256 ? 2 : dim == 128 ? 3 : 4; }

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
    int tiles; // column tiles: an upper bound over the batch
    int line, join;
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
    // cache tiles of the longest sequence the table can hold
    int64_t span = b.width * c.page_size;
    if (window && window + sinks + b.rows + 2 * kTile < span)
        span = window + sinks + b.rows + 2 * kTile;
    const int64_t most = (span + kTile - 1) / kTile, groups = (int64_t)s.tiles * c.heads;
    // what a join and its launch take, in tiles of a workgroup
    s.join = s.many ? 32 : 48;
    if (b.seqs > kLineSeqs || most <= s.join)
        return s;
    const int resident = !s.many         ? few_resident(c.dim, s.nq, b.seqs)
                         : c.dim == 64   ? 4
                         : c.dim == 128  ? 2
                                         : 1; // by LDS
    const int64_t fill = (int64_t)resident * device_cus();
    // with many column tiles the chip evens out by itself
    if (groups <= 4 * fill && s.tiles * most <= kLineMost / 2) {
        s.line = (int)((fill + c.heads - 1) / c.heads);
        s.parts = 2 * (int64_t)s.line * c.heads * s.R;
    }
    return s;
}

template <int NB, int kNQ, int kW, int kD>
hipError_t launch_few(const AttnArgs &a, int64_t grid, hipStream_t stream)
{
    constexpr int most = few_lds<NB, kNQ, kW, kD>() + line_lds(kLineSeqs);
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
    const int64_t grid = (int64_t)(s.line ? s.line : s.tiles) * a.c.heads;
    if (grid > 0x7FFFFFFF)
        return hipErrorInvalidConfiguration;
    const dim3 g((unsigned)grid), w(64 * kWaves);
    constexpr int kMost = NB == 8 ? 1 : 2; // column tiles a wave has registers for
    if (s.many) {
        constexpr int bytes = 2 * (int)sizeof(WideStage<NB>), most = bytes + line_lds(kLineSeqs);
        static_assert(most <= 160 * 1024, "LDS of a CU");
        const hipError_t e = allow_dynamic_lds((const void *)attention_many_kernel<NB, kMost>, most);
        if (e != hipSuccess)
            return e;
        attention_many_kernel<NB, kMost><<<g, w, bytes + line_lds(a.line ? a.b.seqs : 0), stream>>>(a);
    } else {
        hipError_t e;
        constexpr int kD = few_depth(32 * NB);
        // A workgroup that has a CU to itself takes eight waves (one token over
        // 1001, dim 128: 11.4 -> 11.0 us; 16 tokens over 1400: 14.9 -> 13.2; over
        // 300: 7.8 -> 8.0).  Not at dim 256, where the join of eight costs more
        // (4 tokens over 1200: 20.1 -> 21.2), nor with two column tiles a wave,
        // which then has too few registers.
        constexpr bool kMore = NB < 8;
        constexpr int kLoneWaves = kMore ? 2 * kWaves : kWaves, kLoneD = kMore ? 2 : kD;
        if (s.nq > 1)
            e = launch_few<NB, kMost, kWaves, kD>(a, grid, stream);
        else if (kMore && s.line == 0 && grid <= device_cus())
            e = launch_few<NB, 1, kLoneWaves, kLoneD>(a, grid, stream);
        else
            e = launch_few<NB, 1, kWaves, kD>(a, grid, stream);
        if (e != hipSuccess)
            return e;
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || s.parts == 0)
        return e;
    // about 2048 workgroups (8 a CU), at most one for each column
    const int64_t groups = (int64_t)s.tiles * a.c.heads;
    int64_t per = 2048 / groups;
    per = per < 1 ? 1 : per > s.R ? s.R : per;
    attention_join_kernel<NB><<<dim3((unsigned)(groups * per)), dim3(256), 0, stream>>>(a, s.R, (int)per);
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
    a.line = s.line;
    a.join = s.join;
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
