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
// row c = l % 16 and eight k of group g = l / 16.  Which eight is free as long
// as both operands agree, so group g takes the whole MX block 4u + g of a step
// u of 128 k: a 16-byte piece of codes and one scale feed four matrix
// instructions, the j-th on the block's elements 8j..8j+7.  The 16 columns are
// tokens.  The accumulator holds W row 4g + i, token c in element i.
//
// The bound is reading W once, so everything else is kept off the vector
// memory path, whose loads complete in order: a load of x between two loads
// of codes would have to wait for them.  Both kernels hold x in LDS.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kq_device.h"
#include "kq_internal.h"

namespace kq {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

// Codes and scales of two steps (256 k) of 16 weight rows, as one wave holds
// them.
struct Pair {
    u32x4 w[2];
    unsigned s[2];
};

// Where one lane reads them.  Codes: eight rows x 128 bytes a load, whole
// cache lines (16 rows x 64 bytes read a 300 MB matrix at 4.8 instead of 6.9
// TB/s).  Lane (c, g) of the first load has row c % 8, block g + 4 (c / 8), of
// the second the same of rows 8..15; exchanged between the lanes c and c ^ 8
// that is row c, block g of both steps.  Scales: kS4, where the rows and the
// base are 4-byte aligned, two dwords of row c (byte g of each is the lane's);
// otherwise two bytes.  Rows past N and blocks past K read zeros: their
// offsets lie past the buffers or have bit 31 set.
template <bool kS4>
struct Reader {
    __amdgpu_buffer_rsrc_t rq, rs;
    unsigned row_bytes, blocks;
    int c, g;

    __device__ __forceinline__ Reader(const uint8_t *qw, const uint8_t *sw, int n0, int rows, int K, int lane)
    {
        blocks = (unsigned)K / 32u;
        row_bytes = (unsigned)K / 2u;
        rq = out_buffer((void *)(qw + (int64_t)n0 * row_bytes), (int64_t)rows * row_bytes);
        rs = out_buffer((void *)(sw + (int64_t)n0 * blocks), (int64_t)rows * blocks);
        c = lane & 15;
        g = lane >> 4;
    }

    // Row tile r of steps 2 p and 2 p + 1.
    __device__ __forceinline__ void load(Pair &v, int r, int p) const
    {
        const unsigned b = 8u * (unsigned)p + (unsigned)(g + 4 * (c >> 3));
        const unsigned drop = (unsigned)(b >= blocks) << 31;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const unsigned row = (unsigned)(16 * r + 8 * h + (c & 7));
            v.w[h] = __builtin_bit_cast(
                u32x4, __builtin_amdgcn_raw_buffer_load_b128(rq, (int)((row * row_bytes + b * 16u) | drop), 0, 0));
        }
        const unsigned at = (unsigned)(16 * r + c) * blocks + 8u * (unsigned)p;
        if constexpr (kS4) {
            const u32x2 s = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rs, (int)at, 0, 0));
            v.s[0] = s[0];
            v.s[1] = s[1];
        } else {
            v.s[0] = __builtin_amdgcn_raw_buffer_load_b8(rs, (int)(at + g), 0, 0);
            v.s[1] = __builtin_amdgcn_raw_buffer_load_b8(rs, (int)(at + 4 + g), 0, 0);
        }
    }

    __device__ __forceinline__ void exchange(Pair &v) const
    {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int a = (int)v.w[0][e], b = (int)v.w[1][e];
            v.w[0][e] = (unsigned)__builtin_amdgcn_update_dpp(a, b, 0x128, 0xF, 0xC, false); // row_ror:8, lanes 8..15
            v.w[1][e] = (unsigned)__builtin_amdgcn_update_dpp(b, a, 0x128, 0xF, 0x3, false); // lanes 0..7
        }
    }

    // The scale of step u of the pair; past K the code is zero, but the byte
    // there is another row's and may be NaN.
    __device__ __forceinline__ float scale(const Pair &v, int u, int p) const
    {
        const unsigned byte = (kS4 ? v.s[u] >> (8 * g) : v.s[u]) & 0xFFu;
        return scale_operand(8u * (unsigned)p + 4u * u + g < blocks ? byte : 0u);
    }
};

// Where the sums go: rows of out are 4-element aligned (vec) or not.
struct Out {
    void *p;
    int bf16, vec;
};

// A finished tile: W rows n + i, i = 0..3, of token m.
__device__ __forceinline__ void store4(const Out &o, const f32x4 &v, int m, int n, int M, int N)
{
    if (m >= M)
        return;
    const int64_t at = (int64_t)m * N + n;
    if (o.bf16) {
        __bf16 *p = (__bf16 *)o.p + at;
        const bf16x2 a = __builtin_convertvector((f32x2){v[0], v[1]}, bf16x2);
        const bf16x2 b = __builtin_convertvector((f32x2){v[2], v[3]}, bf16x2);
        if (o.vec && n < N) {
            *(u32x2 *)p = (u32x2){__builtin_bit_cast(unsigned, a), __builtin_bit_cast(unsigned, b)};
            return;
        }
        const __bf16 e[4] = {a[0], a[1], b[0], b[1]};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + i < N)
                p[i] = e[i];
    } else {
        float *p = (float *)o.p + at;
        if (o.vec && n < N) {
            *(f32x4 *)p = v;
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + i < N)
                p[i] = v[i];
    }
}

// LDS row of x in the first kernel: whole 16-byte pieces, an odd number of
// them modulo 16, so that one piece of 16 tokens lies in 16 different banks.
__host__ __device__ constexpr int x_pitch(int K) { return (K * 2 + 255) / 256 * 256 + 16; }

// All of x in LDS (M K <= kXElems), 16 tokens at most.  kRT tiles of 16 weight
// rows a wave, kW waves that split k pair by pair, kRing pairs of steps in
// registers.
constexpr int kXElems = 32768;

template <int kRT, int kW, int kRing, bool kS4>
__global__ __launch_bounds__(64 * kW, 2) void mx_gemv_kernel(const uint16_t *__restrict__ x,
                                                             const uint8_t *__restrict__ qw,
                                                             const uint8_t *__restrict__ sw, Out out, int M, int N, int K)
{
    __shared__ f32x4 red[kW - 1][kRT][64];
    extern __shared__ __align__(16) unsigned char xs[]; // M rows of x_pitch(K), then 16 zero bytes
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int n0 = (int)blockIdx.x * (16 * kRT);
    const int rows = N - n0 < 16 * kRT ? N - n0 : 16 * kRT;
    const Reader<kS4> in(qw, sw, n0, rows, K, lane);
    const int pairs = (K + 255) / 256, pitch = x_pitch(K);

    Pair ring[kRing][kRT];
#pragma unroll
    for (int i = 0; i < kRing; ++i)
#pragma unroll
        for (int r = 0; r < kRT; ++r)
            in.load(ring[i][r], r, i * kW + wave);
    // four pieces a thread in flight
    const int row_pieces = K / 8, pieces = M * row_pieces;
    for (int i = (int)threadIdx.x; i < pieces; i += 4 * 64 * kW) {
        u32x4 v[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const int p = i + y * 64 * kW;
            v[y] = *(const u32x4 *)(x + (p < pieces ? p : i) * 8);
        }
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const int p = i + y * 64 * kW, m = p / row_pieces;
            if (p < pieces)
                *(u32x4 *)(xs + m * pitch + (p - m * row_pieces) * 16) = v[y];
        }
    }
    const int zeros = M * pitch;
    if (threadIdx.x == 0)
        *(u32x4 *)(xs + zeros) = (u32x4){0, 0, 0, 0};
    __syncthreads();

    f32x4 acc[kRT];
#pragma unroll
    for (int r = 0; r < kRT; ++r)
        acc[r] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
    const int row = c * pitch + g * 64;
    for (int i = 0; i * kW + wave < pairs; i += kRing) {
#pragma unroll
        for (int y = 0; y < kRing; ++y) {
            const int p = (i + y) * kW + wave;
#pragma unroll
            for (int r = 0; r < kRT; ++r)
                in.exchange(ring[y][r]);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int k0 = 256 * p + 128 * u;
                const int at = c < M && k0 + 32 * g < K ? row + 2 * k0 : zeros;
                const int next = c < M && k0 + 32 * g < K ? 16 : 0;
                bf16x8 v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[j] = __builtin_bit_cast(bf16x8, *(const u32x4 *)(xs + at + next * j));
#pragma unroll
                for (int r = 0; r < kRT; ++r) {
                    const float sc = in.scale(ring[y][r], u, p);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(mx_bf16x8(ring[y][r].w[u][j], sc), v[j],
                                                                         acc[r], 0, 0, 0);
                }
            }
#pragma unroll
            for (int r = 0; r < kRT; ++r)
                in.load(ring[y][r], r, p + kRing * kW);
        }
    }
    if (wave) {
#pragma unroll
        for (int r = 0; r < kRT; ++r)
            red[wave - 1][r][lane] = acc[r];
    }
    __syncthreads();
    if (wave)
        return;
#pragma unroll
    for (int r = 0; r < kRT; ++r) {
#pragma unroll
        for (int w = 0; w < kW - 1; ++w)
            acc[r] += red[w][r][lane];
        store4(out, acc[r], c, n0 + 16 * r + 4 * g, M, N);
    }
}

// x through LDS in chunks of kWK pairs of steps, two buffers: kWR waves with a
// row tile each share a pair, kWK of them side by side split k.  kMT tiles of
// 16 tokens.  A chunk lies in LDS as the products read it: piece (pair, step,
// token tile, j) is 64 lanes x 16 bytes, the slots of a group permuted so that
// the pieces of one token, written together, lie in different banks, and so do
// the quads of two groups, read together (64 x 32768 x 8192: 70 us rotated by
// 4 j + g, 63 so).
__device__ __forceinline__ int turned(int c, int j, int g) { return c ^ (2 * j + (g & 1) + 8 * (g >> 1)); }

template <int kMT, int kWR, int kWK, int kRing, bool kS4>
__global__ __launch_bounds__(64 * kWR * kWK, 2) void mx_gemv_chunk_kernel(const uint16_t *__restrict__ x,
                                                                          const uint8_t *__restrict__ qw,
                                                                          const uint8_t *__restrict__ sw, Out out,
                                                                          int M, int N, int K)
{
    constexpr int T = 64 * kWR * kWK;
    constexpr int kPieces = kWK * 2 * kMT * 4 * 64; // of a chunk
    constexpr int kMine = kPieces / T;
    static_assert(kPieces % T == 0, "whole pieces per thread");
    extern __shared__ __align__(16) unsigned char lds[];
    u32x4 *xs = (u32x4 *)lds; // [2][kPieces]
    const int t = (int)threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int wr = wave / kWK, wk = wave % kWK;
    const int n0 = ((int)blockIdx.x * kWR + wr) * 16;
    const int rows = N - n0 < 0 ? 0 : N - n0 < 16 ? N - n0 : 16;
    const Reader<kS4> in(qw, sw, rows > 0 ? n0 : 0, rows, K, lane);
    const __amdgpu_buffer_rsrc_t rx = out_buffer((void *)x, (int64_t)M * K * 2);
    const int chunks = (K + 256 * kWK - 1) / (256 * kWK);

    // this thread's pieces of a chunk: token, and eight k from kk.  Four token
    // tiles with four row tiles keep two chunks on the way, in an order that
    // the compiler leaves alone (it would load them right before they are
    // stored): 64 x 28672 x 8192 75 -> 68 us, 64 x 12288 x 4608 23.2 -> 21.4.
    // The other forms gain nothing, or have no registers for it.
    constexpr bool kOrdered = kMT == 4 && kWR == 4;
    constexpr int kAhead = kOrdered ? 2 : 1;
    static_assert(kRing % kAhead == 0, "a chunk's registers are known at compile time");
    u32x4 xr[kAhead][kMine];
    auto load_x = [&](int ch, u32x4 (&to)[kMine]) {
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int p = t + T * i, token = p / (32 * kWK), kk = p % (32 * kWK);
            const unsigned k = 256u * kWK * (unsigned)ch + 8u * (unsigned)kk;
            const unsigned drop = (unsigned)(k >= (unsigned)K) << 31;
            to[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                  rx, (int)((((unsigned)token * (unsigned)K + k) * 2u) | drop), 0, 0));
        }
    };
    auto store_x = [&](u32x4 *to, const u32x4 (&from)[kMine]) {
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int p = t + T * i, token = p / (32 * kWK), kk = p % (32 * kWK);
            const int pu = kk / 16, gg = kk / 4 % 4, j = kk % 4;
            to[((pu * kMT + token / 16) * 4 + j) * 64 + gg * 16 + turned(token % 16, j, gg)] = from[i];
        }
    };

    // this wave's pair of chunk ch is k pair ch kWK + wk
    Pair ring[kRing];
    load_x(0, xr[0]);
#pragma unroll
    for (int i = 0; i < kRing; ++i)
        in.load(ring[i], 0, i * kWK + wk);
    store_x(xs, xr[0]);
#pragma unroll
    for (int i = 1; i <= kAhead; ++i)
        load_x(i, xr[i % kAhead]);
    f32x4 acc[kMT];
#pragma unroll
    for (int a = 0; a < kMT; ++a)
        acc[a] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
    for (int i = 0; i < chunks; i += kRing) {
#pragma unroll
        for (int z = 0; z < kRing; ++z) {
            const int ch = i + z;
            if (ch >= chunks)
                break;
            // this chunk is written, and every wave is done with the other buffer
            __syncthreads();
            store_x(xs + ((ch + 1) & 1) * kPieces, xr[(z + 1) % kAhead]);
            load_x(ch + 1 + kAhead, xr[(z + 1) % kAhead]); // before the codes that are loaded here: loads complete in order
            if constexpr (kOrdered)
                __builtin_amdgcn_sched_barrier(0);
            const u32x4 *from = xs + (ch & 1) * kPieces + wk * (2 * kMT * 4 * 64);
            Pair &v = ring[z];
            in.exchange(v);
            const int p = ch * kWK + wk;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float sc = in.scale(v, u, p);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bf16x8 w = mx_bf16x8(v.w[u][j], sc);
                    const int slot = j * 64 + g * 16 + turned(c, j, g);
#pragma unroll
                    for (int a = 0; a < kMT; ++a)
                        acc[a] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            w, __builtin_bit_cast(bf16x8, from[(u * kMT + a) * 256 + slot]), acc[a], 0, 0, 0);
                }
            }
            // LDS reads two products ahead (13 x 8960 x 2240: 8.8 -> 8.4 us; the
            // other forms with four token tiles lose by it)
            if constexpr (kMT <= 2 || kOrdered) {
                __builtin_amdgcn_sched_group_barrier(0x100, 2 * kMT, 0);
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                    __builtin_amdgcn_sched_group_barrier(0x008, kMT, 0);
                    if (n < 6)
                        __builtin_amdgcn_sched_group_barrier(0x100, kMT, 0);
                }
            }
            in.load(v, 0, p + kRing * kWK);
        }
    }
    if constexpr (kWK > 1) {
        // the k parts of a row tile, through the chunk buffers
        f32x4 *red = (f32x4 *)lds; // [kWR][kWK - 1][kMT][64]
        __syncthreads();
        if (wk) {
#pragma unroll
            for (int a = 0; a < kMT; ++a)
                red[((wr * (kWK - 1) + wk - 1) * kMT + a) * 64 + lane] = acc[a];
        }
        __syncthreads();
        if (wk)
            return;
#pragma unroll
        for (int a = 0; a < kMT; ++a)
#pragma unroll
            for (int w = 0; w < kWK - 1; ++w)
                acc[a] += red[((wr * (kWK - 1) + w) * kMT + a) * 64 + lane];
    }
#pragma unroll
    for (int a = 0; a < kMT; ++a)
        store4(out, acc[a], 16 * a + c, n0 + 4 * g, M, N);
}

struct GemvArgs {
    const uint16_t *x;
    const uint8_t *qw, *sw;
    Out out;
    int M, N, K;
    hipStream_t stream;
    bool s4() const { return K % 128 == 0 && (uintptr_t)sw % 4 == 0; }
};

template <int kRT, int kW, int kRing>
hipError_t launch_gemv(const GemvArgs &a)
{
    const dim3 grid((unsigned)((a.N + 16 * kRT - 1) / (16 * kRT))), wg(64 * kW);
    const unsigned lds = (unsigned)(a.M * x_pitch(a.K) + 16);
    auto run = [&](auto kernel) {
        const hipError_t e = allow_dynamic_lds((const void *)kernel, 16 * x_pitch(kXElems / 16) + 65536);
        if (e != hipSuccess)
            return e;
        kernel<<<grid, wg, lds, a.stream>>>(a.x, a.qw, a.sw, a.out, a.M, a.N, a.K);
        return hipGetLastError();
    };
    return a.s4() ? run(mx_gemv_kernel<kRT, kW, kRing, true>) : run(mx_gemv_kernel<kRT, kW, kRing, false>);
}

template <int kMT, int kWR, int kWK, int kRing>
hipError_t launch_gemv_chunk(const GemvArgs &a)
{
    const dim3 grid((unsigned)((a.N + 16 * kWR - 1) / (16 * kWR))), wg(64 * kWR * kWK);
    constexpr unsigned lds = 2u * kWK * 2 * kMT * 4 * 64 * 16;
    auto run = [&](auto kernel) {
        const hipError_t e = allow_dynamic_lds((const void *)kernel, (int)lds);
        if (e != hipSuccess)
            return e;
        kernel<<<grid, wg, lds, a.stream>>>(a.x, a.qw, a.sw, a.out, a.M, a.N, a.K);
        return hipGetLastError();
    };
    return a.s4() ? run(mx_gemv_chunk_kernel<kMT, kWR, kWK, kRing, true>)
                  : run(mx_gemv_chunk_kernel<kMT, kWR, kWK, kRing, false>);
}

} // namespace

hipError_t launch_mx_gemv(const uint16_t *x, int64_t M, const uint8_t *qw, const uint8_t *sw, int64_t N, int64_t K,
                          void *out, int bf16, hipStream_t stream)
{
    // vector stores: whole groups of four rows of W, aligned in out
    const int vec = N % 4 == 0 && (uintptr_t)out % (bf16 ? 8 : 16) == 0;
    const GemvArgs a{x, qw, sw, {out, bf16, vec}, (int)M, (int)N, (int)K, stream};
    // Few tokens (x is little next to the rows of W that a workgroup reads):
    // x whole in LDS.  1 x 49152 x 12288: 66 us with two row tiles a wave, 72
    // with one; 1 x 12288 x 4608: 9.7 with one, 11.8 with two; 1 x 4096 x 4096:
    // 5.5 us with eight waves on k, 5.7 with four (1 x 1152 x 1152: 3.6, 3.2).
    // 8 x 8192 x 4096: 9.0 us, in chunks 11.4; 13 x 8960 x 2240: 11.5, 8.4.
    if (M <= 8 && M * K <= kXElems) {
        if (N >= 32768)
            return launch_gemv<2, 4, 2>(a);
        return N <= 4096 && K >= 2048 ? launch_gemv<1, 8, 2>(a) : launch_gemv<1, 4, 2>(a);
    }
    // Chunks: four row tiles a workgroup where that still gives 128 of them
    // (13 x 8960 x 2240: 8.4 us, 10.8 with two; 32 x 4096 x 4096: 13.3, 10.6),
    // eight for many tokens and rows (64 x 32768 x 8192: 64 us, 77 with four).
    const bool four = N / 64 >= 128;
    if (M <= 16)
        return four ? launch_gemv_chunk<1, 4, 2, 4>(a) : launch_gemv_chunk<1, 2, 4, 4>(a);
    if (M <= 32)
        return four ? launch_gemv_chunk<2, 4, 2, 4>(a) : launch_gemv_chunk<2, 2, 4, 4>(a);
    if (N / 128 >= 256)
        return launch_gemv_chunk<4, 8, 1, 4>(a);
    return four ? launch_gemv_chunk<4, 4, 2, 4>(a) : launch_gemv_chunk<4, 2, 2, 4>(a);
}

} // namespace kq
