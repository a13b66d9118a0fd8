// Attention over a paged NVFP4 key/value cache on MI355X (gfx950).
//
//   out = sum_t p_t V[t],   p = softmax over the visible t of scale * q . K[t]
//
// Two kernels: one for sequences of few rows (queries times the heads that share a key
// head), one for many; a call with both kinds launches both, and each leaves the
// other's sequences alone. Positions are split over workgroups where sequences and heads are
// few; a third kernel, or the last workgroup of a few rows, joins the splits in their order.
//
// The softmax is taken in one pass: weights are relative to the largest logit so far, sums
// are rescaled when it rises. Codes times scales have 6 significant bits and are exact in float16,
// so both products are float16 matrix products of exact keys and values.
//
// What bounds it (bfloat16 unless said otherwise; copies on this card reach 4.8 TB/s, large float16 products
// 1.3 PFLOP/s):
//   few rows: the cache's bytes. 64 sequences of 1024 to 8192 positions, 32 query and 8 key heads of 128:
//     95 us, 3.6 TB/s; loading alone takes 84, the instructions alone 72. One sequence of 8192
//     positions: 14.5 us, half of it launch and join.
//   many rows: matrix and vector instructions of two waves a SIMD, which share its issue. 2 prompts
//     of 4096, 32 heads of 128: 320 us, 860 TFLOP/s. 515 float32 queries at 20011 positions:
//     154 us, of which the products of two parts each need 96.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "nvfp4_device.h"
#include "nvfp4_gemv.h"
#include "nvfp4_internal.h"
#include "nvfp4_lds.h"

namespace {

constexpr int64_t kMaxGrid = 0x7FFFFF;          // workgroups of up to 512 threads in 2^32 work items
constexpr int64_t kMaxStride = INT64_C(1) << 40;

struct AttParams {
    const uint8_t *q, *kc, *ks, *vc, *vs;
    const float *gk, *gv;
    uint8_t *out;
    float *lse;
    const int32_t *offsets, *lengths, *table;
    int64_t q_token, q_head;                    // bytes
    uint32_t code_page, scale_page;
    int32_t T, H, B, width, pages, shift, heads, G, D;
    int32_t max_q, max_length, window, causal, dtype;
    int32_t splits, chunk;                      // of a sequence's positions; chunk in tiles of 64
    int32_t few_rows;                           // sequences of so many rows are the rows kernel's
    int32_t row_tiles;                          // at most, for a sequence and key head
    int32_t most_rows;                          // of a partial result
    int32_t join_here;                          // rows kernel: the last workgroup of a tile joins its splits
    uint32_t *tickets;
    float *sums, *norms;                        // partial results: [tile][split][most_rows][D], [..][2]
    float scale;
};

// A sequence's rows of q and positions, clamped.
struct Sequence {
    int32_t first, n, length;
};

__device__ __attribute__((always_inline)) inline Sequence sequence_of(const AttParams &p, int b)
{
    const int32_t first = min(max(p.offsets[b], 0), p.T), end = min(max(p.offsets[b + 1], first), p.T);
    return {first, end - first, min(max(p.lengths[b], 0), p.max_length)};
}

// ------------------------------------------------------------------ rows kernel

typedef float float4_t __attribute__((ext_vector_type(4)));
typedef int32_t int4_t __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
// Weights are 2^(logit - top + 8), where `top` is the row's largest logit when it was last
// looked at: sums are only rescaled when a logit exceeds it by 7, so weights stay below 2^15
// and in float16 are normal numbers from 2^-22 of the largest on (their error is at most 2^-33
// of it below). A row rarely needs that behind its first tile; before, a wave's 32 rows
// rescaled nearly every one (128 values a row: 66 of 400 instructions of a tile).
constexpr float kShift = 8.0f, kSlack = 7.0f;
constexpr int kCus = 256;
// Sequences of up to 64 rows are the rows kernel's, 16 or 32 at a time: 33 sequences' 40 rows at 1000
// visible positions took 24 us in the tile kernel.
constexpr int kFewRows = 64, kJoinHere = 8, kMaxSplits = 64, kTileLeast = 4;

// The head's D values go through the matrix instruction in steps of 32. A lane (row
// lane % 16, g = lane / 16) has 8 of a step's; which 8 is free while q and K agree: runs
// of 128 (64, 32) values are cut into 4 pieces of 16 (8, 4) bytes of codes, piece g the
// lane's, so it reads its codes in one. Value of K step f and lane group g: base + mult * g + add.
template <int D>
struct Steps {
    static constexpr int N = D / 32, n128 = D / 128, n64 = D % 128 / 64, n32 = D % 64 / 32;
    static constexpr int base(int f) { return f < 4 * n128 ? f / 4 * 128 : f < 4 * n128 + 2 * n64 ? n128 * 128 : n128 * 128 + n64 * 64; }
    static constexpr int mult(int f) { return f < 4 * n128 ? 32 : f < 4 * n128 + 2 * n64 ? 16 : 8; }
    static constexpr int add(int f) { return f < 4 * n128 ? f % 4 * 8 : f < 4 * n128 + 2 * n64 ? (f - 4 * n128) * 8 : 0; }
};

// A tile of 64 positions: 4 subtiles of 16 (a page holds whole subtiles). Codes and scales
// of the next tile wait in registers, K's as the products take them; V's codes and scales
// go through the wave's own LDS to be transposed.
template <int D>
struct RowsTile {
    static constexpr int RB = D / 2, SB = D / 16, NB = D / 16;     // bytes of a row's codes, of its scales; blocks
    static constexpr int kRuns = D / 128 + D % 128 / 64 + D % 64 / 32;
    static constexpr int PB = D == 64 ? 8 : 16;                    // bytes of V's codes that a lane loads at once
    static constexpr int kLoads = (16 * RB / PB + 63) / 64;        // of them per subtile
    static constexpr int kScales = NB * 64 * 2;                    // V's scales as float16 [block][64]
    static constexpr int kWave = 64 * RB + kScales;
    // Places of a row's pieces of PB bytes, so that the lanes that read at once, four rows of each
    // subtile, meet more banks: all of them for 64, 128 and 256.
    __device__ static constexpr int swizzle_v(int r)
    {
        return D == 64 || D == 128 ? r / 16 & 3 : D == 192 ? r / 16 & 1 : D == 256 ? (r / 16 * 2 + r % 4 / 2) & 7 : 0;
    }
    using Piece = std::conditional_t<PB == 8, uint2_t, uint4_t>;
    struct Raw {
        uint4_t k128[4][D / 128 ? D / 128 : 1];                    // a lane's codes of each run, and its scales
        uint2_t k64[4];
        uint32_t k32[4], k_scales[4][kRuns];
        Piece v[4][kLoads];
        uint32_t v_scales[(NB + 3) / 4];
    };
};

// 8 neighbouring values of q as float32
__device__ __attribute__((always_inline)) inline void load8(const uint8_t *x, int dtype, float (&v)[8])
{
    if (dtype == NVFP4_F32) {
        __builtin_memcpy(v, x, 32);
        return;
    }
    uint32_t w[4];
    __builtin_memcpy(w, x, 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (dtype == NVFP4_BF16) {
            v[2 * e] = __builtin_bit_cast(float, w[e] << 16);
            v[2 * e + 1] = __builtin_bit_cast(float, w[e] & 0xFFFF0000u);
        } else {
            v[2 * e] = (float)as_h2(w[e]).x;
            v[2 * e + 1] = (float)as_h2(w[e]).y;
        }
    }
}

// A row of q as float16 times 2^e, the largest value in [2^14, 2^15): bfloat16 and float16
// rows are exact so (below 2^-29 of the largest to 2^-40 of it), of float32 ones the second part
// holds what the first leaves. The logits' factor of the row is NaN if a value is not finite.
template <int N, int PARTS>
struct QRow {
    half8_t part[PARTS][N];
};

struct RowScale {
    float sign;                                 // of the factor, or 0: it goes into q
    int e;
    float factor;                               // what is left: positive, or NaN
};

// With a positive factor the largest logit is that of the largest product, and a mask's
// -inf stays -inf through the multiplication.
__device__ __attribute__((always_inline)) inline RowScale row_scale(float top, float factor, bool real, bool finite)
{
    const int e = top > 0.0f ? 15 - __builtin_amdgcn_frexp_expf(top) : 0;
    const float f = real ? __builtin_ldexpf(factor, -e) : 0.0f;
    const bool zero = f == 0.0f;
    return {zero ? 0.0f : f < 0.0f ? -1.0f : 1.0f, e, !finite ? __builtin_nanf("") : zero ? 1.0f : fabsf(f)};
}

template <int N, int PARTS>
__device__ __attribute__((always_inline)) inline void to_parts(const float (&v)[8], const RowScale &scale, QRow<N, PARTS> &q, int f)
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float x = __builtin_ldexpf(v[j] * scale.sign, scale.e);
        const _Float16 high = (_Float16)x;
        q.part[0][f][j] = high;
        if constexpr (PARTS == 2)
            q.part[1][f][j] = (_Float16)(x - (float)high);
    }
}

// Results of one tile of rows, joined over W lots (waves, or splits): weights of
// the lots by their maxima (log2, -inf where a lot saw nothing), and the norm.
struct Norm {
    float top, sum;
};

__device__ __attribute__((always_inline)) inline float weight_of(float top, float above)
{
    return top == -__builtin_inff() ? (above == -__builtin_inff() ? 1.0f : 0.0f) : __builtin_amdgcn_exp2f(top - above);
}

// Row r of a sequence's (head, queries): its place among the T * H rows of out.
__device__ __attribute__((always_inline)) inline int64_t out_row(const AttParams &p, const Sequence &s, int hk, int r)
{
    return (int64_t)(s.first + r / p.G) * p.H + hk * p.G + r % p.G;
}

// N (2 or 4) neighbouring values of a row, divided by the norm and scaled; a row that saw nothing is zero.
template <int N>
__device__ __attribute__((always_inline)) inline void store_values(const AttParams &p, int64_t at, const float (&x)[N], float sum, float gv)
{
    const float f = sum == 0.0f ? 0.0f : gv / sum;
    float v[N];
#pragma unroll
    for (int e = 0; e < N; ++e)
        v[e] = sum == 0.0f ? 0.0f : x[e] * f;
    if (p.dtype == NVFP4_F32) {
        __builtin_memcpy((float *)p.out + at, v, 4 * N);
        return;
    }
    uint32_t w[N / 2];
#pragma unroll
    for (int e = 0; e < N / 2; ++e)
        w[e] = p.dtype == NVFP4_BF16 ? bf16_bits(v[2 * e]) | bf16_bits(v[2 * e + 1]) << 16
                                     : (uint32_t)f16_bits(v[2 * e]) | (uint32_t)f16_bits(v[2 * e + 1]) << 16;
    __builtin_memcpy((uint16_t *)p.out + at, w, 2 * N);
}

__device__ __attribute__((always_inline)) inline void store_lse(const AttParams &p, int64_t row, Norm n)
{
    if (p.lse)
        p.lse[row] = n.sum == 0.0f ? -__builtin_inff() : kLn2 * (n.top - kShift + __builtin_amdgcn_logf(n.sum));
}

// Partial results, two values at a time, past the caches that the XCDs do not share.
typedef float float2_u __attribute__((ext_vector_type(2)));

__device__ __attribute__((always_inline)) inline void store_partial(float *to, float2_u v)
{
    __hip_atomic_store((uint64_t *)to, __builtin_bit_cast(uint64_t, v), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __attribute__((always_inline)) inline float2_u load_partial(const float *from)
{
    return __builtin_bit_cast(float2_u, __hip_atomic_load((const uint64_t *)from, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
}

// Takes the tile's ticket after this workgroup's partial results; true for the last of
// its `splits` workgroups, which clears the ticket. All threads call it.
__device__ __attribute__((always_inline)) inline bool last_of_splits(const AttParams &p, uint32_t tile, int splits, uint32_t *s_ticket)
{
    asm volatile("s_waitcnt vmcnt(0)" : : : "memory");          // this wave's partial results are out
    __syncthreads();
    if (threadIdx.x == 0)
        *s_ticket = __hip_atomic_fetch_add(&p.tickets[tile], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (*s_ticket != (uint32_t)splits - 1)
        return false;
    if (threadIdx.x == 0)
        __hip_atomic_store(&p.tickets[tile], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return true;
}

// Lanes l and l ^ 32 (l ^ 16): both values in both, in one order, without LDS.
struct Both {
    float a, b;
};
__device__ __attribute__((always_inline)) inline Both across32(float v)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
    return {__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1])};
}
__device__ __attribute__((always_inline)) inline Both across16(float v)
{
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
    return {__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1])};
}
// largest (sum) over lanes l and l ^ 32; over l, l ^ 16, l ^ 32, l ^ 48
__device__ __attribute__((always_inline)) inline float max_of_2(float v)
{
    const Both x = across32(v);
    return fmaxf(x.a, x.b);
}
__device__ __attribute__((always_inline)) inline float max_of_4(float v)
{
    const Both x = across16(v);
    return max_of_2(fmaxf(x.a, x.b));
}
__device__ __attribute__((always_inline)) inline float sum_of_2(float v)
{
    const Both x = across32(v);
    return x.a + x.b;
}
__device__ __attribute__((always_inline)) inline float sum_of_4(float v)
{
    const Both x = across16(v);
    return sum_of_2(x.a + x.b);
}

// Over all 64 lanes, in every lane: within rows of 16 by rotations.
template <int N>
__device__ __attribute__((always_inline)) inline float rotated(float v)
{
    return as_f32(__builtin_amdgcn_update_dpp(0, as_i32(v), 0x120 + N, 0xF, 0xF, true));
}
__device__ __attribute__((always_inline)) inline float max_of_64(float v)
{
    v = fmaxf(v, rotated<1>(v));
    v = fmaxf(v, rotated<2>(v));
    v = fmaxf(v, rotated<4>(v));
    return max_of_4(fmaxf(v, rotated<8>(v)));
}
__device__ __attribute__((always_inline)) inline float sum_of_64(float v)
{
    v += rotated<1>(v);
    v += rotated<2>(v);
    v += rotated<4>(v);
    return sum_of_4(v + rotated<8>(v));
}

// Adds the splits' partial results of rows first .. first + rows - 1 of a tile in the order of the
// splits and stores them; row0 is the tile's first row among the sequence's. `weights`: LDS for
// [splits][rows] of them, and behind them for [rows] sums. V values of a row at a time, U such at once,
// AHEAD splits' loads in flight (where fewer are left the last one's again). FENCED: a kernel
// before this one wrote the partial results; else other workgroups of this one, past the
// caches that the XCDs do not share, two values at a time.
template <int D, int THREADS, int V, int U, int AHEAD, bool FENCED>
__device__ __attribute__((always_inline)) inline void join_splits(const AttParams &p, const Sequence &s, int hk, uint32_t tile,
                                                                  int row0, int first, int rows, int splits, float gv, float *weights)
{
    static_assert(kMaxSplits <= 64);
    static_assert(V == 2 || (V == 4 && FENCED));
    const float *sums = p.sums + ((int64_t)tile * p.splits * p.most_rows + first) * D;
    const float *from = p.norms + ((int64_t)tile * p.splits * p.most_rows + first) * 2;
    row0 += first;
    float *const total = weights + splits * rows;
    const int units = rows * (D / V);
    float x[U][AHEAD][V];
    auto load = [&](int u0, int k0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = min(u0 + u * THREADS, units - 1);
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                const float *one = sums + ((int64_t)min(k0 + k, splits - 1) * p.most_rows + at / (D / V)) * D + at % (D / V) * V;
                if constexpr (FENCED) {
                    __builtin_memcpy(x[u][k], __builtin_assume_aligned(one, 4 * V), 4 * V);
                } else {
                    const float2_u y = load_partial(one);
                    x[u][k][0] = y.x, x[u][k][1] = y.y;
                }
            }
        }
    };
    load((int)threadIdx.x, 0);                                  // under way while the weights are found
    // each row's weights of the splits, a lane each: R rows of a wave at once
    constexpr int R = 4, WAVES = THREADS / 64;
    const int lane = (int)threadIdx.x % 64, wave = (int)threadIdx.x / 64;
    for (int r0 = wave; r0 < rows; r0 += R * WAVES) {
        float2_u one[R];
#pragma unroll
        for (int j = 0; j < R; ++j)
            one[j] = load_partial(from + (min(lane, splits - 1) * p.most_rows + min(r0 + j * WAVES, rows - 1)) * 2);
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const int r = r0 + j * WAVES;
            const float top = max_of_64(lane < splits ? one[j].x : -__builtin_inff());
            const float w = lane < splits ? weight_of(one[j].x, top) : 0.0f;
            const float sum = sum_of_64(lane < splits ? one[j].y * w : 0.0f);
            if (r < rows && lane < splits)
                weights[lane * rows + r] = w;
            if (r < rows && lane == 0) {
                total[r] = sum;
                store_lse(p, out_row(p, s, hk, row0 + r), {top, sum});
            }
        }
    }
    __syncthreads();
    for (int u0 = (int)threadIdx.x; u0 < units; u0 += U * THREADS) {
        float v[U][V];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < V; ++e)
                v[u][e] = 0.0f;
        for (int k0 = 0; k0 < splits; k0 += AHEAD) {
            if (u0 != (int)threadIdx.x || k0 != 0)
                load(u0, k0);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = min(u0 + u * THREADS, units - 1) / (D / V);
#pragma unroll
                for (int k = 0; k < AHEAD; ++k)
                    if (k0 + k < splits) {
                        const float w = weights[(k0 + k) * rows + r];
#pragma unroll
                        for (int e = 0; e < V; ++e)
                            v[u][e] += x[u][k][e] * w;
                    }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = u0 + u * THREADS;
            if (at < units)
                store_values<V>(p, out_row(p, s, hk, row0 + at / (D / V)) * D + at % (D / V) * V, v[u], total[at / (D / V)], gv);
        }
    }
}

// Which of a sequence's positions a workgroup takes: tiles of 64 from `lo` on.
struct Span {
    int32_t lo, hi;                             // visible to some row of the tile
    int32_t first, end;                         // tiles of this workgroup, counted from lo / 64
    int32_t splits;                             // that take part
};

// Rows of queries tok0 .. tok1 - 1.
__device__ __attribute__((always_inline)) inline Span span_of(const AttParams &p, const Sequence &s, int tok0, int tok1, int split)
{
    Span v;
    v.hi = p.causal ? max(0, min(s.length, s.length - s.n + tok1)) : s.length;
    v.lo = p.window ? max(0, s.length - s.n + tok0 - p.window + 1) : 0;
    const int32_t tiles = v.hi > v.lo ? (v.hi - v.lo / 64 * 64 + 63) / 64 : 0;
    const int32_t chunk = max(p.chunk, (tiles + p.splits - 1) / p.splits);
    v.splits = max(1, (tiles + chunk - 1) / chunk);
    v.first = min(tiles, split * chunk);
    v.end = min(tiles, v.first + chunk);
    return v;
}

// Accesses to LDS of this wave's lanes stay on their side of this point. The hardware
// carries a wave's out in order; nothing is waited for.
__device__ __attribute__((always_inline)) inline void settle_order()
{
    asm volatile("" : : : "memory");
    __builtin_amdgcn_wave_barrier();
}

// Few rows: n queries times the heads that share a key head, at most 16 * NQ. Every wave
// takes tiles of 64 positions in turn; the next one's codes and scales come while it works on one.
//   S^T = K Q^T by 16 x 16 x 32 products, K the first operand: a lane then has the logits
//     of one row (lane % 16), positions 16 a + 4 g + b in register b of subtile a.
//   O^T = V^T P^T: a lane's P registers are its k-range as they stand, if V's operand has the same
//     order. Its codes come from LDS transposed (16 positions of one value per
//     lane), so a pair of codes is two positions, and so is a pair of scales.
template <int D, int NQ, bool F32, int WAVES>
__global__ __launch_bounds__(64 * WAVES, WAVES == 8 ? 2 : D <= 64 && NQ == 1 ? 4 : D <= 128 || NQ == 1 ? 2 : 1) void nvfp4_attention_rows_kernel(AttParams p)
{
    using S = RowsTile<D>;
    using St = Steps<D>;
    constexpr int PARTS = F32 ? 2 : 1, NB = S::NB;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    __shared__ uint32_t s_ticket;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / 64), lane = (int)threadIdx.x % 64;
    const int i = lane % 16, g = lane / 16;
    // Splits outermost: neighbouring workgroups, which run on different XCDs, are different
    // sequences and heads. (Innermost, every XCD had one of the splits: those whose splits
    // lie behind most sequences' ends stood idle, 172 us for 64 sequences of 1024 to 8192 positions.)
    const uint32_t pairs = (uint32_t)p.B * (uint32_t)p.heads, tiles = pairs * (uint32_t)p.row_tiles, tile = blockIdx.x % tiles;
    const int split = (int)(blockIdx.x / tiles), row0 = (int)(tile / pairs) * 16 * NQ;
    const int b = (int)(tile % pairs / (uint32_t)p.heads), hk = (int)(tile % pairs % (uint32_t)p.heads);
    const Sequence s = sequence_of(p, b);
    const int queries = min(s.n, p.max_q);
    if (queries > kFewRows || queries * p.G > p.few_rows || row0 >= queries * p.G)
        return;
    const int rows = min(16 * NQ, queries * p.G - row0);
    const int tok0 = row0 / p.G, tok1 = (row0 + rows - 1) / p.G + 1;
    const Span span = span_of(p, s, tok0, tok1, split);
    if (split >= span.splits)
        return;

    float4_t acc[NQ][NB];
    float top[NQ], sum[NQ];
    uint32_t nan_blocks[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        top[n] = -__builtin_inff();
        sum[n] = 0.0f;
        nan_blocks[n] = 0u;
#pragma unroll
        for (int k = 0; k < NB; ++k)
            acc[n][k] = {0.0f, 0.0f, 0.0f, 0.0f};
    }

    // --- loads
    uint8_t *const mine = lds + wave * S::kWave;
    const int32_t mask = (1 << p.shift) - 1;
    const int32_t first_position = span.lo / 64 * 64;
    const int32_t *const table = p.table + (int64_t)b * p.width;
    auto entry_of = [&](int32_t n, int a) -> int32_t {
        const int32_t t = first_position + n * 64 + a * 16;
        return n < span.end && t < span.hi ? table[t >> p.shift] : -1;
    };
    auto entries = [&](int32_t n) -> int4_t { return {entry_of(n, 0), entry_of(n, 1), entry_of(n, 2), entry_of(n, 3)}; };
    // A subtile that is not there is read from the cache's first page; its bit is 0.
    typename S::Raw raw;
    auto there_of = [&](int4_t e) -> uint32_t {
        uint32_t there = 0u;
#pragma unroll
        for (int a = 0; a < 4; ++a)
            there |= (uint32_t)((uint32_t)e[a] < (uint32_t)p.pages) << a;
        return there;
    };
    auto page_of = [&](int32_t e) -> uint64_t { return (uint32_t)e < (uint32_t)p.pages ? (uint32_t)e : 0u; };
    auto row_of = [&](int32_t n, int a) -> uint32_t {
        return ((uint32_t)hk << p.shift) + (uint32_t)((first_position + n * 64 + a * 16) & mask);
    };
    auto load_k = [&](int32_t n, int4_t e, int a) {
        const uint64_t page = page_of(e[a]);
        const uint32_t row = row_of(n, a);
        const uint8_t *codes = p.kc + (page * p.code_page + row * S::RB), *scales = p.ks + (page * p.scale_page + row * S::SB);
#pragma unroll
        for (int x = 0; x < St::n128; ++x) {
            raw.k128[a][x] = *(const uint4_t *)(codes + (uint32_t)(i * S::RB + 64 * x + 16 * g));
            raw.k_scales[a][x] = *(const uint16_t *)(scales + (uint32_t)(i * S::SB + 8 * x + 2 * g));
        }
        if constexpr (St::n64 != 0) {
            raw.k64[a] = *(const uint2_t *)(codes + (uint32_t)(i * S::RB + 64 * St::n128 + 8 * g));
            raw.k_scales[a][St::n128] = scales[(uint32_t)(i * S::SB + 8 * St::n128 + g)];
        }
        if constexpr (St::n32 != 0) {
            raw.k32[a] = *(const uint32_t *)(codes + (uint32_t)(i * S::RB + 64 * St::n128 + 32 * St::n64 + 4 * g));
            raw.k_scales[a][S::kRuns - 1] = scales[(uint32_t)(i * S::SB + 8 * St::n128 + 4 * St::n64 + g / 2)];
        }
    };
    // V's codes as they lie; lanes behind a subtile's end read its start again
    auto load_v = [&](int32_t n, int4_t e) {
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            const uint8_t *codes = p.vc + (page_of(e[a]) * p.code_page + row_of(n, a) * S::RB);
#pragma unroll
            for (int c = 0; c < S::kLoads; ++c) {
                const uint32_t o = (uint32_t)(c * 64 + lane) * S::PB;
                raw.v[a][c] = *(const typename S::Piece *)(codes + (o < 16 * S::RB ? o : 0u));
            }
        }
        // a lane has the scales of one position
        const int32_t mine_e = lane < 32 ? (lane < 16 ? e[0] : e[1]) : (lane < 48 ? e[2] : e[3]);
        const uint32_t row = ((uint32_t)hk << p.shift) + (uint32_t)((first_position + n * 64 + lane) & mask);
        const uint8_t *scales = p.vs + (page_of(mine_e) * p.scale_page + row * S::SB);
        if constexpr (S::SB % 4 == 0) {
#pragma unroll
            for (int k = 0; k < S::SB / 4; ++k)
                raw.v_scales[k] = ((const uint32_t *)scales)[k];
        } else {
            const uint16_t *two = (const uint16_t *)scales;
            raw.v_scales[0] = (uint32_t)two[0] | (uint32_t)two[1] << 16;
            raw.v_scales[1] = two[2];
        }
    };

    // the first tile's loads are out before q's
    int32_t n = span.first + wave;
    int4_t e = entries(n);
    uint32_t there = there_of(e);
    load_v(n, e);
#pragma unroll
    for (int a = 0; a < 4; ++a)
        load_k(n, e, a);
    e = entries(n + WAVES);

    // --- this lane's rows of q
    const float factor = p.scale * (p.gk ? *p.gk : 1.0f) * kLog2e;
    QRow<St::N, PARTS> q[NQ];
    float rf[NQ];
    int32_t begin[NQ], end[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        const int r = row0 + 16 * n + i, tok = r / p.G, pos = s.length - s.n + tok;
        const bool real = r < row0 + rows;
        end[n] = p.causal ? min(s.length, pos + 1) : s.length;
        begin[n] = p.window ? max(0, pos - p.window + 1) : 0;
        const uint8_t *x = p.q + (int64_t)(s.first + (real ? tok : 0)) * p.q_token +
                           (int64_t)(hk * p.G + (real ? r % p.G : 0)) * p.q_head;
        float v[St::N][8], top = 0.0f;
        bool finite = true;
#pragma unroll
        for (int f = 0; f < St::N; ++f) {
            load8(x + (St::base(f) + St::mult(f) * g + St::add(f)) * (F32 ? 4 : 2), F32 ? NVFP4_F32 : p.dtype, v[f]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool good = __builtin_isfinite(v[f][j]);
                finite &= good;
                v[f][j] = good ? v[f][j] : 0.0f;
                top = fmaxf(top, fabsf(v[f][j]));
            }
        }
        top = max_of_4(top);
        finite = max_of_4(finite ? 0.0f : 1.0f) == 0.0f;
        const RowScale scale = row_scale(top, factor, real, finite);
#pragma unroll
        for (int f = 0; f < St::N; ++f)
            to_parts(v[f], scale, q[n], f);
        rf[n] = scale.factor;
    }
    // positions that all rows see: no mask within them
    const int32_t all_from = p.window ? max(0, s.length - s.n + tok1 - p.window) : 0;
    const int32_t all_to = p.causal ? min(s.length, s.length - s.n + tok0 + 1) : s.length;

    // --- the loop: what the next tile needs is loaded as soon as its registers are free
    for (; n < span.end; n += WAVES) {
        const int32_t t0 = first_position + n * 64;
        // --- V's codes and, as float16 in the order of the k-ranges, its scales to LDS; a position that no
        // row sees has 0 there, and so has a NaN, which is noted for the rows that see it
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int c = 0; c < S::kLoads; ++c) {
                const int o = c * 64 + lane, r = 16 * a + o / (S::RB / S::PB), piece = o % (S::RB / S::PB);
                if (16 * S::RB % (64 * S::PB) == 0 || o < 16 * S::RB / S::PB)
                    *(typename S::Piece *)(mine + r * S::RB + (piece ^ S::swizzle_v(r)) * S::PB) = raw.v[a][c];
            }
        {
            const int32_t t = t0 + lane;
            const bool seen = (there >> (lane / 16) & 1u) && t >= span.lo && t < span.hi;
            uint32_t nan = 0u;
            uint32_t w[(NB + 3) / 4];
#pragma unroll
            for (int k = 0; k < (NB + 3) / 4; ++k) {
                w[k] = seen ? raw.v_scales[k] : 0u;
                nan |= ((w[k] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;      // bytes of 0x7F and 0xFF
            }
            uint64_t left = __ballot(nan != 0u);
            if (left) {
                asm volatile("" : : : "memory");
                uint32_t bad_blocks = 0u;
#pragma unroll
                for (int k = 0; k < NB; ++k) {
                    const bool bad = (w[k / 4] >> (8 * (k % 4)) & 0x7Fu) == 0x7Fu;
                    bad_blocks |= (uint32_t)bad << k;
                    w[k / 4] &= bad ? ~(0xFFu << (8 * (k % 4))) : ~0u;
                }
                while (left) {
                    const int k = __builtin_ctzll(left);
                    left &= left - 1;
                    const uint32_t blocks = (uint32_t)__builtin_amdgcn_readlane((int)bad_blocks, k);
#pragma unroll
                    for (int m = 0; m < NQ; ++m)
                        if (t0 + k >= begin[m] && t0 + k < end[m])
                            nan_blocks[m] |= blocks;
                }
            }
            _Float16 *to = (_Float16 *)(mine + 64 * S::RB) + (lane / 4 % 4) * 16 + lane / 16 * 4 + lane % 4;
#pragma unroll
            for (int k = 0; k < NB; k += 4) {
                const half2_t low = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[k / 4], 1.0f, false);
                to[k * 64] = low.x;
                to[k * 64 + 64] = low.y;
                if (k + 2 < NB) {
                    const half2_t high = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[k / 4], 1.0f, true);
                    to[k * 64 + 128] = high.x;
                    to[k * 64 + 192] = high.y;
                }
            }
        }
        load_v(n + WAVES, e);
        // --- S^T
        float logit[NQ][4][4];
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            float4_t c[NQ];
#pragma unroll
            for (int m = 0; m < NQ; ++m)
                c[m] = {0.0f, 0.0f, 0.0f, 0.0f};
            auto step = [&](int f, uint32_t w, half2_t s2) {
                const half8_t k8 = decode8(w, s2);
#pragma unroll
                for (int m = 0; m < NQ; ++m)
#pragma unroll
                    for (int part = 0; part < PARTS; ++part)
                        c[m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k8, q[m].part[part][f], c[m], 0, 0, 0);
            };
#pragma unroll
            for (int x = 0; x < S::kRuns; ++x) {
                const half2_t both = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(raw.k_scales[a][x], 1.0f, false);
                const half2_t s0 = {both.x, both.x}, s1 = {both.y, both.y};
                if (x < St::n128) {
                    const uint4_t w = raw.k128[a][x < St::n128 ? x : 0];
                    step(4 * x, w.x, s0);
                    step(4 * x + 1, w.y, s0);
                    step(4 * x + 2, w.z, s1);
                    step(4 * x + 3, w.w, s1);
                } else if (x < St::n128 + St::n64) {
                    step(4 * St::n128, raw.k64[a].x, s0);
                    step(4 * St::n128 + 1, raw.k64[a].y, s0);
                } else {
                    step(St::N - 1, raw.k32[a], s0);
                }
            }
            load_k(n + WAVES, e, a);
#pragma unroll
            for (int m = 0; m < NQ; ++m)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    logit[m][a][x] = c[m][x];
        }
        if (there != 15u || t0 < all_from || t0 + 64 > all_to) {
#pragma unroll
            for (int m = 0; m < NQ; ++m) {
                // what this lane's row sees of its positions, bit 16 a + x for register x of subtile a
                int32_t from = begin[m] - t0, to = end[m] - t0;
                asm volatile("" : "+v"(from), "+v"(to));                // a branch, not 16 selects in every tile
                uint64_t seen = ((there & 1u ? 0xFFFFull : 0ull) | (there & 2u ? 0xFFFFull << 16 : 0ull)) |
                                ((there & 4u ? 0xFFFFull << 32 : 0ull) | (there & 8u ? 0xFFFFull << 48 : 0ull));
                seen = from <= 0 ? seen : from < 64 ? seen & ~0ull << from : 0ull;
                seen = to >= 64 ? seen : to > 0 ? seen & ~(~0ull << to) : 0ull;
                seen >>= 4 * g;
#pragma unroll
                for (int a = 0; a < 4; ++a)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        logit[m][a][x] = (uint32_t)(seen >> (32 * (a / 2))) >> (16 * (a % 2) + x) & 1u ? logit[m][a][x] : -__builtin_inff();
            }
        }
        there = there_of(e);
        e = entries(n + 2 * WAVES);
        // --- softmax
        half8_t prob[PARTS][NQ][2];
#pragma unroll
        for (int m = 0; m < NQ; ++m) {
            float most = logit[m][0][0];
#pragma unroll
            for (int k = 1; k < 16; ++k)
                most = fmaxf(most, logit[m][k / 4][k % 4]);
            most = fmaxf(top[m], max_of_4(most) * rf[m]);
            if (__ballot(most > top[m] + kSlack)) {
                const float keep = weight_of(top[m], most);
                sum[m] *= keep;
#pragma unroll
                for (int k = 0; k < NB; ++k)
                    acc[m][k] *= keep;
                top[m] = most;
            }
            const float less = kShift - (top[m] == -__builtin_inff() ? 0.0f : top[m]);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const float w = __builtin_amdgcn_exp2f(fmaf(logit[m][k / 4][k % 4], rf[m], less));
                sum[m] += w;
                const _Float16 high = (_Float16)w;
                prob[0][m][k / 8][k % 8] = high;
                if constexpr (PARTS == 2)
                    prob[PARTS - 1][m][k / 8][k % 8] = (_Float16)(w - (float)high);
            }
        }
        // --- O^T. A wave's accesses to LDS are carried out in order: V is there when it is read.
        settle_order();
        const int vr = 16 * (i / 4) + 4 * g + i % 4;
        const uint8_t *row = mine + vr * S::RB;
        const int sw = S::swizzle_v(vr);
        const uint8_t *sc = mine + 64 * S::RB + g * 32;
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const int at = S::PB == 8 ? (k ^ sw) * 8 : ((k / 2) ^ sw) * 16 + k % 2 * 8;
            const uint2_t w = read_transposed4(row + at);
            const uint4_t a0 = *(const uint4_t *)(sc + k * 128), a1 = *(const uint4_t *)(sc + k * 128 + 16);
            const half8_t v0 = decode8_by(w.x, a0), v1 = decode8_by(w.y, a1);
#pragma unroll
            for (int m = 0; m < NQ; ++m)
#pragma unroll
                for (int part = 0; part < PARTS; ++part) {
                    acc[m][k] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, prob[part][m][0], acc[m][k], 0, 0, 0);
                    acc[m][k] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, prob[part][m][1], acc[m][k], 0, 0, 0);
                }
        }
        settle_order();
    }

    // --- the waves' results through LDS: sums [wave][16 NQ][D], norms
    __syncthreads();                                                   // every wave's V is read
    float *const w_sums = (float *)lds;
    Norm *const w_norms = (Norm *)(lds + WAVES * 16 * NQ * D * 4);
#pragma unroll
    for (int m = 0; m < NQ; ++m) {
        sum[m] = sum_of_4(sum[m]);
        const int r = wave * 16 * NQ + 16 * m + i;
        if (g == 0)
            w_norms[r] = {top[m], sum[m]};
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            float4_t v = acc[m][k];
            if (nan_blocks[m] >> k & 1u)
                v = {__builtin_nanf(""), __builtin_nanf(""), __builtin_nanf(""), __builtin_nanf("")};
            *(float4_t *)(w_sums + r * D + 16 * k + 4 * g) = v;
        }
    }
    __syncthreads();
    const float gv = p.gv ? *p.gv : 1.0f;
    float *const sums = p.sums + ((int64_t)tile * p.splits + split) * p.most_rows * D;
    float *const norms = p.norms + ((int64_t)tile * p.splits + split) * p.most_rows * 2;
    for (int u = (int)threadIdx.x; u < rows * (D / 4); u += (64 * WAVES)) {
        const int r = u / (D / 4), d = u % (D / 4) * 4;
        Norm all{-__builtin_inff(), 0.0f};
#pragma unroll
        for (int w = 0; w < WAVES; ++w)
            all.top = fmaxf(all.top, w_norms[w * 16 * NQ + r].top);
        float4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const Norm one = w_norms[w * 16 * NQ + r];
            const float part = weight_of(one.top, all.top);
            all.sum += one.sum * part;
            v += *(const float4_t *)(w_sums + (w * 16 * NQ + r) * D + d) * part;
        }
        if (span.splits == 1) {
            const int64_t row = out_row(p, s, hk, row0 + r);
            store_values<4>(p, row * D + d, {v.x, v.y, v.z, v.w}, all.sum, gv);
            if (d == 0)
                store_lse(p, row, all);
            continue;
        }
        if (p.join_here) {
            store_partial(sums + r * D + d, (float2_u){v.x, v.y});
            store_partial(sums + r * D + d + 2, (float2_u){v.z, v.w});
            if (d == 0)
                store_partial(norms + r * 2, (float2_u){all.top, all.sum});
        } else {
            *(float4_t *)(sums + r * D + d) = v;
            if (d == 0)
                *(Norm *)(norms + r * 2) = all;
        }
    }
    if (span.splits == 1 || !p.join_here || !last_of_splits(p, tile, span.splits, &s_ticket))
        return;
    join_splits<D, 64 * WAVES, 2, 1, 8, false>(p, s, hk, tile, row0, 0, rows, span.splits, gv, (float *)lds);
}

// ------------------------------------------------------------------ tile kernel

typedef float float16_t __attribute__((ext_vector_type(16)));

// Rows of a wave: 32, or 16 where the sums and queries of 32 do not fit into 256 registers
// (D = 256 with 32 rows, one wave on a SIMD: 772 us for 2 x 2048 queries at 2048 to 4096
// positions, 8 heads of 32). Waves of a workgroup.
constexpr int wave_rows(int D, bool f32) { return D == 256 || (D == 192 && f32) ? 16 : 32; }
constexpr int tile_waves(int D, bool f32) { return D >= 192 ? 8 : 4; }
constexpr int tile_rows(int D, bool f32) { return wave_rows(D, f32) * tile_waves(D, f32); }

// 64 positions in LDS as float16, [position][D] for K and for V. Places of a row's 16-byte
// pieces: 16 neighbouring rows meet every bank where K is read, 64 bytes of 4 neighbouring rows
// do where V is read, and 4 pieces of 4 neighbouring rows where either is written (less well for 96).
template <int D, int THREADS>
struct WideTile {
    static constexpr int kRow = 2 * D, kBytes = 64 * kRow, kBuffer = 2 * kBytes, PR = D / 32;  // pieces of 32 codes in a row
    static constexpr int kPieces = (2 * 64 * PR + THREADS - 1) / THREADS;
    __device__ static constexpr int swizzle_k(int t)
    {
        return D == 64 || D == 192 ? t / 2 & 7 : D == 96 ? t / 4 & 3 : t & 15;
    }
    __device__ static constexpr int swizzle_v(int t)
    {
        return D == 64 || D == 192 ? (t / 2 & 1) * 4 + (t / 2 & 3) : D == 96 ? t / 4 & 3 : (t & 3) * 4 + ((t & 3) ^ (t / 4 & 1) * 2);
    }
};

__device__ __attribute__((always_inline)) inline void lds_barrier()
{
    asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" : : : "memory");
}

// Many rows (prompts): a workgroup has 128 or 256 of a sequence's rows for one key head, a wave RW = 32 or
// 16 of them. Codes of 64 positions come in registers while the 64 before are worked on, are
// decoded once for all rows into LDS, and go through 32 x 32 x 16 (16 x 16 x 32) products:
//   S^T = K Q^T: a lane has the logits of one row (lane % RW), positions RW t + 8 (r / 4) + 4 h
//     + r % 4 in register r (h = lane / RW).
//   O^T = V^T P^T: P's registers are the k-range of the second operand as they stand; V's operand is read
//     transposed in that order, 4 positions of a value at a time.
template <int RW>
struct Product;
template <>
struct Product<32> {
    using Sum = float16_t;
    static constexpr int kValues = 16, kStep = 16;
    __device__ static __attribute__((always_inline)) inline Sum of(half8_t a, half8_t b, Sum c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    }
    __device__ static __attribute__((always_inline)) inline float max_of(float v) { return max_of_2(v); }
    __device__ static __attribute__((always_inline)) inline float sum_of(float v) { return sum_of_2(v); }
};
template <>
struct Product<16> {
    using Sum = float4_t;
    static constexpr int kValues = 4, kStep = 32;
    __device__ static __attribute__((always_inline)) inline Sum of(half8_t a, half8_t b, Sum c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
    __device__ static __attribute__((always_inline)) inline float max_of(float v) { return max_of_4(v); }
    __device__ static __attribute__((always_inline)) inline float sum_of(float v) { return sum_of_4(v); }
};

template <int D, bool F32>
__global__ __launch_bounds__(64 * tile_waves(D, F32), 2) void nvfp4_attention_tile_kernel(AttParams p)
{
    constexpr int kTileThreads = 64 * tile_waves(D, F32), kTileRows = tile_rows(D, F32);
    using S = WideTile<D, kTileThreads>;
    constexpr int RW = wave_rows(D, F32);
    using M = Product<RW>;
    // All 64 positions at once, or 32 after the other, where the logits of 64 do not fit into 256 registers
    // beside sums and queries.
    constexpr int GROUPS = RW == 32 && (D > 128 || F32) ? 2 : 1, TT = 64 / RW / GROUPS, NV = M::kValues;
    constexpr int PARTS = F32 ? 2 : 1, NK = D / M::kStep, ND = D / RW;
    // The products of K (of V) go before the other wave's vector instructions where that is faster: 2 x 4096
    // queries, 32 heads of 128, 323 us for 335 with K's, 359 with V's; 8 heads of 256, 2048 queries, 568 for 625
    // with both
    constexpr bool kFirst = RW == 32 || !F32, kSecond = RW == 16 && !F32;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    __shared__ uint32_t s_flag[3], s_nan[3][64];
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / 64), lane = (int)threadIdx.x % 64;
    const int i = lane % RW, h = lane / RW;
    // the last rows, which see most under the causal mask, first
    const uint32_t pairs = (uint32_t)p.B * (uint32_t)p.heads, tiles = pairs * (uint32_t)p.row_tiles, id = blockIdx.x % tiles;
    const int split = (int)(blockIdx.x / tiles), rt = (int)(((uint32_t)p.row_tiles - 1u) - id / pairs);
    const int b = (int)(id % pairs / (uint32_t)p.heads), hk = (int)(id % pairs % (uint32_t)p.heads);
    const Sequence s = sequence_of(p, b);
    const int queries = min(s.n, p.max_q);
    const int64_t all_rows = (int64_t)queries * p.G;
    if (all_rows <= p.few_rows || (int64_t)rt * kTileRows >= all_rows)
        return;
    const int row0 = rt * kTileRows, rows = (int)min((int64_t)kTileRows, all_rows - row0);
    const int tok0 = row0 / p.G, tok1 = (row0 + rows - 1) / p.G + 1;
    const Span span = span_of(p, s, tok0, tok1, split);
    if (split >= span.splits)
        return;

    // --- this lane's row of q
    const int r = RW * wave + i;
    const bool real = r < rows;
    const int tok = (row0 + (real ? r : 0)) / p.G, pos = s.length - s.n + tok;
    const int32_t end = p.causal ? min(s.length, pos + 1) : s.length;
    const int32_t begin = p.window ? max(0, pos - p.window + 1) : 0;
    QRow<NK, PARTS> q;
    float rf;
    {
        const float factor = p.scale * (p.gk ? *p.gk : 1.0f) * kLog2e;
        const uint8_t *x = p.q + (int64_t)(s.first + tok) * p.q_token + (int64_t)(hk * p.G + (row0 + (real ? r : 0)) % p.G) * p.q_head;
        // twice from memory, so that the row is not held as float32
        float top = 0.0f;
        bool finite = true;
        auto piece = [&](int c, float (&v)[8]) { load8(x + (M::kStep * c + 8 * h) * (F32 ? 4 : 2), F32 ? NVFP4_F32 : p.dtype, v); };
#pragma unroll
        for (int c = 0; c < NK; ++c) {
            float v[8];
            piece(c, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool good = __builtin_isfinite(v[j]);
                finite &= good;
                top = fmaxf(top, good ? fabsf(v[j]) : 0.0f);
            }
        }
        top = M::max_of(top);
        finite = M::max_of(finite ? 0.0f : 1.0f) == 0.0f;
        const RowScale scale = row_scale(top, factor, real, finite);
        asm volatile("" : : : "memory");
#pragma unroll
        for (int c = 0; c < NK; ++c) {
            float v[8];
            piece(c, v);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = __builtin_isfinite(v[j]) ? v[j] : 0.0f;
            to_parts(v, scale, q, c);
        }
        rf = scale.factor;
    }
    // positions that some, and that all, of the wave's rows see
    const int w0 = min(RW * wave, rows - 1), w1 = min(RW * wave + RW - 1, rows - 1);
    const int32_t pos0 = s.length - s.n + (row0 + w0) / p.G, pos1 = s.length - s.n + (row0 + w1) / p.G;
    const int32_t some_from = p.window ? max(0, pos0 - p.window + 1) : 0, some_to = p.causal ? min(s.length, pos1 + 1) : s.length;
    const int32_t all_from = p.window ? max(0, pos1 - p.window + 1) : 0, all_to = p.causal ? min(s.length, pos0 + 1) : s.length;
    const bool has_rows = RW * wave < rows;

    typename M::Sum acc[ND];
#pragma unroll
    for (int k = 0; k < ND; ++k)
#pragma unroll
        for (int x = 0; x < NV; ++x)
            acc[k][x] = 0.0f;
    float top = -__builtin_inff(), sum = 0.0f;
    uint32_t nan_blocks = 0u;

    // --- staging. The table's entry of position lane of a tile, -1 past the end. It is not looked
    // at before the next round: a wait for it would wait for the loads before it too.
    const int32_t mask = (1 << p.shift) - 1, first_position = span.lo / 64 * 64;
    const int32_t *const table = p.table + (int64_t)b * p.width;
    const uint32_t tid = threadIdx.x % kTileThreads;            // known to be below kTileThreads
    auto entry = [&](int32_t n) -> int32_t {
        const int32_t t = first_position + n * 64 + lane;
        return n < span.end && t < span.hi ? table[t >> p.shift] : -1;
    };
    auto page_of = [&](int32_t e) -> int32_t { return (uint32_t)e < (uint32_t)p.pages ? e : -1; };
    uint4_t codes[S::kPieces];
    uint32_t scales[S::kPieces];
    auto load = [&](int32_t n, int32_t e) {
#pragma unroll
        for (int k = 0; k < S::kPieces; ++k) {
            const int u = k * kTileThreads + (int)tid, v = u % (64 * S::PR), t = v / S::PR, piece = v % S::PR;
            const int32_t page = __shfl(e, t);
            codes[k] = (uint4_t){0u, 0u, 0u, 0u};
            scales[k] = 0u;
            if (page < 0 || u >= 2 * 64 * S::PR)
                continue;
            const bool values = u >= 64 * S::PR;
            const int64_t row = ((int64_t)hk << p.shift) + ((first_position + n * 64 + t) & mask);
            codes[k] = *(const uint4_t *)((values ? p.vc : p.kc) + (uint64_t)(uint32_t)page * p.code_page + row * (D / 2) + piece * 16);
            scales[k] = *(const uint16_t *)((values ? p.vs : p.ks) + (uint64_t)(uint32_t)page * p.scale_page + row * (D / 16) + piece * 2);
        }
    };
    auto stage = [&](uint8_t *buffer, int slot) {
#pragma unroll
        for (int k = 0; k < S::kPieces; ++k) {
            const int u = k * kTileThreads + (int)tid, v = u % (64 * S::PR), t = v / S::PR, piece = v % S::PR;
            if (2 * 64 * S::PR % kTileThreads != 0 && u >= 2 * 64 * S::PR)
                continue;
            const bool values = u >= 64 * S::PR;
            half2_t both = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(scales[k], 1.0f, false);
            if (values) {
                // a NaN scale is noted for the rows that see it and counts as 0 in the products
                const uint32_t nan = (uint32_t)((scales[k] & 0x7Fu) == 0x7Fu) | (uint32_t)((scales[k] & 0x7F00u) == 0x7F00u) << 1;
                if (nan) {
                    atomicOr(&s_nan[slot][t], nan << (2 * piece));
                    s_flag[slot] = 1u;
                    both.x = nan & 1u ? (_Float16)0.0f : both.x;
                    both.y = nan & 2u ? (_Float16)0.0f : both.y;
                }
            }
            const half2_t s0 = {both.x, both.x}, s1 = {both.y, both.y};
            uint8_t *row = buffer + (values ? S::kBytes : 0) + t * S::kRow;
            const int sw = values ? S::swizzle_v(t) : S::swizzle_k(t);
            *(half8_t *)(row + ((4 * piece) ^ sw) * 16) = decode8(codes[k].x, s0);
            *(half8_t *)(row + ((4 * piece + 1) ^ sw) * 16) = decode8(codes[k].y, s0);
            *(half8_t *)(row + ((4 * piece + 2) ^ sw) * 16) = decode8(codes[k].z, s1);
            *(half8_t *)(row + ((4 * piece + 3) ^ sw) * 16) = decode8(codes[k].w, s1);
        }
    };

    if (threadIdx.x < 64) {
        s_nan[0][threadIdx.x] = s_nan[1][threadIdx.x] = s_nan[2][threadIdx.x] = 0u;
        s_flag[0] = s_flag[1] = s_flag[2] = 0u;
    }
    // One barrier a tile: behind it this tile's buffer is filled and the other one read. While the
    // products of K are under way the next tile is decoded, and the one after it loaded.
    int32_t e = -1;
    uint64_t there = 0ull, next = 0ull;
    if (span.first < span.end) {
        e = page_of(entry(span.first));
        there = __ballot(e >= 0);
        load(span.first, e);
        e = page_of(entry(span.first + 1));
        lds_barrier();                                          // the notes are clear
        stage(lds, 0);
        next = __ballot(e >= 0);
        load(span.first + 1, e);                                // past the end no position has a page: nothing is read
        e = entry(span.first + 2);
    }
    int slot = 0;
    for (int32_t n = span.first; n < span.end; ++n) {
        uint8_t *const buffer = lds + ((n - span.first) & 1) * S::kBuffer, *const other = lds + ((n - span.first + 1) & 1) * S::kBuffer;
        const int slot1 = slot == 2 ? 0 : slot + 1, slot2 = slot1 == 2 ? 0 : slot1 + 1;
        lds_barrier();
        // nobody reads the notes of the tile before any more
        if (threadIdx.x < 64) {
            s_nan[slot2][threadIdx.x] = 0u;
            s_flag[slot2] = 0u;
        }
        const int32_t t0 = first_position + n * 64;
        const bool busy = has_rows && t0 < some_to && t0 + 64 > some_from;
        uint64_t now = 0ull;
        int noted = 0;
#pragma unroll
        for (int group = 0; group < GROUPS; ++group) {
            // --- S^T
            float logit[TT][NV];
            if (busy) {
                if constexpr (kFirst)
                    __builtin_amdgcn_s_setprio(1);
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    typename M::Sum c;
#pragma unroll
                    for (int x = 0; x < NV; ++x)
                        c[x] = 0.0f;
                    const int kr = RW * (group * TT + t) + i;
                    const uint8_t *row = buffer + kr * S::kRow;
                    int sw = S::swizzle_k(kr);
                    if constexpr (D == 192 && RW == 32)
                        asm volatile("" : "+v"(sw));                // places computed anew, not kept in 12 registers
#pragma unroll
                    for (int k = 0; k < NK; ++k) {
                        const half8_t k8 = *(const half8_t *)(row + ((M::kStep / 8 * k + h) ^ sw) * 16);
#pragma unroll
                        for (int part = 0; part < PARTS; ++part)
                            c = M::of(k8, q.part[part][k], c);
                    }
#pragma unroll
                    for (int x = 0; x < NV; ++x)
                        logit[t][x] = c[x];
                }
            }
            if constexpr (kFirst)
                __builtin_amdgcn_s_setprio(0);
            if (group == 0) {
                now = there;
                there = next;
                if (n + 1 < span.end) {
                    stage(other, slot1);
                    const int32_t page = page_of(e);
                    next = __ballot(page >= 0);
                    load(n + 2, page);
                    e = entry(n + 3);
                }
                noted = slot;
                slot = slot1;
            }
            if (!busy)
                break;
            if (now != ~0ull || t0 < all_from || t0 + 64 > all_to) {
                // what this lane's row sees of the tile, bit RW t + 8 (r / 4) + r % 4 for register r
                int32_t from = begin - t0, to = end - t0;
                asm volatile("" : "+v"(from), "+v"(to));            // a branch, not 32 selects in every tile
                uint64_t seen = from <= 0 ? now : from < 64 ? now & ~0ull << from : 0ull;
                seen = to >= 64 ? seen : to > 0 ? seen & ~(~0ull << to) : 0ull;
                seen >>= 4 * h;
#pragma unroll
                for (int t = 0; t < TT; ++t)
#pragma unroll
                    for (int x = 0; x < NV; ++x) {
                        const int at = RW * (group * TT + t) + 8 * (x / 4) + x % 4;
                        logit[t][x] = (uint32_t)(seen >> (at / 32 * 32)) >> (at % 32) & 1u ? logit[t][x] : -__builtin_inff();
                    }
            }
            if (group == 0 && s_flag[noted]) {
                for (int t = 0; t < 64; ++t) {
                    const uint32_t blocks = s_nan[noted][t];
                    if (t0 + t >= begin && t0 + t < end)
                        nan_blocks |= blocks;
                }
            }
            // --- softmax
            float most = logit[0][0];
#pragma unroll
            for (int x = 1; x < NV * TT; ++x)
                most = fmaxf(most, logit[x / NV][x % NV]);
            most = fmaxf(top, M::max_of(most) * rf);
            if (__ballot(most > top + kSlack)) {
                const float keep = weight_of(top, most);
                sum *= keep;
#pragma unroll
                for (int k = 0; k < ND; ++k)
                    acc[k] *= keep;
                top = most;
            }
            const float less = kShift - (top == -__builtin_inff() ? 0.0f : top);
            constexpr int NP = NV * TT / 8;                             // k-ranges of 8 positions a lane
            half8_t prob[PARTS][NP];
#pragma unroll
            for (int x = 0; x < NV * TT; ++x) {
                const float w = __builtin_amdgcn_exp2f(fmaf(logit[x / NV][x % NV], rf, less));
                sum += w;
                const _Float16 high = (_Float16)w;
                prob[0][x / 8][x % 8] = high;
                if constexpr (PARTS == 2)
                    prob[PARTS - 1][x / 8][x % 8] = (_Float16)(w - (float)high);
            }
            // --- O^T: lanes of 16 give the places of 4 rows, 4 values each
            if constexpr (kSecond)
                __builtin_amdgcn_s_setprio(1);
            const int vi = lane % 16, vd = RW == 32 ? lane / 16 % 2 : 0;
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                const int r0 = M::kStep * (NP * group + k) + 4 * h + vi / 4, r1 = r0 + M::kStep / 2;
                const uint8_t *a0 = buffer + S::kBytes + r0 * S::kRow + vi % 2 * 8, *a1 = buffer + S::kBytes + r1 * S::kRow + vi % 2 * 8;
                int sw0 = S::swizzle_v(r0), sw1 = S::swizzle_v(r1);
                if constexpr (D == 192 && RW == 32)
                    asm volatile("" : "+v"(sw0), "+v"(sw1));
#pragma unroll
                for (int d = 0; d < ND; ++d) {
                    const int piece = RW / 8 * d + 2 * vd + vi % 4 / 2;
                    const uint2_t x0 = read_transposed16(a0 + (piece ^ sw0) * 16), x1 = read_transposed16(a1 + (piece ^ sw1) * 16);
                    const uint4_t x = {x0.x, x0.y, x1.x, x1.y};
                    const half8_t v8 = __builtin_bit_cast(half8_t, x);
#pragma unroll
                    for (int part = 0; part < PARTS; ++part)
                        acc[d] = M::of(v8, prob[part][k], acc[d]);
                }
            }
            if constexpr (kSecond)
                __builtin_amdgcn_s_setprio(0);
        }
    }

    // --- results
    sum = M::sum_of(sum);
    const float gv = p.gv ? *p.gv : 1.0f;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int x = 0; x < NV; ++x)
            if (nan_blocks >> ((RW * d + 8 * (x / 4)) / 16) & 1u)
                acc[d][x] = __builtin_nanf("");
    if (span.splits == 1) {
        if (!real)
            return;
        const int64_t row = out_row(p, s, hk, row0 + r);
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int x = 0; x < NV; x += 4)
                store_values<4>(p, row * D + RW * d + 2 * x + 4 * h, {acc[d][x], acc[d][x + 1], acc[d][x + 2], acc[d][x + 3]}, sum, gv);
        if (h == 0)
            store_lse(p, row, {top, sum});
        return;
    }
    const uint32_t tile = id;
    if (real) {
        float *const sums = p.sums + (((int64_t)tile * p.splits + split) * kTileRows + r) * D;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int x = 0; x < NV; x += 4) {
                const float4_t v = {acc[d][x], acc[d][x + 1], acc[d][x + 2], acc[d][x + 3]};
                *(float4_t *)(sums + RW * d + 2 * x + 4 * h) = v;
            }
        if (h == 0)
            *(Norm *)(p.norms + (((int64_t)tile * p.splits + split) * kTileRows + r) * 2) = {top, sum};
    }
}

// The rows of split tiles, kJoinRows a workgroup, over the whole card: all of the tile
// kernel's, and of the rows kernel's where a tile has many rows. (Joined by the last workgroup of each
// tile instead: 80 us more for 515 queries at 20011 positions, where few tiles have
// many splits and one workgroup moved 2.8 MB.) FEW: the rows kernel's tiles.
constexpr int kJoinThreads = 256, kJoinRows = 8;

template <int D, bool FEW>
__global__ __launch_bounds__(kJoinThreads) void nvfp4_attention_join_kernel(AttParams p, int32_t tile_rows)
{
    __shared__ float s_weights[(kMaxSplits + 1) * kJoinRows];
    const uint32_t parts = (uint32_t)((p.most_rows + kJoinRows - 1) / kJoinRows), id = blockIdx.x / parts;
    const int first = (int)(blockIdx.x % parts) * kJoinRows;
    const uint32_t pairs = (uint32_t)p.B * (uint32_t)p.heads;
    const int rt = FEW ? (int)(id / pairs) : (int)(((uint32_t)p.row_tiles - 1u) - id / pairs);
    const int b = (int)(id % pairs / (uint32_t)p.heads), hk = (int)(id % pairs % (uint32_t)p.heads);
    const Sequence s = sequence_of(p, b);
    const int64_t all_rows = (int64_t)min(s.n, p.max_q) * p.G;
    if ((all_rows <= p.few_rows) != FEW || (int64_t)rt * tile_rows + first >= all_rows)
        return;
    const int row0 = rt * tile_rows, rows = (int)min((int64_t)tile_rows, all_rows - row0);
    const Span span = span_of(p, s, row0 / p.G, (row0 + rows - 1) / p.G + 1, 0);
    if (span.splits > 1 && first < rows)
        join_splits<D, kJoinThreads, 4, 1, 16, true>(p, s, hk, id, row0, first, min(kJoinRows, rows - first), span.splits,
                                                     p.gv ? *p.gv : 1.0f, s_weights);
}

// ------------------------------------------------------------------ host

constexpr int64_t kTicketBytes = 65536, kMaxPartialBytes = INT64_C(64) << 20;
constexpr int64_t kMaxTickets = kTicketBytes / 4;
static_assert(kTicketBytes + kMaxPartialBytes == NVFP4_WORKSPACE_MAX_BYTES);

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

nvfp4_status_t check(const nvfp4_cache_t *cache, int dtype, int64_t T, int64_t H, int64_t B, const nvfp4_attention_t *a)
{
    if (!a)
        return NVFP4_ERR_NULL_POINTER;
    if (dtype != NVFP4_F16 && dtype != NVFP4_BF16 && dtype != NVFP4_F32)
        return NVFP4_ERR_INVALID_TYPE;
    const nvfp4_status_t st = nvfp4_check_cache(cache);
    if (st != NVFP4_OK)
        return st;
    const int64_t D = cache->head_size;
    if (D != 64 && D != 96 && D != 128 && D != 192 && D != 256)
        return NVFP4_ERR_INVALID_CACHE;
    const int64_t most = INT64_C(1) << 30;
    if (T < 1 || B < 1 || H < 1 || T > most || B > most || H % cache->heads || H / cache->heads > 1024 || a->max_q < 1 ||
        a->max_q > T || a->max_q > most / B || a->max_q > most / (H / cache->heads) || a->max_length < 1 || a->max_length > most)
        return NVFP4_ERR_INVALID_SHAPE;
    if (a->window < 0 || a->window > INT32_MAX || (a->causal != 0 && a->causal != 1))
        return NVFP4_ERR_INVALID_CACHE;
    if (!std::isfinite(a->scale))
        return NVFP4_ERR_INVALID_SCALE;
    if (a->q_token_stride < 0 || a->q_head_stride < 0 || a->q_token_stride >= kMaxStride || a->q_head_stride >= kMaxStride)
        return NVFP4_ERR_INVALID_STRIDE;
    return NVFP4_OK;
}

// How the positions are shared out: `tiles` workgroups if none were split.
struct Plan {
    int64_t tiles;
    int32_t splits, chunk, most_rows, row_tiles, waves;
    size_t bytes;                               // of workspace
};

int64_t partial_bytes(int64_t tiles, int64_t splits, int64_t rows, int64_t D)
{
    return tiles * splits * rows * (D + 2) * 4;
}

// Rows of a workgroup of the rows kernel, and how many such a sequence's have at most.
int rows_at_once(int64_t most) { return most <= 16 ? 16 : 32; }

Plan rows_plan(const nvfp4_cache_t &c, int64_t H, int64_t B, const nvfp4_attention_t &a)
{
    Plan p{};
    const int64_t most_rows = std::min<int64_t>(kFewRows, a.max_q * (H / c.heads));
    const int rows = rows_at_once(most_rows);
    p.row_tiles = (int32_t)((most_rows + rows - 1) / rows);
    p.tiles = B * c.heads * p.row_tiles;
    p.most_rows = (int32_t)std::min<int64_t>(rows, most_rows);
    // most tiles of 64 positions that a sequence's rows see
    const int64_t span = a.window ? std::min<int64_t>(a.max_length, a.window + std::min<int64_t>(a.max_q, rows) + 64) : a.max_length;
    const int64_t most = (span + 63) / 64 + (a.window ? 1 : 0);       // a window starts inside a tile
    // Waves of a workgroup: 8, so that half the partial results have to be joined, where 4 with a tile each
    // would be more than 16 splits and 8 fill the CUs once at most (one sequence, 8 key heads: 16384
    // positions 17.5 us, with 4 waves 21.5; 4096 positions 13.0 and 12.5)
    p.waves = rows == 16 && most > 64 && p.tiles * ((most + 7) / 8) <= kCus ? 8 : 4;
    // workgroups: 1024 keep the card loading (64 sequences of 1024 to 8192 positions, 4 rows: 93 us, 114 with
    // 512, 99 with 2048); more rows mean larger partial results (16 sequences of up to 4000, 32 rows: 34 us
    // with 512, 42 with 1024)
    const int64_t target = most_rows <= 4 ? 1024 : 512;
    int64_t splits = std::min<int64_t>((target + p.tiles - 1) / p.tiles, (most + p.waves - 1) / p.waves);
    splits = std::max<int64_t>(1, std::min<int64_t>(splits, kMaxSplits));
    if (p.tiles > kMaxTickets)
        splits = 1;
    while (splits > 1 && partial_bytes(p.tiles, splits, p.most_rows, c.head_size) > kMaxPartialBytes)
        --splits;
    p.chunk = (int32_t)((most + splits - 1) / splits + p.waves - 1) / p.waves * p.waves;
    p.splits = (int32_t)((most + p.chunk - 1) / p.chunk);
    p.bytes = p.splits > 1 ? kTicketBytes + (partial_bytes(p.tiles, p.splits, p.most_rows, c.head_size) + 255) / 256 * 256 : 0;
    return p;
}

// 2^30 rows of a sequence at most (max_q * G), so row_tiles and rows fit 32 bits.
Plan tile_plan(const nvfp4_cache_t &c, int dtype, int64_t H, int64_t B, const nvfp4_attention_t &a)
{
    Plan p{};
    const int rows = tile_rows((int)c.head_size, dtype == NVFP4_F32);
    const int64_t G = H / c.heads, row_tiles = (a.max_q * G + rows - 1) / rows;
    p.row_tiles = (int32_t)row_tiles;
    p.tiles = B * c.heads * row_tiles;
    p.most_rows = rows;
    const int64_t span = a.window ? std::min<int64_t>(a.max_length, a.window + rows + 64) : a.max_length;
    const int64_t most = (span + 63) / 64 + (a.window ? 1 : 0);       // a window starts inside a tile
    // As many as fill the places for workgroups once (two on a CU up to 128 values, one beyond), or
    // twice where that leaves fewer of them idle
    const int64_t places = c.head_size <= 128 ? 512 : 256, once = places / p.tiles, twice = 2 * places / p.tiles;
    int64_t splits = twice * p.tiles * 10 > once * p.tiles * 22 ? twice : once;
    splits = std::max<int64_t>(1, std::min<int64_t>({splits, kMaxSplits, (most + kTileLeast - 1) / kTileLeast}));
    while (splits > 1 && partial_bytes(p.tiles, splits, rows, c.head_size) > kMaxPartialBytes)
        --splits;
    p.chunk = (int32_t)((most + splits - 1) / splits);
    p.splits = (int32_t)((most + p.chunk - 1) / p.chunk);
    p.bytes = p.splits > 1 ? kTicketBytes + (partial_bytes(p.tiles, p.splits, rows, c.head_size) + 255) / 256 * 256 : 0;
    return p;
}

// Sequences of more rows than the rows kernel takes.
bool has_many(const nvfp4_cache_t &c, int64_t H, const nvfp4_attention_t &a) { return a.max_q * (H / c.heads) > kFewRows; }

// A lone sequence that may have many rows is the tile kernel's whatever it has: beside it the rows kernel
// would find nothing to do (515 queries of 4 shared heads of 192, bfloat16, at 2500 positions: 47 us, 51 with it)
bool has_few(const nvfp4_cache_t &c, int64_t H, int64_t B, const nvfp4_attention_t &a) { return B > 1 || !has_many(c, H, a); }

size_t need_of(const nvfp4_cache_t &c, int dtype, int64_t H, int64_t B, const nvfp4_attention_t &a)
{
    return std::max(has_few(c, H, B, a) ? rows_plan(c, H, B, a).bytes : 0, has_many(c, H, a) ? tile_plan(c, dtype, H, B, a).bytes : 0);
}

void set_plan(AttParams &p, const Plan &plan, void *workspace)
{
    p.splits = plan.splits, p.chunk = plan.chunk, p.most_rows = plan.most_rows, p.row_tiles = plan.row_tiles;
    p.tickets = (uint32_t *)workspace;
    p.sums = workspace ? (float *)((uint8_t *)workspace + kTicketBytes) : nullptr;
    p.norms = p.sums ? p.sums + plan.tiles * plan.splits * plan.most_rows * p.D : nullptr;
}

template <int D, bool FEW>
hipError_t launch_join(const AttParams &p, int64_t tiles, int rows, hipStream_t st)
{
    const int64_t parts = (p.most_rows + kJoinRows - 1) / kJoinRows;
    hipLaunchKernelGGL((nvfp4_attention_join_kernel<D, FEW>), dim3((uint32_t)(tiles * parts)), dim3(kJoinThreads), 0, st, p, rows);
    return hipGetLastError();
}

template <int D, bool F32>
hipError_t launch_tile(const AttParams &p, int64_t grid, hipStream_t st)
{
    constexpr int threads = 64 * tile_waves(D, F32), rows = tile_rows(D, F32), buffers = 2 * WideTile<D, threads>::kBuffer;
    static_assert(buffers + 1024 <= 160 * 1024);
    hipLaunchKernelGGL((nvfp4_attention_tile_kernel<D, F32>), dim3((uint32_t)grid), dim3(threads), buffers, st, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1)
        return e;
    return launch_join<D, false>(p, grid / p.splits, rows, st);
}

template <int D, int NQ, bool F32, int WAVES>
hipError_t launch_rows(const AttParams &p, int64_t grid, hipStream_t st)
{
    using S = RowsTile<D>;
    const int lds = std::max({WAVES * S::kWave, WAVES * 16 * NQ * (D * 4 + 8), (p.splits + 1) * 4 * p.most_rows});
    static_assert(WAVES * S::kWave + 64 <= 160 * 1024 && WAVES * 16 * NQ * (D * 4 + 8) + 64 <= 160 * 1024 && (kMaxSplits + 1) * 4 * 64 < 64 * 1024);
    hipLaunchKernelGGL((nvfp4_attention_rows_kernel<D, NQ, F32, WAVES>), dim3((uint32_t)grid), dim3(64 * WAVES), lds, st, p);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess || p.splits == 1 || p.join_here ? e : launch_join<D, true>(p, grid / p.splits, 16 * NQ, st);
}

template <int D, bool F32>
hipError_t launch_rows_of(const AttParams &p, int waves, int64_t grid, hipStream_t st)
{
    if (waves == 8)
        return launch_rows<D, 1, F32, 8>(p, grid, st);
    return rows_at_once(p.most_rows) == 16 ? launch_rows<D, 1, F32, 4>(p, grid, st) : launch_rows<D, 2, F32, 4>(p, grid, st);
}

template <typename F>
hipError_t by_head(int D, F f)
{
    switch (D) {
    case 64: return f(std::integral_constant<int, 64>{});
    case 96: return f(std::integral_constant<int, 96>{});
    case 128: return f(std::integral_constant<int, 128>{});
    case 192: return f(std::integral_constant<int, 192>{});
    default: return f(std::integral_constant<int, 256>{});
    }
}

} // namespace

extern "C" {

size_t nvfp4_cache_attention_workspace_bytes(const nvfp4_cache_t *cache, int dtype, int64_t T, int64_t H, int64_t B,
                                             const nvfp4_attention_t *attention)
{
    if (check(cache, dtype, T, H, B, attention) != NVFP4_OK)
        return 0;
    return need_of(*cache, dtype, H, B, *attention);
}

nvfp4_status_t nvfp4_cache_attention(const nvfp4_cache_t *cache, const void *q, int dtype, void *out, float *lse,
                                     const int32_t *offsets, const int32_t *lengths, const int32_t *table, int64_t T,
                                     int64_t H, int64_t B, int64_t table_width, const nvfp4_attention_t *attention,
                                     void *workspace, size_t workspace_bytes, void *stream)
{
    if (!q || !out || !offsets || !lengths || !table)
        return NVFP4_ERR_NULL_POINTER;
    const nvfp4_status_t st = check(cache, dtype, T, H, B, attention);
    if (st != NVFP4_OK)
        return st;
    if (table_width < 1 || table_width > (INT64_C(1) << 30) / cache->page_size ||
        attention->max_length > table_width * cache->page_size)
        return NVFP4_ERR_INVALID_SHAPE;
    const uintptr_t size = dtype == NVFP4_F32 ? 4 : 2;
    if (!aligned(q, size) || !aligned(out, size) || (lse && !aligned(lse, 4)) || !aligned(offsets, 4) ||
        !aligned(lengths, 4) || !aligned(table, 4))
        return NVFP4_ERR_MISALIGNED;
    AttParams p{};
    p.q = (const uint8_t *)q, p.out = (uint8_t *)out, p.lse = lse;
    p.kc = (const uint8_t *)cache->k_codes, p.ks = (const uint8_t *)cache->k_scales;
    p.vc = (const uint8_t *)cache->v_codes, p.vs = (const uint8_t *)cache->v_scales;
    p.gk = cache->k_scale, p.gv = cache->v_scale;
    p.offsets = offsets, p.lengths = lengths, p.table = table;
    p.q_token = attention->q_token_stride * (int64_t)size, p.q_head = attention->q_head_stride * (int64_t)size;
    p.code_page = (uint32_t)cache->code_page_stride, p.scale_page = (uint32_t)cache->scale_page_stride;
    p.T = (int32_t)T, p.H = (int32_t)H, p.B = (int32_t)B, p.width = (int32_t)table_width, p.pages = (int32_t)cache->pages;
    p.shift = __builtin_ctzll((uint64_t)cache->page_size);
    p.heads = (int32_t)cache->heads, p.G = (int32_t)(H / cache->heads), p.D = (int32_t)cache->head_size;
    p.max_q = (int32_t)attention->max_q, p.max_length = (int32_t)attention->max_length;
    // a window as long as the longest sequence hides nothing
    p.window = attention->window >= attention->max_length ? 0 : (int32_t)attention->window, p.causal = attention->causal, p.dtype = dtype, p.scale = attention->scale;
    const Plan few = rows_plan(*cache, H, B, *attention), many = tile_plan(*cache, dtype, H, B, *attention);
    const bool has[2] = {has_few(*cache, H, B, *attention), has_many(*cache, H, *attention)};
    if ((has[0] && few.tiles > kMaxGrid / few.splits) || (has[1] && many.tiles > kMaxGrid / many.splits))
        return NVFP4_ERR_INVALID_SHAPE;
    const size_t need = need_of(*cache, dtype, H, B, *attention);
    if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
        return NVFP4_ERR_WORKSPACE;
    p.few_rows = has[0] ? kFewRows : 0;
    p.join_here = few.most_rows <= kJoinHere;
    const hipStream_t hs = (hipStream_t)stream;
    // one after the other on the stream, so one workspace serves both
    hipError_t e = hipSuccess;
    if (has[0]) {
        set_plan(p, few, need ? workspace : nullptr);
        e = by_head(p.D, [&](auto d) {
            const int64_t grid = few.tiles * few.splits;
            return dtype == NVFP4_F32 ? launch_rows_of<d(), true>(p, few.waves, grid, hs) : launch_rows_of<d(), false>(p, few.waves, grid, hs);
        });
    }
    if (e == hipSuccess && has[1]) {
        set_plan(p, many, need ? workspace : nullptr);
        e = by_head(p.D, [&](auto d) {
            const int64_t grid = many.tiles * many.splits;
            return dtype == NVFP4_F32 ? launch_tile<d(), true>(p, grid, hs) : launch_tile<d(), false>(p, grid, hs);
        });
    }
    if (e == hipSuccess)
        return NVFP4_OK;
    nvfp4_record_hip_error((int)e);
    return NVFP4_ERR_HIP;
}

} // extern "C"
