// NVFP4 products with any number of rows on MI355X (gfx950): dense (nvfp4_gemm)
// and routed to experts (nvfp4_gemm_experts).
//
//   c[n][m] = scale * sum_k a'[m][k] b'[n][k],   a' = e2m1(A) e4m3(SFA), b' = e2m1(B) e4m3(SFB)
//
// Mathematics. a' and b' have at most 6 significant bits, |a'| <= 2688 and the
// smallest nonzero one is 2^-10: float16 holds them exactly, no 8-bit type
// does. So the product is a float16 matrix product with float32 accumulation.
// The FP4 matrix instruction cannot apply an E4M3 scale per 16: its block
// scales are powers of two per 32.
//
// Common to both kernels. Packed codes and scale words (4 scales: 64 k of one
// row) go straight from global memory into a ring of LDS stages, by copies that
// need no register; a stage is 128 k. Waves read the packed codes and decode
// their own fragments (one conversion and one packed multiply per two values),
// so LDS holds and moves 4 bits per value, not 16.
//   MFMA 32x32x16: lane i holds row i % 32; lanes 0..31 take a stage's first 64
// k, lanes 32..63 the other 64 (the order of k inside a stage is free as long
// as A and B agree). Rows of B are the instruction's rows, rows of A its
// columns, so a lane's results are neighbours in m of its neighbours'.
//   LDS rows are 64 bytes (128 codes). 16-byte piece c of row r lies at piece
// c ^ ((r / 4) % 4): any 16 consecutive rows' pieces c fall on all banks.
//   Scale words lie as in the 128x4 blocked layout, word (r, half) at half * tile
// + (r % 32) * 16 + (r / 32) * 4, so one read gives a lane the words of its row
// in up to four 32-row fragments. Blocked or plain, rows in order or gathered:
// the address of each word is computed once and steps by a constant. Plain
// rows of K % 64 = 32 are 2-byte aligned: their words are copied in halves.
//
// Wide kernel (many rows of B): 4 or 8 waves share a tile's stages, one barrier
// per stage. Bound by the matrix cores at the clock that the power limit leaves:
// 7168 x 4096 x 16384 takes 757 us (1.27 PFLOP/s; a float16 library product of
// the same size 794).
//   Wave kernel (few rows of B: bound by the weights' bytes, or small tiles by
// decoding): each wave has a ring of its own and takes every KW-th stage, no
// barrier in the loop; the waves' sums are added in LDS in the order of the waves.
// Its K can also be split over workgroups: float32 partial sums in the workspace,
// the last workgroup of a tile (by ticket) adds them in the order of the slices.
// 64 tokens x 4 of 64 experts, 4096 x 2048: 59 us (5.0 TB/s); 7168 x 16 x 2048: 6.0.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "nvfp4_device.h"
#include "nvfp4_gemv.h"
#include "nvfp4_internal.h"

namespace {

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float float16_t __attribute__((ext_vector_type(16)));

constexpr int kLdsBytes = 160 * 1024;           // LDS of a CU
constexpr int kStaticLds = 2048;                // slot table and ticket, at most
constexpr int kStageK = 128;                    // k per stage
constexpr int kMaxExperts = 1024;
constexpr int kMaxTickets = 16384;              // tiles of a split product
constexpr int64_t kTicketBytes = kMaxTickets * 4;
constexpr int64_t kMaxPartialBytes = INT64_C(64) << 20;
static_assert(kTicketBytes + kMaxPartialBytes == NVFP4_WORKSPACE_MAX_BYTES && NVFP4_WORKSPACE_MAX_BYTES % 256 == 0);
constexpr int kMaxSplits = 16;
constexpr int64_t kMaxGrid = 0x7FFFFF;          // workgroups of up to 512 threads in 2^32 work items

// ------------------------------------------------------------------ copies to LDS

// A pointer that is the same in every lane, in scalar registers (nothing to do
// where the compiler has it there).
__device__ __attribute__((always_inline)) inline const uint8_t *uniform_ptr(const uint8_t *p)
{
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)p);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uintptr_t)p >> 32));
    return (const uint8_t *)(uintptr_t)((uint64_t)hi << 32 | lo);
}

// 16, 4 or 2 bytes per lane from base + off into LDS at dst + lane * 16 (lane *
// 4; 2 bytes land in the low half of a dword). The base is uniform and steps
// along K in scalar registers, the lane's offset stays. The compiler does not
// count the copies: the kernels wait for them themselves.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __attribute__((always_inline)) inline void copy16(const uint8_t *base, uint32_t off, uint32_t dst)
{
    asm volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_dwordx4 %0, %1" : : "v"(off), "s"(uniform_ptr(base)), "s"(dst) : "memory", "m0");
}
__device__ __attribute__((always_inline)) inline void copy4(const uint8_t *base, uint32_t off, uint32_t dst)
{
    asm volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_dword %0, %1" : : "v"(off), "s"(uniform_ptr(base)), "s"(dst) : "memory", "m0");
}
__device__ __attribute__((always_inline)) inline void copy2(const uint8_t *base, uint32_t off, uint32_t dst)
{
    asm volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_ushort %0, %1" : : "v"(off), "s"(uniform_ptr(base)), "s"(dst) : "memory", "m0");
}
#pragma clang diagnostic pop

// s_waitcnt vmcnt(N), other counters unconstrained
template <int N>
__device__ __attribute__((always_inline)) inline void wait_copies()
{
    static_assert(N >= 0 && N < 64, "vmcnt holds 0..63");
    __builtin_amdgcn_s_waitcnt((0x0F70 & ~0xC00F) | (N & 15) | ((N >> 4) << 14));
}

// Past it, what any wave has read from LDS before may be overwritten: each waits
// for its own reads to return. The compiler waits where it uses a read, which may
// be after a barrier that it does not know to free the place that was read.
__device__ __attribute__((always_inline)) inline void barrier()
{
    asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" : : : "memory");
}

// ------------------------------------------------------------------ parameters

struct GemmParams {
    const uint8_t *a, *b, *sfa, *sfb;
    uint8_t *c;
    const float *scale_a, *scale_b;
    const int32_t *offsets, *order;             // experts
    uint32_t *tickets;
    float *partials;                            // [splits][slots][M] (dense: slots = L * N)
    int64_t sfa_batch, sfb_batch;               // bytes
    int32_t M, N, K, L;                         // experts: N = slots, L = experts
    int32_t slots_per_row;
    int32_t tiles_m, tiles_n;                   // dense: per batch
    int32_t splits, stages_per_split, stages;
    int32_t blocked, dtype;
    float alpha;
};

// (row, first of 4 scales) of a rows x nkb scale matrix; the step of 2 words is constant in k
__device__ __attribute__((always_inline)) inline int64_t scale_word_at(bool blocked, int32_t r, int32_t half,
                                                                       int32_t nkb)
{
    if (blocked)
        return ((int64_t)(r / 128) * ((nkb + 3) / 4) + half) * 512 + (r % 32) * 16 + ((r % 128) / 32) * 4;
    return (int64_t)r * nkb + half * 4;
}

// dtype is uniform: one branch per value, the same for all (a template on it
// would build every kernel three times)
__device__ __attribute__((always_inline)) inline void store_value(uint8_t *c, int64_t i, float v, int dtype)
{
    if (dtype == NVFP4_F32)
        ((float *)c)[i] = v;
    else
        ((uint16_t *)c)[i] = dtype == NVFP4_BF16 ? (uint16_t)bf16_bits(v) : f16_bits(v);
}

// 8 codes (a dword) times a scale -> 8 float16
__device__ __attribute__((always_inline)) inline half8_t decode8(uint32_t w, half2_t s)
{
    const half2_t v0 = fp4x2<0>(w) * s, v1 = fp4x2<1>(w) * s, v2 = fp4x2<2>(w) * s, v3 = fp4x2<3>(w) * s;
    return (half8_t){v0.x, v0.y, v1.x, v1.y, v2.x, v2.y, v3.x, v3.y};
}

// NW consecutive scale words (1, 2 or 4) from LDS
template <int NW>
__device__ __attribute__((always_inline)) inline void read_words(const uint8_t *p, uint32_t (&w)[NW])
{
    if constexpr (NW == 4) {
        const uint4_t v = *(const uint4_t *)p;
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (NW == 2) {
        const uint2_t v = *(const uint2_t *)p;
        w[0] = v.x, w[1] = v.y;
    } else {
        w[0] = *(const uint32_t *)p;
    }
}

// words of FM fragments from LDS: whole, or in halves `hi` bytes apart
template <int FM, bool ODD>
__device__ __attribute__((always_inline)) inline void load_words(const uint8_t *p, uint32_t hi, uint32_t (&w)[FM])
{
    read_words<FM>(p, w);
    if constexpr (ODD) {
        uint32_t h[FM];
        read_words<FM>(p + hi, h);
#pragma unroll
        for (int i = 0; i < FM; ++i)
            w[i] = (w[i] & 0xFFFFu) | (h[i] << 16);
    }
}

// The word's scales that lie before K's end; `left`: k from the word's first to the end.
__device__ __attribute__((always_inline)) inline uint32_t word_mask(int left)
{
    return left >= 64 ? ~0u : left == 32 ? 0xFFFFu : 0u;
}

// Copies one 64-lane group of scale words. A word past K's end is replaced by
// the stage's first of the same row (`back` bytes before), its upper half by its
// lower: nothing past a row is read, and the reader masks what it gets.
template <bool ODD>
__device__ __attribute__((always_inline)) inline void copy_words(const uint8_t *base, uint32_t off, int left,
                                                                 uint32_t back, uint32_t dst, uint32_t hi)
{
    off -= left <= 0 ? back : 0u;
    if constexpr (ODD) {
        copy2(base, off, dst);
        copy2(base, off + (left == 32 || left == -32 ? 0u : 2u), dst + hi);
    } else {
        copy4(base, off, dst);
    }
}

// A row range's part of an operand: codes and scale words from its first row on.
struct Source {
    const uint8_t *codes, *words;
};

// ------------------------------------------------------------------ which tile

struct Where {
    int l, m0, n0, count;                       // batch or expert (-1: none), first rows, rows of B
    uint32_t tile;
    int split;
};

// The experts e0 .. e0 + 63, one per lane: start and length of the list, and the
// lists' tiles summed up to and including the lane's.
struct Lists {
    int from, n, tiles, upto;
};

template <int BN>
__device__ __attribute__((always_inline)) inline Lists lists_at(const GemmParams &p, int e0)
{
    const int lane = threadIdx.x % 64, e = e0 + lane;
    Lists s{};
    if (e < p.L) {
        s.from = min(max(p.offsets[e], 0), p.N);
        s.n = max(min(max(p.offsets[e + 1], 0), p.N) - s.from, 0);
    }
    s.tiles = s.upto = (s.n + BN - 1) / BN;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(s.upto, d);
        s.upto += lane >= d ? v : 0;
    }
    return s;
}

template <bool EXPERTS, int BM, int BN, int THREADS>
__device__ __attribute__((always_inline)) inline Where locate(const GemmParams &p, int32_t *s_slot)
{
    Where w;
    if constexpr (EXPERTS) {
        // The grid holds as many workgroups as any lists may need; the first
        // `total` of them work, so that all XCDs get their share of these.
        const Lists head = lists_at<BN>(p, 0);
        int64_t total = __shfl(head.upto, 63);
        for (int e0 = 64; e0 < p.L; e0 += 64)
            total += __shfl(lists_at<BN>(p, e0).upto, 63);
        const uint32_t wgs = __builtin_amdgcn_readfirstlane((uint32_t)min(total * p.tiles_m * p.splits, (int64_t)gridDim.x));
        w.l = -1;
        if (blockIdx.x >= wgs)
            return w;                           // the whole workgroup
        uint32_t id = xcd_remap(blockIdx.x, wgs);
        w.split = (int)(id % (uint32_t)p.splits);
        id /= (uint32_t)p.splits;
        w.tile = id;
        // Tiles in the order of experts, then rows of A, then the list's tiles, so
        // that neighbours share the expert's weights.
        int64_t want = id;
        int found = -1, row = 0;
        w.n0 = w.count = 0;
        for (int e0 = 0; e0 < p.L; e0 += 64) {
            const Lists s = e0 == 0 ? head : lists_at<BN>(p, e0);
            const uint64_t past = __ballot((int64_t)s.upto * p.tiles_m > want);
            if (past) {
                const int src = __ffsll((unsigned long long)past) - 1;
                const int own = __shfl(s.tiles, src);
                const uint32_t in_list = (uint32_t)(want - (int64_t)(__shfl(s.upto, src) - own) * p.tiles_m);
                found = e0 + src;
                row = (int)(in_list / (uint32_t)own);
                const int at = (int)(in_list % (uint32_t)own) * BN;
                w.n0 = __shfl(s.from, src) + at;
                w.count = min(BN, __shfl(s.n, src) - at);
                break;
            }
            want -= (int64_t)__shfl(s.upto, 63) * p.tiles_m;
        }
        w.m0 = __builtin_amdgcn_readfirstlane(row) * BM;
        w.l = __builtin_amdgcn_readfirstlane(found);
        w.n0 = __builtin_amdgcn_readfirstlane(w.n0);
        w.count = __builtin_amdgcn_readfirstlane(w.count);
        if (w.l < 0)
            return w;
        for (int i = threadIdx.x; i < BN; i += THREADS) {
            const int s = i < w.count ? p.order[w.n0 + i] : -1;
            s_slot[i] = s >= 0 && s < p.N ? s : -1;
        }
        __syncthreads();
    } else {
        uint32_t id = xcd_remap(blockIdx.x, gridDim.x);
        w.split = (int)(id % (uint32_t)p.splits);
        id /= (uint32_t)p.splits;
        w.tile = id;
        // bands of 8 tiles along n, so that one XCD's tiles share rows of both
        const uint32_t per = (uint32_t)p.tiles_m * (uint32_t)p.tiles_n;
        w.l = (int)(id / per);
        id %= per;
        const uint32_t band = id / ((uint32_t)p.tiles_m * 8u);
        id -= band * (uint32_t)p.tiles_m * 8u;
        const uint32_t wide = min(8u, (uint32_t)p.tiles_n - band * 8u);
        w.m0 = (int)(id / wide) * BM;
        w.n0 = (int)(band * 8u + id % wide) * BN;
        w.count = min(BN, p.N - w.n0);
    }
    return w;
}

// Operand A from the tile's first 128-row block on (rows of codes from m0 on).
__device__ __attribute__((always_inline)) inline Source source_a(const GemmParams &p, const Where &w)
{
    const int64_t words = p.blocked ? (int64_t)(w.m0 / 128) * ((p.K / 16 + 3) / 4) * 512 : (int64_t)w.m0 * (p.K / 16);
    return {p.a + ((int64_t)w.l * p.M + w.m0) * (p.K / 2), p.sfa + w.l * p.sfa_batch + words};
}
// Offsets of the tile's row i (any i below BM; rows past M are row M - 1) in source_a.
__device__ __attribute__((always_inline)) inline uint32_t codes_at_a(const GemmParams &p, const Where &w, int i)
{
    return (uint32_t)min(i, p.M - 1 - w.m0) * (uint32_t)(p.K / 2);
}
__device__ __attribute__((always_inline)) inline uint32_t words_at_a(const GemmParams &p, const Where &w, int i, int half)
{
    const int r = min(i, p.M - 1 - w.m0) + (p.blocked ? w.m0 % 128 : 0);
    return (uint32_t)scale_word_at(p.blocked, r, half, p.K / 16);
}

// Operand B: dense from the tile's first row on; experts' rows are gathered
// from all of it (at most 2^32 bytes, the entry point checks).
template <bool EXPERTS>
__device__ __attribute__((always_inline)) inline Source source_b(const GemmParams &p, const Where &w)
{
    if constexpr (EXPERTS)
        return {p.b, p.sfb};
    const int64_t words = p.blocked ? (int64_t)(w.n0 / 128) * ((p.K / 16 + 3) / 4) * 512 : (int64_t)w.n0 * (p.K / 16);
    return {p.b + ((int64_t)w.l * p.N + w.n0) * (p.K / 2), p.sfb + w.l * p.sfb_batch + words};
}
template <bool EXPERTS>
__device__ __attribute__((always_inline)) inline uint32_t codes_at_b(const GemmParams &p, const Where &w,
                                                                     const int32_t *s_slot, int i)
{
    if constexpr (EXPERTS)
        return (uint32_t)(max(s_slot[i], 0) / p.slots_per_row) * (uint32_t)(p.K / 2);
    return (uint32_t)min(i, w.count - 1) * (uint32_t)(p.K / 2);
}
template <bool EXPERTS>
__device__ __attribute__((always_inline)) inline uint32_t words_at_b(const GemmParams &p, const Where &w,
                                                                     const int32_t *s_slot, int i, int half)
{
    if constexpr (EXPERTS)
        return (uint32_t)scale_word_at(p.blocked, max(s_slot[i], 0) / p.slots_per_row, half, p.K / 16);
    return (uint32_t)scale_word_at(p.blocked, min(i, w.count - 1) + (p.blocked ? w.n0 % 128 : 0), half, p.K / 16);
}

// alpha and the global scales, as a size of 1/8 to 1 and a power of two: their
// product may leave float32's range where the scaled sum does not (two scales of
// 2^-75, or 2^100 and 2^100 beside a sum of zero), and the sum, 2^-20 to 2^46 or
// zero, times the size does not leave it. Rounds as the product of the floats.
// Loaded before the product and kept: read at the end, they would add a memory
// round trip to every tile.
struct Scale {
    float size;
    int power;

    __device__ __attribute__((always_inline)) inline void times(float v)
    {
        size *= __builtin_amdgcn_frexp_mantf(v);
        power += __builtin_amdgcn_frexp_expf(v);
    }
    // the one rounding of the scaled sum (two where it is subnormal)
    __device__ __attribute__((always_inline)) inline float of(float sum) const { return __builtin_ldexpf(sum * size, power); }
};

template <bool EXPERTS>
__device__ __attribute__((always_inline)) inline Scale total_scale(const GemmParams &p, int l)
{
    Scale s{1.0f, 0};
    s.times(p.alpha);
    if (p.scale_a)
        s.times(p.scale_a[EXPERTS ? l : 0]);
    if (p.scale_b)
        s.times(*p.scale_b);
    return s;
}

// Offset in c (and in a slice of partial sums) of the tile's row n, -1: not stored.
template <bool EXPERTS>
__device__ __attribute__((always_inline)) inline int64_t row_at(const GemmParams &p, const Where &w,
                                                                const int32_t *s_slot, int n)
{
    if (n >= w.count)
        return -1;
    if constexpr (EXPERTS)
        return s_slot[n] < 0 ? -1 : (int64_t)s_slot[n] * p.M;
    else
        return ((int64_t)w.l * p.N + w.n0 + n) * p.M;
}

// Takes the tile's ticket after this workgroup's partial sums; true for the
// last of the tile's workgroups. All threads call it.
__device__ __attribute__((always_inline)) inline bool last_of_tile(const GemmParams &p, uint32_t tile,
                                                                   uint32_t *s_ticket)
{
    asm volatile("s_waitcnt vmcnt(0)" : : : "memory");          // this wave's partial sums are out
    barrier();
    if (threadIdx.x == 0)
        *s_ticket = __hip_atomic_fetch_add(&p.tickets[tile], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (*s_ticket != (uint32_t)p.splits - 1)
        return false;
    if (threadIdx.x == 0)
        __hip_atomic_store(&p.tickets[tile], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return true;
}

// Sums of R values over the slices, in order: 4 slices' loads in flight.
template <int R>
__device__ __attribute__((always_inline)) inline void add_slices(const GemmParams &p, int64_t one,
                                                                 const int64_t (&at)[R], float (&sum)[R])
{
#pragma unroll
    for (int r = 0; r < R; ++r)
        sum[r] = 0.0f;
    for (int s0 = 0; s0 < p.splits; s0 += 4) {
        float v[4][R];
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int r = 0; r < R; ++r)
                v[s][r] = s0 + s < p.splits && at[r] >= 0
                              ? __hip_atomic_load(&p.partials[(s0 + s) * one + at[r]], __ATOMIC_RELAXED,
                                                  __HIP_MEMORY_SCOPE_AGENT)
                              : 0.0f;
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int r = 0; r < R; ++r)
                sum[r] += v[s][r];
    }
}

// ------------------------------------------------------------------ wide kernel

// FM x FN fragments of 32 x 32 per wave, WM x WN waves, NS stages in the ring,
// registers for PER_CU workgroups per CU.
template <int FM, int FN, int WM, int WN, int NS, int PER_CU>
struct Tile {
    static_assert(NS >= 2);
    static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves, kPerSimd = PER_CU * kWaves / 4;
    static constexpr int kFM = FM, kFN = FN, kWM = WM, kWN = WN, kNS = NS, kPerCu = PER_CU;
    static constexpr int BM = 32 * FM * WM, BN = 32 * FN * WN;
    // words per line of a scale tile: 32-row groups that share a line
    static constexpr int LA = BM >= 128 ? 4 : BM / 32, LB = BN >= 128 ? 4 : BN / 32;
    static constexpr int kCodesA = BM * 64, kCodesB = BN * 64;
    static constexpr int kOffB = kCodesA, kOffSA = kCodesA + kCodesB;
    // wave copies per stage: codes in 1 KiB, scale words in 256 bytes
    static constexpr int TA = kCodesA / 1024, TB = kCodesB / 1024, TSA = BM * 8 / 256, TSB = BN * 8 / 256;
    static_assert(TA % kWaves == 0 && TB % kWaves == 0 && TSA % kWaves == 0);
    static_assert(TSB % kWaves == 0 || TSB < kWaves);
    static constexpr int stage_bytes(bool odd) { return kOffSA + (BM + BN) * (odd ? 16 : 8); }
    // one stage fewer where the halves of the words leave no room for NS
    static constexpr int ring(bool odd) { return NS * stage_bytes(odd) + kStaticLds <= kLdsBytes ? NS : NS - 1; }
    // results of one fragment row per wave pass through LDS: 32 rows of FM * 32 values
    static constexpr int kPitch = FM * 128 + 16, kOutLds = kWaves * 32 * kPitch;
    static constexpr int lds_bytes(bool odd) { return std::max(ring(odd) * stage_bytes(odd), kOutLds); }
    static_assert(ring(true) >= 2 && PER_CU * (lds_bytes(false) + kStaticLds) <= kLdsBytes && lds_bytes(true) + kStaticLds <= kLdsBytes && ring(false) == NS);
};

template <class T, bool EXPERTS, bool ODD>
__global__ __launch_bounds__(T::kThreads, T::kPerSimd) void nvfp4_gemm_wide_kernel(GemmParams p)
{
    constexpr int FM = T::kFM, FN = T::kFN, NS = T::ring(ODD), BM = T::BM, BN = T::BN, F = FM + FN, kWaves = T::kWaves;
    constexpr int kStage = T::stage_bytes(ODD), kWordsA = BM * 8, kWordsB = BN * 8;
    constexpr int kOffSB = T::kOffSA + kWordsA * (ODD ? 2 : 1);
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    __shared__ int32_t s_slot[EXPERTS ? BN : 1];
    const int lane = threadIdx.x % 64;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const Where w = locate<EXPERTS, BM, BN, T::kThreads>(p, s_slot);
    if (EXPERTS && w.l < 0)
        return;

    // --- this wave's copies
    const int stages = p.stages;
    constexpr int CA = T::TA / kWaves, CB = T::TB / kWaves;
    constexpr int CSA = T::TSA / kWaves, CSB = (T::TSB + kWaves - 1) / kWaves;
    // where B's words are fewer than a copy per wave, the first TSB waves make them
    const bool has_sb = T::TSB % kWaves == 0 || wave < T::TSB;
    const uint32_t step_words = p.blocked ? 1024 : 8, back_words = p.blocked ? 512 : 4;
    Source a = source_a(p, w), b = source_b<EXPERTS>(p, w);
    uint32_t oa[CA], ob[CB], osa[CSA], osb[CSB];
    int half_a[CSA], half_b[CSB];
    // lane's 16 bytes of a 1 KiB copy: row lane / 4 of 16, piece swizzled back
    const int piece = (lane % 4) ^ ((lane / 16) % 4);
#pragma unroll
    for (int i = 0; i < CA; ++i)
        oa[i] = codes_at_a(p, w, (wave + kWaves * i) * 16 + lane / 4) + piece * 16;
#pragma unroll
    for (int i = 0; i < CB; ++i)
        ob[i] = codes_at_b<EXPERTS>(p, w, s_slot, (wave + kWaves * i) * 16 + lane / 4) + piece * 16;
    // word v of a stage's scale words: block of 32 * LW rows, half, line, word
    auto word_row = [](int v, int LW) { return v / (LW * 64) * (LW * 32) + (v % LW) * 32 + (v / LW) % 32; };
    auto word_half = [](int v, int LW) { return (v / (LW * 32)) % 2; };
#pragma unroll
    for (int i = 0; i < CSA; ++i) {
        const int v = (wave + kWaves * i) * 64 + lane;
        half_a[i] = word_half(v, T::LA);
        osa[i] = words_at_a(p, w, word_row(v, T::LA), half_a[i]);
    }
#pragma unroll
    for (int i = 0; i < CSB; ++i) {
        const int v = has_sb ? (wave + kWaves * i) * 64 + lane : 0;
        half_b[i] = word_half(v, T::LB);
        osb[i] = words_at_b<EXPERTS>(p, w, s_slot, word_row(v, T::LB), half_b[i]);
    }
    const uint32_t lds_base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;

    // issues the copies of the next stage, `st` of all K, into ring slot `slot`
    auto issue = [&](int st, int slot) {
        const uint32_t base = lds_base + slot * kStage;
        const int left = p.K - st * kStageK;
        // codes past K's end: the row's first of the stage (their scales are masked)
        const uint32_t back = left <= piece * 32 ? piece * 16 : 0;
#pragma unroll
        for (int i = 0; i < CA; ++i)
            copy16(a.codes, oa[i] - back, base + (wave + kWaves * i) * 1024);
#pragma unroll
        for (int i = 0; i < CB; ++i)
            copy16(b.codes, ob[i] - back, base + T::kOffB + (wave + kWaves * i) * 1024);
#pragma unroll
        for (int i = 0; i < CSA; ++i)
            copy_words<ODD>(a.words, osa[i], left - half_a[i] * 64, back_words,
                            base + T::kOffSA + (wave + kWaves * i) * 256, kWordsA);
        if (has_sb) {
#pragma unroll
            for (int i = 0; i < CSB; ++i)
                copy_words<ODD>(b.words, osb[i], left - half_b[i] * 64, back_words,
                                base + kOffSB + (wave + kWaves * i) * 256, kWordsB);
        }
        a.codes += 64, b.codes += 64;
        a.words += step_words, b.words += step_words;
    };
    // waits until only the `younger` last stages' copies are out
    constexpr int kW = ODD ? 2 : 1, kBase = CA + CB + CSA * kW + (T::TSB % kWaves == 0 ? CSB * kW : 0);
    auto wait_stage = [&](auto younger) {
        if (T::TSB % kWaves != 0 && has_sb)
            wait_copies<younger() * (kBase + CSB * kW)>();
        else
            wait_copies<younger() * kBase>();
    };
    typedef std::integral_constant<int, 0> None;

    // --- the product
    float16_t acc[FN][FM];
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                acc[j][i][r] = 0.0f;
    const int wm = wave / T::kWN, wn = wave % T::kWN;
    const int half = lane / 32, l32 = lane % 32, swz = (l32 / 4) % 4;
    const int ra0 = wm * FM * 32, rb0 = wn * FN * 32;
    const uint32_t codes_a = (ra0 + l32) * 64, codes_b = T::kOffB + (rb0 + l32) * 64;
    const uint32_t words_a = T::kOffSA + (ra0 / (32 * T::LA)) * (T::LA * 256) + half * (T::LA * 128) +
                             l32 * (T::LA * 4) + (ra0 / 32 % T::LA) * 4;
    const uint32_t words_b = kOffSB + (rb0 / (32 * T::LB)) * (T::LB * 256) + half * (T::LB * 128) +
                             l32 * (T::LB * 4) + (rb0 / 32 % T::LB) * 4;
    // A stage is 8 steps of 16 k (per half of the lanes: one dword of codes per
    // row), codes being read 16 bytes at a time. A wave whose rows of B all lie past
    // the list's end works as the others do (12% of the rows of 16384 slots of 32 experts).
    auto compute = [&](int st, int slot) {
        const uint8_t *base = lds + slot * kStage;
        uint32_t word[F], sa[FM], sb[FN];
        load_words<FM, ODD>(base + words_a, kWordsA, sa);
        load_words<FN, ODD>(base + words_b, kWordsB, sb);
        // past K's end: scales of 0
        const uint32_t valid = word_mask(p.K - st * kStageK - half * 64);
#pragma unroll
        for (int f = 0; f < F; ++f)
            word[f] = (f < FM ? sa[f < FM ? f : 0] : sb[f < FM ? 0 : f - FM]) & valid;
#pragma unroll
        for (int part = 0; part < 2; ++part) {
            const uint32_t pc = ((2 * half + part) ^ swz) * 16;
            uint4_t q[F];
            half2_t sc[F];
#pragma unroll
            for (int f = 0; f < F; ++f) {
                q[f] = f < FM ? *(const uint4_t *)(base + codes_a + f * 2048 + pc)
                              : *(const uint4_t *)(base + codes_b + (f - FM) * 2048 + pc);
                sc[f] = part ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(word[f], 1.0f, true)
                             : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(word[f], 1.0f, false);
            }
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                half8_t v[F];
#pragma unroll
                for (int f = 0; f < F; ++f) {
                    const half2_t s = d < 2 ? (half2_t){sc[f].x, sc[f].x} : (half2_t){sc[f].y, sc[f].y};
                    const uint32_t codes[4] = {q[f].x, q[f].y, q[f].z, q[f].w};
                    v[f] = decode8(codes[d], s);
                }
#pragma unroll
                for (int j = 0; j < FN; ++j)
#pragma unroll
                    for (int i = 0; i < FM; ++i)
                        acc[j][i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v[FM + j], v[i], acc[j][i], 0, 0, 0);
            }
        }
    };

#pragma unroll
    for (int s = 0; s < NS - 1; ++s)
        if (s < stages)
            issue(s, s);
    const Scale scale = total_scale<EXPERTS>(p, w.l);
    int slot = 0, i = 0;
    for (; i + NS - 1 < stages; ++i) {
        // stage i has landed when only the NS - 2 younger ones are out; past the
        // barrier every wave has done with stage i - 1, whose slot is next
        wait_stage(std::integral_constant<int, NS - 2>{});
        barrier();
        issue(i + NS - 1, slot == 0 ? NS - 1 : slot - 1);
        compute(i, slot);
        slot = slot + 1 == NS ? 0 : slot + 1;
    }
    for (; i < stages; ++i) {
        wait_stage(None{});
        barrier();
        compute(i, slot);
        slot = slot + 1 == NS ? 0 : slot + 1;
    }

    // --- results. Register r of fragment (j, i): row of B rb0 + 32 j + 8 (r / 4) + 4 (lane / 32) + r % 4,
    // row of A ra0 + 32 i + lane % 32.
    // Through LDS, so that a lane stores 16 bytes of a row at a time (2-byte
    // stores of 32 neighbours took 17 us per 256 x 256 tile, most of it these).
    barrier();                                  // all waves have read their last stage
    uint8_t *const out = lds + wave * (32 * T::kPitch);
    const int size = p.dtype == NVFP4_F32 ? 4 : 2;
    const int per_row = FM * 32 * size / 16, rows_at_once = 64 / per_row, per_piece = 16 / size;
    const int piece_n = lane / per_row, piece_m = lane % per_row * per_piece;
    const int m = w.m0 + ra0 + piece_m;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
#pragma unroll
        for (int r = 0; r < 16; ++r)
#pragma unroll
            for (int i = 0; i < FM; ++i)
                store_value(out + (8 * (r / 4) + 4 * half + r % 4) * T::kPitch, 32 * i + l32, scale.of(acc[j][i][r]), p.dtype);
        asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
        for (int n = piece_n; n < 32; n += rows_at_once) {
            const uint4_t v = *(const uint4_t *)(out + n * T::kPitch + piece_m * size);
            const int64_t row = row_at<EXPERTS>(p, w, s_slot, rb0 + 32 * j + n);
            if (row < 0 || m >= p.M)
                continue;
            uint8_t *c = p.c + (row + m) * size;
            if (m + per_piece <= p.M) {
                __builtin_memcpy(c, &v, 16);
            } else {
                for (int x = 0; x < p.M - m; ++x) {
                    if (size == 4)
                        ((uint32_t *)c)[x] = *(const uint32_t *)(out + n * T::kPitch + (piece_m + x) * 4);
                    else
                        ((uint16_t *)c)[x] = *(const uint16_t *)(out + n * T::kPitch + (piece_m + x) * 2);
                }
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
    }
}

// ------------------------------------------------------------------ wave kernel

// WM x KW waves: WM of them share the rows of A, each with FM x FN fragments, and
// KW take a row range's stages in turn, RUN (1 or 2) neighbouring ones at a time;
// NS stages in each wave's ring.
template <int FM, int FN, int WM, int KW, int NS, int PER_CU, int RUN>
struct WaveTile {
    static constexpr int kRun = RUN, kFM = FM, kFN = FN, kWM = WM, kKW = KW, kNS = NS, kPerCu = PER_CU;
    static constexpr int kWaveM = 32 * FM, BM = kWaveM * WM, BN = 32 * FN, kThreads = 64 * WM * KW;
    static constexpr int kOffB = kWaveM * 64, kOffSA = kOffB + BN * 64;
    static constexpr int stage_bytes(bool odd) { return kOffSA + (kWaveM + BN) * (odd ? 16 : 8); }
    static constexpr int lds_bytes(bool odd) { return std::max(WM * KW * NS * stage_bytes(odd), KW > 1 ? WM * KW * FM * FN * 4096 : 0); }
    static_assert(lds_bytes(true) + kStaticLds <= kLdsBytes);
    // the KW waves share the registers of a range evenly, and slices are added 8 at a time
    static_assert(FN * FM * 16 % KW == 0 && (FN * FM * 16 / KW < 8 || FN * FM * 16 / KW % 8 == 0));
};

template <class T, bool EXPERTS, bool ODD>
__global__ __launch_bounds__(T::kThreads, T::kPerCu) void nvfp4_gemm_wave_kernel(GemmParams p)
{
    constexpr int FM = T::kFM, FN = T::kFN, KW = T::kKW, NS = T::kNS, BM = T::BM, BN = T::BN, F = FM + FN;
    constexpr int kStage = T::stage_bytes(ODD), kWordsA = T::kWaveM * 8, kWordsB = BN * 8;
    constexpr int kOffSB = T::kOffSA + kWordsA * (ODD ? 2 : 1);
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    __shared__ int32_t s_slot[EXPERTS ? BN : 1];
    __shared__ uint32_t s_ticket;
    const int lane = threadIdx.x % 64;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    Where w = locate<EXPERTS, BM, BN, T::kThreads>(p, s_slot);
    if (EXPERTS && w.l < 0)
        return;
    // this wave's rows (its first may lie past M: then it works on row M - 1 and stores nothing)
    const int wk = wave % KW, rows0 = w.m0 + wave / KW * T::kWaveM;
    w.m0 = min(rows0, p.M - 1);
    // and stages: RUN from first on, then those RUN * KW further
    constexpr int RUN = T::kRun;
    const int begin = w.split * p.stages_per_split, count = min(p.stages_per_split, p.stages - begin);
    const int stages = count / (RUN * KW) * RUN + min(max(count % (RUN * KW) - RUN * wk, 0), RUN);
    const int first = begin + RUN * wk;
    auto stage_at = [&](int n) { return first + n / RUN * (RUN * KW) + n % RUN; };
    // copies of B's codes: 16 rows each, only those that hold rows of the tile
    const int groups_b = (w.count + 15) / 16;
    const uint32_t one_words = p.blocked ? 1024 : 8, back_words = p.blocked ? 512 : 4;
    Source a = source_a(p, w), b = source_b<EXPERTS>(p, w);
    a.codes += (int64_t)first * 64, b.codes += (int64_t)first * 64;
    a.words += (int64_t)first * one_words, b.words += (int64_t)first * one_words;
    uint32_t oa[2 * FM], ob[2 * FN], osa[FM], osb[FN];
    const int piece = (lane % 4) ^ ((lane / 16) % 4);
    const int half = lane / 32, l32 = lane % 32, swz = (l32 / 4) % 4;
#pragma unroll
    for (int i = 0; i < 2 * FM; ++i)
        oa[i] = codes_at_a(p, w, i * 16 + lane / 4) + piece * 16;
#pragma unroll
    for (int i = 0; i < 2 * FN; ++i)
        ob[i] = codes_at_b<EXPERTS>(p, w, s_slot, i * 16 + lane / 4) + piece * 16;
    // words: fragment i's 64 words of a stage, half by half, row by row
#pragma unroll
    for (int i = 0; i < FM; ++i)
        osa[i] = words_at_a(p, w, 32 * i + l32, half);
#pragma unroll
    for (int j = 0; j < FN; ++j)
        osb[j] = words_at_b<EXPERTS>(p, w, s_slot, 32 * j + l32, half);
    uint8_t *ring = lds + wave * (NS * kStage);
    const uint32_t ring_base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds + wave * (NS * kStage);

    auto issue = [&](int n, int slot) {                         // the wave's n-th stage, the next one
        const uint32_t base = ring_base + slot * kStage;
        const int left = p.K - stage_at(n) * kStageK;
        const uint32_t back = left <= piece * 32 ? piece * 16 : 0;
#pragma unroll
        for (int i = 0; i < 2 * FM; ++i)
            copy16(a.codes, oa[i] - back, base + i * 1024);
#pragma unroll
        for (int i = 0; i < FM; ++i)
            copy_words<ODD>(a.words, osa[i], left - half * 64, back_words, base + T::kOffSA + i * 256, kWordsA);
#pragma unroll
        for (int j = 0; j < FN; ++j)
            copy_words<ODD>(b.words, osb[j], left - half * 64, back_words, base + kOffSB + j * 256, kWordsB);
#pragma unroll
        for (int i = 0; i < 2 * FN; ++i)
            if (i < groups_b)
                copy16(b.codes, ob[i] - back, base + T::kOffB + i * 1024);
        const int step = RUN == 1 ? KW : (n % 2 ? 2 * KW - 1 : 1);
        a.codes += 64 * step, b.codes += 64 * step;
        a.words += one_words * step, b.words += one_words * step;
    };
    constexpr int kBase = 2 * FM + F * (ODD ? 2 : 1);
    auto wait_younger = [&](auto younger) {
        if (groups_b == 1)
            wait_copies<younger() * (kBase + 1)>();
        else if (2 * FN == 2 || groups_b == 2)
            wait_copies<younger() * (kBase + 2)>();
        else if (groups_b == 3)
            wait_copies<younger() * (kBase + 3)>();
        else
            wait_copies<younger() * (kBase + 4)>();
    };

    float16_t acc[FN][FM];
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                acc[j][i][r] = 0.0f;
    auto compute = [&](int n, int slot) {
        const uint8_t *base = ring + slot * kStage;
        const uint32_t valid = word_mask(p.K - stage_at(n) * kStageK - half * 64);
        uint32_t word[F];
        uint4_t q[F][2];
#pragma unroll
        for (int f = 0; f < F; ++f) {
            const uint32_t row = f < FM ? f * 2048 : T::kOffB + (f - FM) * 2048;
            uint32_t one[1];
            load_words<1, ODD>(base + (f < FM ? T::kOffSA + f * 256 : kOffSB + (f - FM) * 256) + lane * 4,
                               f < FM ? kWordsA : kWordsB, one);
            word[f] = one[0] & valid;
#pragma unroll
            for (int s = 0; s < 2; ++s)
                q[f][s] = *(const uint4_t *)(base + row + l32 * 64 + ((2 * half + s) ^ swz) * 16);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                half8_t v[F];
#pragma unroll
                for (int f = 0; f < F; ++f) {
                    const half2_t two = s ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(word[f], 1.0f, true)
                                          : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(word[f], 1.0f, false);
                    const half2_t sc = d < 2 ? (half2_t){two.x, two.x} : (half2_t){two.y, two.y};
                    const uint32_t codes[4] = {q[f][s].x, q[f][s].y, q[f][s].z, q[f][s].w};
                    v[f] = decode8(codes[d], sc);
                }
#pragma unroll
                for (int j = 0; j < FN; ++j)
#pragma unroll
                    for (int i = 0; i < FM; ++i)
                        acc[j][i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v[FM + j], v[i], acc[j][i], 0, 0, 0);
            }
        }
    };

#pragma unroll
    for (int s = 0; s < NS - 1; ++s)
        if (s < stages)
            issue(s, s);
    const Scale scale = total_scale<EXPERTS>(p, w.l);
    int slot = 0, n = 0;
    for (; n + NS - 1 < stages; ++n) {
        // the slot of stage n - 1, whose reads are done, takes stage n + NS - 1;
        // stage n has landed when only the NS - 1 younger ones are out
        asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
        issue(n + NS - 1, slot == 0 ? NS - 1 : slot - 1);
        wait_younger(std::integral_constant<int, NS - 1>{});
        asm volatile("" : : : "memory");
        compute(n, slot);
        slot = slot + 1 == NS ? 0 : slot + 1;
    }
    wait_copies<0>();
    asm volatile("" : : : "memory");
    for (; n < stages; ++n) {
        compute(n, slot);
        slot = slot + 1 == NS ? 0 : slot + 1;
    }

    // --- the waves' sums through LDS, in the order of the waves: of the KW waves
    // of a row range, wave wk takes registers wk * R .. of its FN * FM * 16
    constexpr int R = FN * FM * 16 / KW;
    float sum[R];
    if constexpr (KW > 1) {
        __syncthreads();
        float *sums = (float *)lds + wave / KW * KW * (FN * FM * 1024);      // [wave][register][lane]
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    sums[(wk * (FN * FM * 16) + (j * FM + i) * 16 + r) * 64 + lane] = acc[j][i][r];
        __syncthreads();
#pragma unroll
        for (int x = 0; x < R; ++x) {
            sum[x] = 0.0f;
#pragma unroll
            for (int o = 0; o < KW; ++o)
                sum[x] += sums[(o * (FN * FM * 16) + wk * R + x) * 64 + lane];
        }
    } else {
#pragma unroll
        for (int x = 0; x < R; ++x)
            sum[x] = acc[x / 16 / FM][x / 16 % FM][x % 16];
    }
    int64_t at[R];
#pragma unroll
    for (int x = 0; x < R; ++x) {
        const int g = wk * R + x, f = g / 16, r = g % 16, j = f / FM, i = f % FM;
        const int64_t row = row_at<EXPERTS>(p, w, s_slot, 32 * j + 8 * (r / 4) + 4 * half + r % 4);
        const int m = rows0 + 32 * i + l32;
        at[x] = row < 0 || m >= p.M ? -1 : row + m;
    }
    if (p.splits > 1) {
        const int64_t one = (int64_t)(EXPERTS ? p.N : p.N * (int64_t)p.L) * p.M;
#pragma unroll
        for (int x = 0; x < R; ++x)
            if (at[x] >= 0)
                __hip_atomic_store(&p.partials[w.split * one + at[x]], sum[x], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (!last_of_tile(p, w.tile, &s_ticket))
            return;
#pragma unroll
        for (int g = 0; g < R; g += R < 8 ? R : 8) {
            constexpr int G = R < 8 ? R : 8;
            int64_t some[G];
            float part[G];
#pragma unroll
            for (int x = 0; x < G; ++x)
                some[x] = at[g + x];
            add_slices<G>(p, one, some, part);
#pragma unroll
            for (int x = 0; x < G; ++x)
                sum[g + x] = part[x];
        }
    }
#pragma unroll
    for (int x = 0; x < R; ++x)
        if (at[x] >= 0)
            store_value(p.c, at[x], scale.of(sum[x]), p.dtype);
}

// ------------------------------------------------------------------ plans

typedef Tile<2, 4, 4, 2, 3, 1> TileLarge;       // 256 x 256, 8 waves
typedef Tile<4, 2, 2, 2, 2, 2> TileTall;        // 256 x 128
typedef Tile<2, 2, 2, 2, 4, 2> TileMid;         // 128 x 128
typedef WaveTile<2, 2, 1, 4, 2, 2, 2> TileSquare;  // 64 x 64, 4 waves along K
typedef WaveTile<2, 1, 2, 2, 2, 3, 1> TileFew;     // 128 x 32, 2 waves along K
typedef WaveTile<2, 1, 1, 4, 2, 3, 1> TileFewK;    // 64 x 32, 4 waves along K
typedef WaveTile<1, 1, 1, 4, 2, 3, 1> TileOne;     // 32 x 32, 4 waves along K
typedef WaveTile<1, 1, 1, 8, 3, 1, 1> TileOneK;    // 32 x 32, 8 waves along K

enum class Kind { Large, Tall, Mid, Square, Few, FewK, One, OneK };

struct Plan {
    Kind kind;
    int32_t bm, bn;
    int64_t tiles_m, tiles_n, tiles;            // tiles: of all batches (experts: upper bound)
    int32_t stages, splits, per_split;
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

bool gemm_shape(int64_t M, int64_t N, int64_t K, int64_t L)
{
    return M >= 1 && N >= 1 && L >= 1 && K >= 32 && K % 32 == 0 && K <= (INT64_C(1) << 22) &&
           M <= (INT64_C(1) << 30) && N <= (INT64_C(1) << 30) && L <= (INT64_C(1) << 30) &&
           L <= (INT64_C(1) << 61) / K / std::max(M, N) && L <= (INT64_C(1) << 60) / M / N;
}

// The tile shapes and what they cost, from which the plans choose. us on one
// MI355X, measured over 60 shapes (M and N 16 .. 7168, K 512 .. 16384, 1 to 16
// slices; 1 to 16384 tokens of 8 to 64 experts): `alone`, a workgroup's time per
// stage (128 k) with its CU to itself;
// `each`, what a stage adds to the CU's time per workgroup when more share it;
// `start`, what a workgroup adds besides (its first copies and its results);
// `listed`, what one of routed experts adds to that (its list and weights that
// nobody has read yet).
//   Large tiles decode less per product (6 vector instructions per MFMA for 256 x
// 256 and 256 x 128, 8 for 128 x 128 and 64 x 64, 12 for 32 wide, 16 for 32 x 32)
// and need many tiles to fill the GPU; small ones put their waves along K. E.g.
// 4096 x 333 x 7168: 64 x 32 33 us, 64 x 64 34, 128 x 32 37, 128 x 128 56, 256 x
// 128 above 100; 4096 x 1024 x 4096: 128 x 128 40, 64 x 64 45, 64 x 32 52, 256 x
// 128 64; 7168 x 4096 x 16384: 256 x 256 760, 256 x 128 810, 64 x 64 970; 4096 x
// 128 x 7168: 64 x 32 14.4, 32 x 32 15.4, 64 x 64 18.2; 7168 x 16 x 16384: 32 x 32
// with 8 waves along K 17.3, with 4 20.2, 64 x 32 in two slices 19.1.
//   The table does not know the result's bytes, and was not measured below K = 512:
// there the result bounds the time, and 128 x 128 tiles with a lone stage or few
// are taken. 4096 x 4096 x 128: 28 us to float32, 22 to bfloat16 (67 and 34 MB
// stored); 8192 x 2900 x 128: 39 and 31 (95 and 48 MB); 4096 x 4096 x 32 as x 128.
//   A shape that is never fastest in a use is not built for it: 256 x 256 against
// 256 x 128 for 16384 slots of 32 experts, 7168 x 4096: 1068 against 970 us; 256 x
// 128 against 128 x 128 and 256 x 256 in dense products: at most 2 % ahead of the
// better one. The wide kernel has no slices: they would be used where few tiles
// have a long K, and there 64 x 64 in slices is ahead.
enum Use { kDense = 1, kExperts = 2, kBoth = 3 };
struct Shape {
    Kind kind;
    int bm, bn, uses, max_splits;
    double alone, each, start, listed;
};
constexpr Shape kShapes[] = {
    {Kind::Large, TileLarge::BM, TileLarge::BN, kDense, 1, 2.85, 2.88, 8.0, 0.0},
    {Kind::Tall, TileTall::BM, TileTall::BN, kExperts, 1, 2.03, 1.58, 5.0, 9.0},
    {Kind::Mid, TileMid::BM, TileMid::BN, kBoth, 1, 1.05, 0.98, 1.0, 4.0},
    {Kind::Square, TileSquare::BM, TileSquare::BN, kBoth, kMaxSplits, 0.38, 0.30, 0.3, 1.7},
    {Kind::Few, TileFew::BM, TileFew::BN, kBoth, kMaxSplits, 0.40, 0.35, 0.3, 1.5},
    {Kind::FewK, TileFewK::BM, TileFewK::BN, kBoth, kMaxSplits, 0.19, 0.185, 0.3, 0.9},
    {Kind::One, TileOne::BM, TileOne::BN, kBoth, kMaxSplits, 0.115, 0.095, 0.2, 0.7},
    {Kind::OneK, TileOneK::BM, TileOneK::BN, kDense, kMaxSplits, 0.085, 0.10, 0.2, 0.0},
};
constexpr double kCus = 256.0, kSplitUs = 1.0, kSliceUs = 0.15, kPartialBytesPerUs = 2.0e6;

// Cheapest shape and number of K slices. tiles_of(shape, plan) fills the tile
// counts and returns the expected number of tiles; rows: of the result.
template <typename F>
Plan choose(int64_t M, int64_t K, int64_t rows, bool experts, F tiles_of)
{
    Plan best{};
    double best_us = 0.0;
    for (const Shape &s : kShapes) {
        if (!(s.uses & (experts ? kExperts : kDense)))
            continue;
        Plan p{};
        p.kind = s.kind, p.bm = s.bm, p.bn = s.bn;
        p.stages = (int32_t)ceil_div(K, kStageK);
        p.tiles_m = ceil_div(M, s.bm);
        const double tiles = tiles_of(s, p);
        for (int64_t splits = 1; splits <= s.max_splits && splits <= p.stages; splits *= 2) {
            p.per_split = (int32_t)ceil_div(p.stages, splits);
            p.splits = (int32_t)ceil_div(p.stages, p.per_split);
            if (p.splits > 1 && (p.tiles > kMaxTickets || p.splits * rows > kMaxPartialBytes / 4 / M))
                break;
            const double n = tiles * p.splits / kCus, load = experts ? std::max(n, 1.0) : std::ceil(n);
            double us = p.per_split * std::max(s.alone, s.each * load) + (s.start + (experts ? s.listed : 0.0)) * load;
            if (p.splits > 1)
                us += kSplitUs + p.splits * (kSliceUs + 8.0 * rows * M / kPartialBytesPerUs);
            if (best_us == 0.0 || us < best_us) {
                best = p;
                best_us = us;
            }
        }
    }
    return best;
}

Plan dense_plan(int64_t M, int64_t N, int64_t K, int64_t L)
{
    return choose(M, K, N * L, false, [&](const Shape &s, Plan &p) {
        p.tiles_n = ceil_div(N, s.bn);
        p.tiles = p.tiles_m * p.tiles_n * L;
        return (double)p.tiles;
    });
}

// The lists are on the device: the grid has room for the most tiles that S slots
// can make, the choice goes by what S slots spread over the experts make.
Plan experts_plan(int64_t M, int64_t K, int64_t E, int64_t S)
{
    const double mean = (double)S / E, hit = E * (1.0 - std::exp(-mean));
    return choose(M, K, S, true, [&](const Shape &s, Plan &p) {
        p.tiles_n = std::min<int64_t>(S, S / s.bn + std::min(E, S));
        p.tiles = p.tiles_m * p.tiles_n;
        return std::max(hit, (double)S / s.bn + 0.5 * hit) * p.tiles_m;
    });
}

size_t plan_workspace(const Plan &p, int64_t rows, int64_t M)
{
    return p.splits > 1 ? (size_t)((kTicketBytes + p.splits * rows * M * 4 + 255) / 256 * 256) : 0;
}

bool known_type(int dtype) { return dtype == NVFP4_F16 || dtype == NVFP4_BF16 || dtype == NVFP4_F32; }
bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

template <class T, bool EXPERTS>
hipError_t launch_wide(const GemmParams &p, int64_t grid, hipStream_t st)
{
    const bool odd = !p.blocked && p.K % 64 != 0;               // plain rows of 2-byte alignment
    auto go = [&](auto kern) {
        hipLaunchKernelGGL(kern, dim3((uint32_t)grid), dim3(T::kThreads), T::lds_bytes(odd), st, p);
    };
    odd ? go(nvfp4_gemm_wide_kernel<T, EXPERTS, true>) : go(nvfp4_gemm_wide_kernel<T, EXPERTS, false>);
    return hipGetLastError();
}

template <class T, bool EXPERTS>
hipError_t launch_wave(const GemmParams &p, int64_t grid, hipStream_t st)
{
    const bool odd = !p.blocked && p.K % 64 != 0;
    auto go = [&](auto kern) {
        hipLaunchKernelGGL(kern, dim3((uint32_t)grid), dim3(T::kThreads), T::lds_bytes(odd), st, p);
    };
    odd ? go(nvfp4_gemm_wave_kernel<T, EXPERTS, true>) : go(nvfp4_gemm_wave_kernel<T, EXPERTS, false>);
    return hipGetLastError();
}

template <bool EXPERTS>
nvfp4_status_t run(const Plan &plan, const GemmParams &p, hipStream_t st)
{
    const int64_t grid = plan.tiles * plan.splits;
    hipError_t e = hipSuccess;
    switch (plan.kind) {
    case Kind::Large:
        if constexpr (!EXPERTS)
            e = launch_wide<TileLarge, EXPERTS>(p, grid, st);
        break;
    case Kind::Tall:
        if constexpr (EXPERTS)
            e = launch_wide<TileTall, EXPERTS>(p, grid, st);
        break;
    case Kind::Mid: e = launch_wide<TileMid, EXPERTS>(p, grid, st); break;
    case Kind::Square: e = launch_wave<TileSquare, EXPERTS>(p, grid, st); break;
    case Kind::Few: e = launch_wave<TileFew, EXPERTS>(p, grid, st); break;
    case Kind::FewK: e = launch_wave<TileFewK, EXPERTS>(p, grid, st); break;
    case Kind::One: e = launch_wave<TileOne, EXPERTS>(p, grid, st); break;
    case Kind::OneK:
        if constexpr (!EXPERTS)
            e = launch_wave<TileOneK, EXPERTS>(p, grid, st);
        break;
    }
    if (e == hipSuccess)
        return NVFP4_OK;
    nvfp4_record_hip_error((int)e);
    return NVFP4_ERR_HIP;
}

nvfp4_status_t check_operands(const void *a, const void *b, const void *sfa, const void *sfb, const void *c, int dtype,
                              int sf_layout, float alpha, const float *scale_a, const float *scale_b)
{
    if (sf_layout != NVFP4_SF_PLAIN && sf_layout != NVFP4_SF_BLOCKED)
        return NVFP4_ERR_INVALID_LAYOUT;
    if (!aligned(a, 16) || !aligned(b, 16) || !aligned(sfa, 16) || !aligned(sfb, 16) ||
        !aligned(c, dtype == NVFP4_F32 ? 4 : 2) || (scale_a && !aligned(scale_a, 4)) ||
        (scale_b && !aligned(scale_b, 4)))
        return NVFP4_ERR_MISALIGNED;
    if (!std::isfinite(alpha))
        return NVFP4_ERR_INVALID_SCALE;
    return NVFP4_OK;
}

GemmParams fill(const Plan &plan, const void *a, const void *b, const void *sfa, const void *sfb, void *c, int dtype,
                int64_t M, int64_t N, int64_t K, int64_t L, int sf_layout, float alpha, const float *scale_a,
                const float *scale_b, void *workspace)
{
    const int64_t nkb = K / 16, ncb = (nkb + 3) / 4;
    GemmParams p{};
    p.a = (const uint8_t *)a, p.b = (const uint8_t *)b, p.sfa = (const uint8_t *)sfa, p.sfb = (const uint8_t *)sfb;
    p.c = (uint8_t *)c, p.dtype = dtype;
    p.scale_a = scale_a, p.scale_b = scale_b;
    p.tickets = (uint32_t *)workspace;
    p.partials = workspace ? (float *)((uint8_t *)workspace + kTicketBytes) : nullptr;
    p.blocked = sf_layout == NVFP4_SF_BLOCKED;
    p.sfa_batch = p.blocked ? (M + 127) / 128 * ncb * 512 : M * nkb;
    p.sfb_batch = p.blocked ? (N + 127) / 128 * ncb * 512 : N * nkb;
    p.M = (int32_t)M, p.N = (int32_t)N, p.K = (int32_t)K, p.L = (int32_t)L;
    p.slots_per_row = 1;
    p.tiles_m = (int32_t)plan.tiles_m, p.tiles_n = (int32_t)plan.tiles_n;
    p.splits = plan.splits, p.stages_per_split = plan.per_split, p.stages = plan.stages;
    p.alpha = alpha;
    return p;
}

} // namespace

extern "C" {

nvfp4_status_t nvfp4_gemm_plan(int64_t M, int64_t N, int64_t K, int64_t L, nvfp4_gemm_plan_t *plan)
{
    if (!plan)
        return NVFP4_ERR_NULL_POINTER;
    if (!gemm_shape(M, N, K, L))
        return NVFP4_ERR_INVALID_SHAPE;
    const Plan p = dense_plan(M, N, K, L);
    if (p.tiles > kMaxGrid / p.splits)
        return NVFP4_ERR_INVALID_SHAPE;
    plan->tile_m = p.bm;
    plan->tile_n = p.bn;
    plan->k_splits = p.splits;
    plan->k_per_split = p.per_split * kStageK;
    plan->workgroups = p.tiles * p.splits;
    return NVFP4_OK;
}

size_t nvfp4_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t L)
{
    return gemm_shape(M, N, K, L) ? plan_workspace(dense_plan(M, N, K, L), N * L, M) : 0;
}

nvfp4_status_t nvfp4_gemm(const void *a, const void *b, const void *sfa, const void *sfb, void *c, int dtype, int64_t M,
                          int64_t N, int64_t K, int64_t L, int sf_layout, float alpha, const float *scale_a,
                          const float *scale_b, void *workspace, size_t workspace_bytes, void *stream)
{
    if (!a || !b || !sfa || !sfb || !c)
        return NVFP4_ERR_NULL_POINTER;
    if (!known_type(dtype))
        return NVFP4_ERR_INVALID_TYPE;
    if (!gemm_shape(M, N, K, L))
        return NVFP4_ERR_INVALID_SHAPE;
    const nvfp4_status_t st = check_operands(a, b, sfa, sfb, c, dtype, sf_layout, alpha, scale_a, scale_b);
    if (st != NVFP4_OK)
        return st;
    const Plan plan = dense_plan(M, N, K, L);
    if (plan.tiles > kMaxGrid / plan.splits)
        return NVFP4_ERR_INVALID_SHAPE;
    const size_t need = plan_workspace(plan, N * L, M);
    if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
        return NVFP4_ERR_WORKSPACE;
    const GemmParams p = fill(plan, a, b, sfa, sfb, c, dtype, M, N, K, L, sf_layout, alpha, scale_a, scale_b, workspace);
    return run<false>(plan, p, (hipStream_t)stream);
}

size_t nvfp4_gemm_experts_workspace_bytes(int64_t M, int64_t K, int64_t E, int64_t S)
{
    if (!gemm_shape(M, S, K, E) || E > kMaxExperts)
        return 0;
    return plan_workspace(experts_plan(M, K, E, S), S, M);
}

nvfp4_status_t nvfp4_gemm_experts(const void *a, const void *b, const void *sfa, const void *sfb, void *c, int dtype,
                                  int64_t M, int64_t K, int64_t E, int64_t rows, int64_t slots_per_row, int sf_layout,
                                  const int32_t *offsets, const int32_t *order, float alpha, const float *scale_a,
                                  const float *scale_b, void *workspace, size_t workspace_bytes, void *stream)
{
    if (!a || !b || !sfa || !sfb || !c || !offsets || !order)
        return NVFP4_ERR_NULL_POINTER;
    if (!known_type(dtype))
        return NVFP4_ERR_INVALID_TYPE;
    if (rows < 1 || slots_per_row < 1 || E > kMaxExperts || rows > (INT64_C(1) << 30) / slots_per_row ||
        !gemm_shape(M, rows * slots_per_row, K, E) || rows > (INT64_C(1) << 32) / (K / 2))
        return NVFP4_ERR_INVALID_SHAPE;
    const nvfp4_status_t st = check_operands(a, b, sfa, sfb, c, dtype, sf_layout, alpha, scale_a, scale_b);
    if (st != NVFP4_OK)
        return st;
    if (!aligned(offsets, 4) || !aligned(order, 4))
        return NVFP4_ERR_MISALIGNED;
    const int64_t S = rows * slots_per_row;
    const Plan plan = experts_plan(M, K, E, S);
    if (plan.tiles > kMaxGrid / plan.splits)
        return NVFP4_ERR_INVALID_SHAPE;
    const size_t need = plan_workspace(plan, S, M);
    if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
        return NVFP4_ERR_WORKSPACE;
    GemmParams p = fill(plan, a, b, sfa, sfb, c, dtype, M, S, K, E, sf_layout, alpha, scale_a, scale_b, workspace);
    p.offsets = offsets, p.order = order;
    p.slots_per_row = (int32_t)slots_per_row;
    return run<true>(plan, p, (hipStream_t)stream);
}

} // extern "C"
