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
// Kernel. A workgroup of 4 waves owns a tile of BM rows of A by BN rows of B
// and walks K in stages of 128. A stage's packed codes and scale words go
// straight from global memory into LDS (copies that need no register), in a
// ring of NS stages; each wave reads the packed codes from LDS and decodes its
// own fragments (one conversion and one packed multiply per two values), so LDS
// holds and moves 4 bits per value, not 16.
//   LDS rows are 64 bytes (128 codes). 16-byte piece c of row r lies at piece
// c ^ ((r / 4) % 4): any 16 consecutive rows' pieces c fall on all banks.
//   Scale words (4 scales: 64 k of one row) lie as in the 128x4 blocked layout,
// word (r, half) at half * tile + (r % 32) * 16 + (r / 32) * 4, so one read
// gives a lane the words of its row in up to four 32-row fragments. Blocked or
// plain, rows in order or gathered: the address of each word is computed once
// per workgroup and steps by a constant.
//   MFMA 32x32x16: lane i holds row i % 32; lanes 0..31 take the stage's first
// 64 k, lanes 32..63 the other 64 (the order of k inside a stage is free as
// long as A and B agree). Rows of B are the instruction's rows, rows of A its
// columns, so that a lane's results are neighbours in m of its neighbours'.
//   K can be split over workgroups: float32 partial sums in the workspace, the
// last workgroup of a tile (by ticket) adds them in the order of the slices.
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

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr int kStageK = 128;                    // k per stage
constexpr int kMaxExperts = 1024;
constexpr int kMaxTickets = 16384;              // tiles of a split product
constexpr int64_t kTicketBytes = kMaxTickets * 4;
constexpr int64_t kMaxPartialBytes = INT64_C(64) << 20;
constexpr int kMaxSplits = 16;
constexpr int64_t kMaxGrid = 0xFFFFFF;          // workgroups of 256 threads in 2^32 work items

// what copies of k past the end read instead
__device__ const uint4_t g_zeros[4] = {};

// ------------------------------------------------------------------ copies to LDS

// 16 or 4 bytes per lane from global memory into LDS at dst + lane * 16 (lane
// * 4). The compiler does not count them: the kernel waits for them itself.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __attribute__((always_inline)) inline void copy16(const void *src, uint32_t dst)
{
    asm volatile("s_mov_b32 m0, %1\n\tglobal_load_lds_dwordx4 %0, off" : : "v"(src), "s"(dst) : "memory", "m0");
}
__device__ __attribute__((always_inline)) inline void copy4(const void *src, uint32_t dst)
{
    asm volatile("s_mov_b32 m0, %1\n\tglobal_load_lds_dword %0, off" : : "v"(src), "s"(dst) : "memory", "m0");
}
#pragma clang diagnostic pop

// s_waitcnt vmcnt(N), other counters unconstrained
template <int N>
__device__ __attribute__((always_inline)) inline void wait_copies()
{
    static_assert(N >= 0 && N < 64, "vmcnt holds 0..63");
    __builtin_amdgcn_s_waitcnt((0x0F70 & ~0xC00F) | (N & 15) | ((N >> 4) << 14));
}

__device__ __attribute__((always_inline)) inline void barrier()
{
    asm volatile("" : : : "memory");
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

// ------------------------------------------------------------------ the kernel

// FM x FN fragments of 32 x 32 per wave, WM x WN waves, NS stages in the ring.
template <int FM, int FN, int WM, int WN, int NS>
struct Tile {
    static_assert(WM * WN == kWaves);
    static constexpr int kFM = FM, kFN = FN, kWM = WM, kWN = WN, kNS = NS;
    static constexpr int BM = 32 * FM * WM, BN = 32 * FN * WN;
    // words per line of a scale tile: 32-row groups that share a line
    static constexpr int LA = BM >= 128 ? 4 : BM / 32, LB = BN >= 128 ? 4 : BN / 32;
    static constexpr int kCodesA = BM * 64, kCodesB = BN * 64;
    static constexpr int kStage = kCodesA + kCodesB + BM * 8 + BN * 8;
    static constexpr int kOffB = kCodesA, kOffSA = kCodesA + kCodesB, kOffSB = kOffSA + BM * 8;
    // wave copies per stage: codes in 1 KiB, scale words in 256 bytes
    static constexpr int TA = kCodesA / 1024, TB = kCodesB / 1024, TSA = BM * 8 / 256, TSB = BN * 8 / 256;
    static constexpr int kLds = NS * kStage;
    static_assert(TA % kWaves == 0 && TSA % kWaves == 0);
    static_assert(TB % kWaves == 0 || TB < kWaves);
    static_assert(TSB % kWaves == 0 || TSB < kWaves);
    // copies that every wave makes, and those of some waves: B's codes by the
    // first TB waves, B's words by the last TSB
    static constexpr int kBase = TA / kWaves + TB / kWaves + TSA / kWaves + TSB / kWaves;
    static_assert((TB % kWaves) + (TSB % kWaves) <= kWaves, "at most one more copy per wave");
};

template <class T, bool EXPERTS, bool REGS>
__global__ __launch_bounds__(kThreads, 1) void nvfp4_gemm_kernel(GemmParams p)
{
    constexpr int FM = T::kFM, FN = T::kFN, NS = T::kNS, BM = T::BM, BN = T::BN;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    __shared__ int32_t s_slot[EXPERTS ? BN : 1];
    __shared__ uint32_t s_ticket;
    const int lane = threadIdx.x % 64;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int nkb = p.K / 16;

    // --- which tile
    uint32_t id = xcd_remap(blockIdx.x, gridDim.x);
    const int split = (int)(id % (uint32_t)p.splits);
    id /= (uint32_t)p.splits;
    const uint32_t tile = id;
    int l = 0, m0, n0, count;                   // batch or expert, first rows, rows of B in the tile
    if constexpr (EXPERTS) {
        m0 = (int)(id % (uint32_t)p.tiles_m) * BM;
        int want = (int)(id / (uint32_t)p.tiles_m);
        // the expert whose list holds tile `want` of all lists' tiles: 64 experts at a time
        int found = -1;
        for (int e0 = 0; e0 < p.L; e0 += 64) {
            const int e = e0 + lane;
            int from = 0, n = 0;
            if (e < p.L) {
                from = min(max(p.offsets[e], 0), p.N);
                n = max(min(max(p.offsets[e + 1], 0), p.N) - from, 0);
            }
            const int tiles = (n + BN - 1) / BN;
            int upto = tiles;                   // inclusive sum over the lanes
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int v = __shfl_up(upto, d);
                upto += lane >= d ? v : 0;
            }
            const uint64_t past = __ballot(upto > want);
            if (past) {
                const int src = __ffsll((unsigned long long)past) - 1;
                const int in_list = want - (__shfl(upto, src) - __shfl(tiles, src));
                found = e0 + src;
                n0 = __shfl(from, src) + in_list * BN;
                count = min(BN, __shfl(n, src) - in_list * BN);
                break;
            }
            want -= __shfl(upto, 63);
        }
        if (found < 0)
            return;                             // past the last tile (the whole workgroup)
        l = __builtin_amdgcn_readfirstlane(found);
        n0 = __builtin_amdgcn_readfirstlane(n0);
        count = __builtin_amdgcn_readfirstlane(count);
        for (int i = threadIdx.x; i < BN; i += kThreads) {
            const int s = i < count ? p.order[n0 + i] : -1;
            s_slot[i] = s >= 0 && s < p.N ? s : -1;
        }
        __syncthreads();
    } else {
        // bands of 8 tiles along n, so that one XCD's tiles share rows of both
        const uint32_t per = (uint32_t)p.tiles_m * (uint32_t)p.tiles_n;
        l = (int)(id / per);
        id %= per;
        const uint32_t band = id / ((uint32_t)p.tiles_m * 8u);
        id -= band * (uint32_t)p.tiles_m * 8u;
        const uint32_t wide = min(8u, (uint32_t)p.tiles_n - band * 8u);
        m0 = (int)(id / wide) * BM;
        n0 = (int)(band * 8u + id % wide) * BN;
        count = min(BN, p.N - n0);
    }
    const uint8_t *A = p.a + (int64_t)l * p.M * (p.K / 2), *SA = p.sfa + l * p.sfa_batch;
    const uint8_t *B = p.b, *SB = p.sfb;
    if constexpr (!EXPERTS) {
        B += (int64_t)l * p.N * (p.K / 2);
        SB += l * p.sfb_batch;
    }
    auto row_b = [&](int i) -> int {            // row of B of the tile's row i (a valid one for any i)
        if constexpr (EXPERTS)
            return max(s_slot[i], 0) / p.slots_per_row;
        else
            return min(n0 + i, p.N - 1);
    };

    // --- this wave's copies: source addresses of the first stage
    const int first = split * p.stages_per_split;
    const int stages = min(p.stages_per_split, p.stages - first);
    constexpr int CA = T::TA / kWaves, CB = (T::TB + kWaves - 1) / kWaves;
    constexpr int CSA = T::TSA / kWaves, CSB = (T::TSB + kWaves - 1) / kWaves;
    const bool has_b = T::TB % kWaves == 0 || wave < T::TB;
    const int wave_sb = T::TSB % kWaves == 0 ? wave : wave - (kWaves - T::TSB);      // B's words: the last waves
    const bool has_sb = wave_sb >= 0;
    const uint8_t *pa[CA], *pb[CB], *psa[CSA], *psb[CSB];
    // lane's 16 bytes of a 1 KiB copy: row lane / 4 of 16, piece swizzled back
    const int piece = (lane % 4) ^ ((lane / 16) % 4);
#pragma unroll
    for (int i = 0; i < CA; ++i) {
        const int r = (wave + kWaves * i) * 16 + lane / 4;
        pa[i] = A + (int64_t)min(m0 + r, p.M - 1) * (p.K / 2) + (int64_t)first * 64 + piece * 16;
    }
#pragma unroll
    for (int i = 0; i < CB; ++i) {
        const int r = has_b ? (wave + kWaves * i) * 16 + lane / 4 : 0;
        pb[i] = B + (int64_t)row_b(r) * (p.K / 2) + (int64_t)first * 64 + piece * 16;
    }
    // word w of a stage's scale words: block of 32 * LW rows, half, line, word
    auto word_row = [](int w, int LW) { return w / (LW * 64) * (LW * 32) + (w % LW) * 32 + (w / LW) % 32; };
    auto word_half = [](int w, int LW) { return (w / (LW * 32)) % 2; };
    const int64_t step_words = p.blocked ? 1024 : 8;
    const int my_half_a = word_half(wave * 64 + lane, T::LA);
    const int my_half_b = word_half(max(wave_sb, 0) * 64 + lane, T::LB);
#pragma unroll
    for (int i = 0; i < CSA; ++i) {
        const int w = (wave + kWaves * i) * 64 + lane;
        psa[i] = SA + scale_word_at(p.blocked, min(m0 + word_row(w, T::LA), p.M - 1), my_half_a, nkb) + first * step_words;
    }
#pragma unroll
    for (int i = 0; i < CSB; ++i) {
        const int w = (max(wave_sb, 0) + kWaves * i) * 64 + lane;
        psb[i] = SB + scale_word_at(p.blocked, row_b(word_row(w, T::LB)), my_half_b, nkb) + first * step_words;
    }
    const uint32_t lds_base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds;

    uint32_t regs_a[CSA], regs_b[CSB];
    // issues the copies of stage `st` (of all K) into ring slot `slot`
    auto issue = [&](int st, int slot) {
        const uint32_t base = lds_base + slot * T::kStage;
        const bool ragged = (st + 1) * kStageK > p.K;
        const int k_piece = st * kStageK + piece * 32;
        const uint8_t *zero = (const uint8_t *)g_zeros;
        if constexpr (REGS) {
            // plain scales of 2-byte aligned rows: two 2-byte loads per word, written to LDS after the stage's work
            const int ka = st * kStageK + my_half_a * 64, kb = st * kStageK + my_half_b * 64;
#pragma unroll
            for (int i = 0; i < CSA; ++i) {
                const uint16_t *q = (const uint16_t *)psa[i];
                regs_a[i] = (ka < p.K ? q[0] : 0u) | (ka + 32 < p.K ? (uint32_t)q[1] << 16 : 0u);
                psa[i] += step_words;
            }
#pragma unroll
            for (int i = 0; i < CSB; ++i) {
                const uint16_t *q = (const uint16_t *)psb[i];
                regs_b[i] = has_sb ? (kb < p.K ? q[0] : 0u) | (kb + 32 < p.K ? (uint32_t)q[1] << 16 : 0u) : 0u;
                psb[i] += step_words;
            }
        }
#pragma unroll
        for (int i = 0; i < CA; ++i) {
            copy16(ragged && k_piece >= p.K ? zero : pa[i], base + (wave + kWaves * i) * 1024);
            pa[i] += 64;
        }
        if (has_b) {
#pragma unroll
            for (int i = 0; i < CB; ++i) {
                copy16(ragged && k_piece >= p.K ? zero : pb[i], base + T::kOffB + (wave + kWaves * i) * 1024);
                pb[i] += 64;
            }
        }
        if constexpr (!REGS) {
            const bool past_a = ragged && st * kStageK + my_half_a * 64 >= p.K;
            const bool past_b = ragged && st * kStageK + my_half_b * 64 >= p.K;
#pragma unroll
            for (int i = 0; i < CSA; ++i) {
                copy4(past_a ? zero : psa[i], base + T::kOffSA + (wave + kWaves * i) * 256);
                psa[i] += step_words;
            }
            if (has_sb) {
#pragma unroll
                for (int i = 0; i < CSB; ++i) {
                    copy4(past_b ? zero : psb[i], base + T::kOffSB + (wave_sb + kWaves * i) * 256);
                    psb[i] += step_words;
                }
            }
        }
    };
    auto write_regs = [&](int slot) {
        if constexpr (REGS) {
            uint8_t *base = lds + slot * T::kStage;
#pragma unroll
            for (int i = 0; i < CSA; ++i)
                *(uint32_t *)(base + T::kOffSA + (wave + kWaves * i) * 256 + lane * 4) = regs_a[i];
            if (has_sb) {
#pragma unroll
                for (int i = 0; i < CSB; ++i)
                    *(uint32_t *)(base + T::kOffSB + (wave_sb + kWaves * i) * 256 + lane * 4) = regs_b[i];
            }
            asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
        }
    };

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
    const uint32_t words_b = T::kOffSB + (rb0 / (32 * T::LB)) * (T::LB * 256) + half * (T::LB * 128) +
                             l32 * (T::LB * 4) + (rb0 / 32 % T::LB) * 4;
    auto compute = [&](int st, int slot) {
        const uint8_t *base = lds + slot * T::kStage;
        uint32_t sa[FM], sb[FN];
        read_words<FM>(base + words_a, sa);
        read_words<FN>(base + words_b, sb);
        // scales past K's end may be anything (blocked padding): cleared
        const uint32_t valid = p.K - st * kStageK - half * 64 == 32 ? 0xFFFFu : ~0u;
#pragma unroll
        for (int i = 0; i < FM; ++i)
            sa[i] &= valid;
#pragma unroll
        for (int j = 0; j < FN; ++j)
            sb[j] &= valid;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const uint32_t pc = ((2 * half + s) ^ swz) * 16;
            uint4_t qa[FM], qb[FN];
            half2_t fa[FM], fb[FN];
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                qa[i] = *(const uint4_t *)(base + codes_a + i * 2048 + pc);
                fa[i] = s ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(sa[i], 1.0f, true)
                          : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(sa[i], 1.0f, false);
            }
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                qb[j] = *(const uint4_t *)(base + codes_b + j * 2048 + pc);
                fb[j] = s ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(sb[j], 1.0f, true)
                          : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(sb[j], 1.0f, false);
            }
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                half8_t va[FM], vb[FN];
#pragma unroll
                for (int i = 0; i < FM; ++i) {
                    const half2_t sc = d < 2 ? (half2_t){fa[i].x, fa[i].x} : (half2_t){fa[i].y, fa[i].y};
                    const uint32_t w[4] = {qa[i].x, qa[i].y, qa[i].z, qa[i].w};
                    va[i] = decode8(w[d], sc);
                }
#pragma unroll
                for (int j = 0; j < FN; ++j) {
                    const half2_t sc = d < 2 ? (half2_t){fb[j].x, fb[j].x} : (half2_t){fb[j].y, fb[j].y};
                    const uint32_t w[4] = {qb[j].x, qb[j].y, qb[j].z, qb[j].w};
                    vb[j] = decode8(w[d], sc);
                }
#pragma unroll
                for (int j = 0; j < FN; ++j)
#pragma unroll
                    for (int i = 0; i < FM; ++i)
                        acc[j][i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vb[j], va[i], acc[j][i], 0, 0, 0);
            }
        }
    };

#pragma unroll
    for (int s = 0; s < NS - 1; ++s) {
        if (s < stages) {
            issue(first + s, s);
            write_regs(s);
        }
    }
    const bool more = (T::TB % kWaves != 0 && has_b) || (!REGS && T::TSB % kWaves != 0 && has_sb);
    constexpr int kBase = REGS ? T::TA / kWaves + T::TB / kWaves : T::kBase;
    int slot = 0;
    int i = 0;
    for (; i + NS - 1 < stages; ++i) {
        // stage i has landed when only the NS - 2 younger stages' copies are out
        if (more)
            wait_copies<(NS - 2) * (kBase + 1)>();
        else
            wait_copies<(NS - 2) * kBase>();
        barrier();
        const int into = slot == 0 ? NS - 1 : slot - 1;
        issue(first + i + NS - 1, into);
        compute(first + i, slot);
        write_regs(into);
        slot = slot + 1 == NS ? 0 : slot + 1;
    }
    for (; i < stages; ++i) {
        wait_copies<0>();
        barrier();
        compute(first + i, slot);
        slot = slot + 1 == NS ? 0 : slot + 1;
    }

    // --- results. Register r of fragment (j, i): row of B rb0 + 32 j + 8 (r / 4) + 4 (lane / 32) + r % 4,
    // row of A ra0 + 32 i + lane % 32.
    const int64_t slot_base = EXPERTS ? 0 : (int64_t)l * p.N + n0;
    auto each = [&](auto f) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int n = rb0 + 32 * j + 8 * (r / 4) + 4 * half + r % 4;
                if (n >= count)
                    continue;
                int64_t row = slot_base + n;
                if constexpr (EXPERTS) {
                    row = s_slot[n];
                    if (row < 0)
                        continue;
                }
#pragma unroll
                for (int i = 0; i < FM; ++i) {
                    const int m = m0 + ra0 + 32 * i + l32;
                    if (m < p.M)
                        f(acc[j][i][r], row * p.M + m);
                }
            }
    };
    auto total_scale = [&]() {
        float scale = p.alpha;
        if (p.scale_a)
            scale *= p.scale_a[EXPERTS ? l : 0];
        if (p.scale_b)
            scale *= *p.scale_b;
        return scale;
    };
    if (p.splits > 1) {
        // partial sums: agent-scope stores (past this XCD's L2), then the ticket
        const int64_t one = (int64_t)(EXPERTS ? p.N : p.N * (int64_t)p.L) * p.M;
        each([&](float v, int64_t at) {
            __hip_atomic_store(&p.partials[split * one + at], v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        });
        asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
        barrier();
        if (threadIdx.x == 0)
            s_ticket = __hip_atomic_fetch_add(&p.tickets[tile], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        if (s_ticket != (uint32_t)p.splits - 1)
            return;
        if (threadIdx.x == 0)
            __hip_atomic_store(&p.tickets[tile], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        const float scale = total_scale();
        each([&](float, int64_t at) {
            float sum = 0.0f;
            for (int s = 0; s < p.splits; ++s)
                sum += __hip_atomic_load(&p.partials[s * one + at], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            store_value(p.c, at, sum * scale, p.dtype);
        });
        return;
    }
    const float scale = total_scale();
    each([&](float v, int64_t at) { store_value(p.c, at, v * scale, p.dtype); });
}

// ------------------------------------------------------------------ plans

typedef Tile<4, 4, 2, 2, 3> TileLarge;          // 256 x 256
typedef Tile<2, 2, 2, 2, 3> TileMid;            // 128 x 128
typedef Tile<2, 1, 2, 2, 4> TileNarrow;         // 128 x 64
typedef Tile<1, 1, 4, 1, 4> TileSkinny;         // 128 x 32

enum class Kind { Large, Mid, Narrow, Skinny };

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

// slices of K that bring the grid to about `want` workgroups, at least `least` stages each
void split_k(Plan &p, int64_t want, int64_t least, int64_t rows, int64_t M)
{
    int64_t s = std::min<int64_t>(want / std::max<int64_t>(p.tiles, 1), kMaxSplits);
    s = std::min<int64_t>(s, p.stages / least);
    s = std::min<int64_t>(s, kMaxPartialBytes / 4 / rows / M);
    if (s < 2 || p.tiles > kMaxTickets)
        s = 1;
    p.per_split = (int32_t)ceil_div(p.stages, s);
    p.splits = (int32_t)ceil_div(p.stages, p.per_split);
}

Plan dense_plan(int64_t M, int64_t N, int64_t K, int64_t L)
{
    Plan p{};
    p.stages = (int32_t)ceil_div(K, kStageK);
    auto tiles = [&](int bm, int bn) {
        p.bm = bm, p.bn = bn;
        p.tiles_m = ceil_div(M, bm), p.tiles_n = ceil_div(N, bn);
        p.tiles = p.tiles_m * p.tiles_n * L;
    };
    if (N <= 32) {
        p.kind = Kind::Skinny;
        tiles(TileSkinny::BM, TileSkinny::BN);
    } else if (N <= 64) {
        p.kind = Kind::Narrow;
        tiles(TileNarrow::BM, TileNarrow::BN);
    } else {
        p.kind = Kind::Large;
        tiles(TileLarge::BM, TileLarge::BN);
        if (p.tiles < 160) {
            p.kind = Kind::Mid;
            tiles(TileMid::BM, TileMid::BN);
        }
    }
    split_k(p, p.kind == Kind::Large ? 256 : 512, 4, N * L, M);
    return p;
}

Plan experts_plan(int64_t M, int64_t K, int64_t E, int64_t S)
{
    Plan p{};
    p.stages = (int32_t)ceil_div(K, kStageK);
    auto tiles = [&](int bm, int bn) {
        p.bm = bm, p.bn = bn;
        p.tiles_m = ceil_div(M, bm), p.tiles_n = std::min<int64_t>(S, S / bn + std::min(E, S));
        p.tiles = p.tiles_m * p.tiles_n;
    };
    const int64_t mean = ceil_div(S, E);
    if (mean <= 32) {
        p.kind = Kind::Skinny;
        tiles(TileSkinny::BM, TileSkinny::BN);
    } else if (mean <= 64) {
        p.kind = Kind::Narrow;
        tiles(TileNarrow::BM, TileNarrow::BN);
    } else {
        p.kind = Kind::Mid;
        tiles(TileMid::BM, TileMid::BN);
    }
    split_k(p, 512, 4, S, M);
    return p;
}

size_t plan_workspace(const Plan &p, int64_t rows, int64_t M)
{
    return p.splits > 1 ? (size_t)((kTicketBytes + p.splits * rows * M * 4 + 255) / 256 * 256) : 0;
}

bool known_type(int dtype) { return dtype == NVFP4_F16 || dtype == NVFP4_BF16 || dtype == NVFP4_F32; }
bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

template <class T, bool EXPERTS>
hipError_t launch(const GemmParams &p, int64_t grid, hipStream_t st)
{
    // plain scales whose rows start at odd multiples of 2 bytes go through registers
    const bool regs = !p.blocked && p.K % 64 != 0;
    auto go = [&](auto kern) {
        hipLaunchKernelGGL(kern, dim3((uint32_t)grid), dim3(kThreads), T::kLds, st, p);
        return hipGetLastError();
    };
    return regs ? go(nvfp4_gemm_kernel<T, EXPERTS, true>) : go(nvfp4_gemm_kernel<T, EXPERTS, false>);
}

template <bool EXPERTS>
nvfp4_status_t run(const Plan &plan, const GemmParams &p, hipStream_t st)
{
    const int64_t grid = plan.tiles * plan.splits;
    hipError_t e = hipSuccess;
    auto typed = [&](auto tile) {
        e = launch<decltype(tile), EXPERTS>(p, grid, st);
    };
    switch (plan.kind) {
    case Kind::Large: typed(TileLarge{}); break;
    case Kind::Mid: typed(TileMid{}); break;
    case Kind::Narrow: typed(TileNarrow{}); break;
    case Kind::Skinny: typed(TileSkinny{}); break;
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
        !gemm_shape(M, rows * slots_per_row, K, E))
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
