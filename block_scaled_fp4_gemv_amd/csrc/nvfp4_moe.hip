// Router and combine of a mixture of experts on MI355X (gfx950).
//
// Router. Picks are compared in float64 by definition. Almost always float32
// picks with a bound on their error tell the same, and much cheaper: the fast path
// gives 16 lanes to a token (64 for many experts or few tokens), 4 tokens to a
// wave, and turns each pick into one 32-bit key, its value in fixed point above
// the expert's index counted down, so that the largest key is the pick and ties
// go to the lower index. Each lane sorts its keys; a round takes the largest head of the lanes.
// Where two neighbours in the ranking (or the last pick and any that is left, or the
// last group kept and the first one left) are closer than the bound, unless they come
// from the same logit and bias, the wave repeats the token in float64. The weights are float64 in both. What
// bounds it: vector instructions, about 1270 per wave, 10 us at 4 per SIMD, after
// the logits have come (4 us) and the waves have started.
// 16384 tokens of 256 experts, 8 of them from 4 of 8 groups: float64 alone 58 us;
// float32 with a wave per token 44; four tokens per wave 23 with the experts of a
// lane 16 apart, 21 with neighbours: groups are then a few lanes, and loads wide.
//   Some routers take float64 for every token, those of a wave one after another:
// softmax weights that are not renormalised (they need the float64 sum over all
// experts), groups that are not the experts of 1, 2, 4, .. whole lanes, and as many
// picks as a token has lanes. 16384 tokens, softmax: 8 of 256 experts 17 us
// renormalised, 51 not; 6 of 64 11 and 32; 6 of 160 in 8 groups 56; 8 of 384 33, in
// 4 groups 105.
//   The one workgroup of up to 64 tokens has 128 registers a thread; its kernels
// spill 41 of them for 129 to 256 experts and more than 16 tokens, 27 for 257 to 512
// experts and 106 beyond. 64 tokens: 8 of 128 experts 8.5 us, of 256 14, of 384 29,
// of 1024 48.
// Lists. A stable counting sort of the slots by expert: counts per chunk of
// slots, then each chunk's places from the counts of the chunks before it. Every
// rank is counted, no atomic's order enters: the lists are the same each time.
// Bound by latency: 131072 slots of 256 experts 5 us and 9 (up to 64 tokens the
// router's one workgroup makes the lists too, in the same launch).
// Combine. One thread per 16 bytes of a token's columns, float32 sums.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "nvfp4_device.h"
#include "nvfp4_gemv.h"
#include "nvfp4_internal.h"

namespace {

constexpr int kRouteWaves = 4;
constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 64;
constexpr int kMaxGroups = 64;
constexpr int kListThreads = 1024;
static_assert(kListThreads >= kMaxExperts);
constexpr int kSmallThreads = 1024;
constexpr int64_t kTicketBytes = 256;
constexpr int64_t kMaxGrid = 0xFFFFFF;

template <int DT>
__device__ __attribute__((always_inline)) inline float load_value(const void *p, int64_t i)
{
    if constexpr (DT == NVFP4_F32)
        return ((const float *)p)[i];
    else if constexpr (DT == NVFP4_BF16)
        return __builtin_bit_cast(float, (uint32_t)((const uint16_t *)p)[i] << 16);
    else
        return (float)((const _Float16 *)p)[i];
}

// orders a wave's LDS accesses (no instruction: a wave's LDS accesses complete in order)
__device__ __attribute__((always_inline)) inline void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __attribute__((always_inline)) inline double wave_max(double v)
{
#pragma unroll
    for (int d = 32; d; d >>= 1)
        v = fmax(v, __shfl_xor(v, d));
    return v;
}
__device__ __attribute__((always_inline)) inline double wave_sum(double v)
{
#pragma unroll
    for (int d = 32; d; d >>= 1)
        v += __shfl_xor(v, d);
    return v;
}
__device__ __attribute__((always_inline)) inline int wave_min(int v)
{
#pragma unroll
    for (int d = 32; d; d >>= 1)
        v = min(v, __shfl_xor(v, d));
    return v;
}

struct RouteParams {
    int32_t T, E, k, score, n_group, topk_group, group_top, renormalize;
    float scaling;
};

constexpr uint64_t kAllLanes = ~0ull;

// ------------------------------------------------------------------ float64: the definition

// The k picks of a token from the wave's picks v[i] (expert lane + 64 i), largest
// first, ties to the lower expert: lane at + j gets the j-th in `id`.
template <int NL>
__device__ __attribute__((always_inline)) inline void pick_k(double (&v)[NL], int k, int lane, int at, int &id)
{
    const double none = -__builtin_inf();
    for (int j = 0; j < k; ++j) {
        double best = none;
        int e = kMaxExperts;
#pragma unroll
        for (int i = 0; i < NL; ++i)
            if (v[i] > best)
                best = v[i], e = lane + 64 * i;
        const double m = wave_max(best);
        if (!(m > none))
            return;
        e = __builtin_amdgcn_readfirstlane(wave_min(best == m ? e : kMaxExperts));
        if (lane == at + j)
            id = e;
#pragma unroll
        for (int i = 0; i < NL; ++i)
            v[i] = e == lane + 64 * i ? none : v[i];
    }
}

// Masks the picks outside of the best groups; `picks`: the wave's picks in LDS.
template <int NL>
__device__ __attribute__((always_inline)) inline void mask_groups(double (&pick)[NL], const double *picks,
                                                                  const RouteParams &p, int lane)
{
    const double none = -__builtin_inf();
    const int size = p.E / p.n_group;
    double value = none;
    if (lane < p.n_group) {
        double a = none, b = none;                              // the two largest
        for (int j = 0; j < size; ++j) {
            const double v = picks[lane * size + j];
            b = v > a ? a : (v > b ? v : b);
            a = v > a ? v : a;
        }
        value = p.group_top > 1 && b > none ? a + b : a;
    }
    uint64_t keep = 0;
    for (int j = 0; j < p.topk_group; ++j) {
        const double m = wave_max(value);
        if (!(m > none))
            break;                                              // the other groups have no expert left
        const int g = __ffsll((unsigned long long)__ballot(value == m)) - 1;
        keep |= 1ull << g;
        value = lane == g ? none : value;
    }
#pragma unroll
    for (int i = 0; i < NL; ++i)
        if (!(keep >> min((lane + 64 * i) / size, 63) & 1ull))
            pick[i] = none;
}

// Logits (masked and past the end: -inf) and biases of the experts l, l + STEP, ..
// Nothing branches but on `bias`: all loads are in flight together.
template <int DT, int N, int STEP>
__device__ __attribute__((always_inline)) inline void load_experts(const void *__restrict__ logits,
                                                                   const float *__restrict__ bias, int64_t t, int32_t E,
                                                                   int l, float (&x)[N], float (&b)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        x[i] = load_value<DT>(logits, t * E + min(l + STEP * i, E - 1));
    if (bias) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            b[i] = bias[min(l + STEP * i, E - 1)];
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            b[i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        x[i] = x[i] == x[i] && l + STEP * i < E ? x[i] : -__builtin_inff();
}

// The same of the experts l * N, l * N + 1, ..; whole rows (E = LPT * N) by 16-byte
// loads, at any address of the type's alignment.
template <int DT, int N, int LPT>
__device__ __attribute__((always_inline)) inline void load_run(const void *__restrict__ logits,
                                                               const float *__restrict__ bias, int64_t t, int32_t E,
                                                               int l, float (&x)[N], float (&b)[N])
{
    using Value = std::conditional_t<DT == NVFP4_F32, float, uint16_t>;
    if (E == LPT * N) {
        Value raw[N];
        __builtin_memcpy(raw, (const Value *)logits + t * E + l * N, sizeof raw);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (DT == NVFP4_F32)
                x[i] = raw[i];
            else if constexpr (DT == NVFP4_BF16)
                x[i] = __builtin_bit_cast(float, (uint32_t)raw[i] << 16);
            else
                x[i] = (float)__builtin_bit_cast(_Float16, raw[i]);
        }
        if (bias)
            __builtin_memcpy(b, bias + l * N, sizeof b);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            x[i] = load_value<DT>(logits, t * E + min(l * N + i, E - 1));
        if (bias) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                b[i] = bias[min(l * N + i, E - 1)];
        }
    }
    if (!bias) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            b[i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        x[i] = x[i] == x[i] && l * N + i < E ? x[i] : -__builtin_inff();
}

// One token by the wave: its picks in lanes at, at + 1, .. of *picked; returns
// the softmax's sum. Not inlined: it is rarely taken, and its registers would
// cost the fast path waves. `lds`: 64 * NL doubles.
template <int DT, int NL>
__device__ __attribute__((noinline)) double route_exact(const void *__restrict__ logits, const float *__restrict__ bias,
                                                        int64_t t, RouteParams p, int at, int *picked, double *lds)
{
    const double none = -__builtin_inf();
    const int lane = threadIdx.x % 64;
    float x[NL], b[NL];
    load_experts<DT, NL, 64>(logits, bias, t, p.E, lane, x, b);
    double pick[NL], top = none, score_sum = 1.0;
#pragma unroll
    for (int i = 0; i < NL; ++i)
        top = fmax(top, (double)x[i]);
    if (p.score == NVFP4_SCORE_SOFTMAX) {
        top = wave_max(top);
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            // +inf: those logits share, the others get nothing
            pick[i] = x[i] > none ? ((double)x[i] == top ? 1.0 : exp((double)x[i] - top)) : 0.0;
            sum += pick[i];
        }
        score_sum = wave_sum(sum);
#pragma unroll
        for (int i = 0; i < NL; ++i)
            pick[i] = score_sum > 0.0 ? pick[i] / score_sum : 0.0;
    } else {
#pragma unroll
        for (int i = 0; i < NL; ++i)
            pick[i] = 1.0 / (1.0 + exp(-(double)x[i]));
    }
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        const double v = pick[i] + (double)b[i];
        pick[i] = x[i] > none && v == v ? v : none;
    }
    if (p.n_group > 1) {
#pragma unroll
        for (int i = 0; i < NL; ++i)
            lds[lane + 64 * i] = pick[i];
        wave_sync();
        mask_groups<NL>(pick, lds, p, lane);
        wave_sync();
    }
    int id = -1;
    pick_k<NL>(pick, p.k, lane, at, id);
    *picked = id;
    return score_sum;
}

// ------------------------------------------------------------------ float32 with a bound

// The value of another lane of the same 16; one instruction with the operation that takes it.
template <int CTRL>
__device__ __attribute__((always_inline)) inline uint32_t from_lane(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}

// Largest value over the token's LPT lanes, in all of them.
template <int LPT>
__device__ __attribute__((always_inline)) inline uint32_t token_max(uint32_t v)
{
    v = max(v, from_lane<0x128>(v));                            // row_ror:8, 4, 2, 1
    v = max(v, from_lane<0x124>(v));
    v = max(v, from_lane<0x122>(v));
    v = max(v, from_lane<0x121>(v));
    if constexpr (LPT == 64) {
        v = max(max((uint32_t)__builtin_amdgcn_readlane((int)v, 0), (uint32_t)__builtin_amdgcn_readlane((int)v, 16)),
                max((uint32_t)__builtin_amdgcn_readlane((int)v, 32), (uint32_t)__builtin_amdgcn_readlane((int)v, 48)));
    }
    return v;
}
template <int LPT>
__device__ __attribute__((always_inline)) inline float token_max(float v)                  // v >= 0
{
    return __builtin_bit_cast(float, token_max<LPT>(__builtin_bit_cast(uint32_t, v)));
}
template <int LPT>
__device__ __attribute__((always_inline)) inline float token_sum(float v)
{
    v += as_f32((int)from_lane<0x128>((uint32_t)as_i32(v)));
    v += as_f32((int)from_lane<0x124>((uint32_t)as_i32(v)));
    v += as_f32((int)from_lane<0x122>((uint32_t)as_i32(v)));
    v += as_f32((int)from_lane<0x121>((uint32_t)as_i32(v)));
    if constexpr (LPT == 64) {
        v += __shfl_xor(v, 16);
        v += __shfl_xor(v, 32);
    }
    return v;
}
// The two largest of two sets.
__device__ __attribute__((always_inline)) inline void join_two(uint32_t &a, uint32_t &b, uint32_t oa, uint32_t ob)
{
    b = max(min(a, oa), max(b, ob));
    a = max(a, oa);
}
// Descending, by merging (Batcher's odd-even merge sort); N a power of two.
template <int N>
__device__ __attribute__((always_inline)) inline void sort_down(uint32_t (&v)[N])
{
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int k = p; k >= 1; k /= 2)
#pragma unroll
            for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (j + i + k < N && (j + i) / (2 * p) == (j + i + k) / (2 * p)) {
                        const uint32_t a = v[j + i], b = v[j + i + k];
                        v[j + i] = max(a, b);
                        v[j + i + k] = min(a, b);
                    }
}

// The wave's 64 / LPT tokens t, t + 1, .. (those below t_end): lane j of a
// token's lanes gets its j-th pick, or -1; `top` its largest logit. Returns
// whether the token's picks are certain (the same in its lanes).
// Expert of key i of lane l: l * NL + i. Groups have to be the experts of 1, 2, 4,
// .. lanes.
template <int DT, int LPT, int NL>
__device__ __attribute__((always_inline)) inline bool route_fast(const void *__restrict__ logits,
                                                                 const float *__restrict__ bias, const RouteParams &p,
                                                                 int64_t t, bool here, int l, int &id, float &top)
{
    constexpr int IB = LPT * NL <= 64 ? 6 : LPT * NL <= 128 ? 7 : LPT * NL <= 256 ? 8 : LPT * NL <= 512 ? 9 : 10;
    constexpr uint32_t kIndex = (1u << IB) - 1;
    constexpr uint32_t kGroup = LPT - 1;                        // a group's value stands above its index
    constexpr int GB = LPT == 16 ? 4 : 6;
    constexpr float kSteps = (float)((1u << (31 - IB)) - 16);   // steps for a pick of the token's largest size
    const float none = -__builtin_inff();
    float x[NL], b[NL], v[NL];
    top = none;
    load_run<DT, NL, LPT>(logits, bias, here ? t : 0, p.E, l, x, b);
#pragma unroll
    for (int i = 0; i < NL; ++i)
        top = fmaxf(top, x[i]);
    // the largest logit: by its order as an integer
    const uint32_t bits = __builtin_bit_cast(uint32_t, top);
    const uint32_t high = token_max<LPT>(bits >> 31 ? ~bits : bits | 0x80000000u);
    top = __builtin_bit_cast(float, high >> 31 ? high & 0x7FFFFFFFu : ~high);
    float score_top = 1.0f;
    if (p.score == NVFP4_SCORE_SOFTMAX) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            v[i] = __expf(x[i] - top);
            sum += v[i];
        }
        score_top = 1.0f / token_sum<LPT>(sum);                 // the largest score: exp(0) / sum
#pragma unroll
        for (int i = 0; i < NL; ++i)
            v[i] *= score_top;
    } else {
#pragma unroll
        for (int i = 0; i < NL; ++i)
            v[i] = __builtin_amdgcn_rcpf(1.0f + __expf(-x[i]));
    }
    float largest = 0.0f;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        const float pick = v[i] + b[i];
        v[i] = x[i] > none && pick > none ? pick : none;        // NaN too
        largest = v[i] > none ? fmaxf(largest, fabsf(v[i])) : largest;
    }
    largest = token_max<LPT>(largest);
    // exp(-d) is off by at most (d + 2) 2^-23 of itself, so a softmax numerator (d e^-d
    // <= 0.37) or a sigmoid by less than 2^-20 of the largest score. The softmax's sum
    // scales every score alike and matters beside a bias only: it is off by at most
    // (0.37 E + 16) 2^-23 of itself. A pick's own rounding is 2^-24 of the largest, its
    // way to a key two steps of 2^-23 and one of the key's.
    const float part = p.score == NVFP4_SCORE_SOFTMAX && bias ? (p.E > 64 ? 0x1p-13f : 0x1p-17f) : 0x1p-20f;
    const float margin = 2.0f * (score_top / largest * part + 0x1p-22f) * kSteps + 3.0f;
    bool sure = largest > 0.0f && largest < __builtin_inff() && margin < 0.25f * kSteps;
    const uint32_t close = sure ? (uint32_t)margin : 0u;
    const float scale = kSteps / largest;
    uint32_t key[NL];
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        const uint32_t step = (uint32_t)(fmaf(v[i], scale, kSteps) + 1.0f);
        key[i] = v[i] > none ? step << IB | (kIndex - (uint32_t)(l * NL + i)) : 0u;
    }
    if (p.n_group > 1) {
        const int lanes = p.E / p.n_group / NL, g = l / lanes;  // lanes per group, this lane's group
        uint32_t a = 0u, c = 0u;                                // the group's two largest
#pragma unroll
        for (int i = 0; i < NL; ++i)
            join_two(a, c, key[i], 0u);
        // each step joins neighbouring halves, whose lanes agree among themselves
        if (lanes > 1)
            join_two(a, c, from_lane<0xB1>(a), from_lane<0xB1>(c));         // quad_perm [1, 0, 3, 2]
        if (lanes > 2)
            join_two(a, c, from_lane<0x4E>(a), from_lane<0x4E>(c));         // quad_perm [2, 3, 0, 1]
        if (lanes > 4)
            join_two(a, c, from_lane<0x141>(a), from_lane<0x141>(c));       // row_half_mirror
        if (lanes > 8)
            join_two(a, c, from_lane<0x140>(a), from_lane<0x140>(c));       // row_mirror
        if (lanes > 16)
            join_two(a, c, (uint32_t)__shfl_xor((int)a, 16), (uint32_t)__shfl_xor((int)c, 16));
        // the group's first lane: its value above its index; a second value that is
        // missing counts as 0
        const uint32_t two = (a >> IB) + (p.group_top > 1 ? (c ? c >> IB : (uint32_t)kSteps + 1u) : 0u);
        uint32_t mine = a && l % lanes == 0 ? two << GB | (kGroup - (uint32_t)g) : 0u;
        uint64_t keep = 0;
        uint32_t last = 0u;
        for (int j = 0; j <= p.topk_group; ++j) {
            const uint32_t m = token_max<LPT>(mine);
            if (j == p.topk_group) {
                sure = sure && !(m && (last >> GB) - (m >> GB) <= 2u * close);
            } else {
                keep |= m ? 1ull << (kGroup - (m & kGroup)) : 0ull;
                mine = mine == m ? 0u : mine;
                last = m;
            }
        }
        const bool kept = keep >> g & 1ull;
#pragma unroll
        for (int i = 0; i < NL; ++i)
            key[i] = kept ? key[i] : 0u;
    }
    sort_down<NL>(key);
    uint32_t got = 0u;
    for (int j = 0; j <= p.k; ++j) {                            // one more: the first that is left out
        const uint32_t m = token_max<LPT>(key[0]);
        got = l == j ? m : got;
        const bool pop = key[0] == m;
#pragma unroll
        for (int i = 0; i + 1 < NL; ++i) {
            uint32_t next = key[i + 1];
            asm("" : "+v"(next));                               // a choice of values, not of an index into key
            key[i] = pop ? next : key[i];
        }
        key[NL - 1] = pop ? 0u : key[NL - 1];
    }
    id = got ? (int)(kIndex - (got & kIndex)) : -1;
    // Neighbours in the ranking closer than the bound: from the same logit and bias? Of
    // those that are left, all within the bound of the last pick have to be its equals:
    // the first one may be, and stand before a larger one by its index.
    const uint32_t next = LPT == 16 ? from_lane<0x101>(got) : (uint32_t)__shfl_down((int)got, 1);      // row_shl:1
    bool doubt = here && l < p.k && got && next && (got >> IB) - (next >> IB) <= close;
    if (__ballot(doubt)) {
        auto differs = [&](uint32_t a, uint32_t b) {
            const int ea = (int)(kIndex - (a & kIndex)), eb = (int)(kIndex - (b & kIndex));
            return load_value<DT>(logits, t * p.E + ea) != load_value<DT>(logits, t * p.E + eb) ||
                   (bias && bias[ea] != bias[eb]);
        };
        doubt = doubt && differs(got, next);
        const uint32_t last = token_max<LPT>(here && l == p.k - 1 ? got : 0u);
        auto left = [&] { return last && key[0] && (last >> IB) - (key[0] >> IB) <= close; };
        while (__ballot(left())) {                              // a lane's keys fall
            if (left())
                doubt = doubt || differs(last, key[0]);
#pragma unroll
            for (int i = 0; i + 1 < NL; ++i)
                key[i] = key[i + 1];
            key[NL - 1] = 0u;
        }
        const uint32_t any = token_max<LPT>(doubt ? 1u : 0u);
        sure = sure && any == 0u;
    }
    if (l >= p.k)
        id = -1;
    return sure;
}

// The tokens t .. t + 64 / LPT - 1 (below T) by one wave. NX: experts per lane of
// the float64 path. `lds`: 64 * NX doubles of the wave's own.
template <int DT, int LPT, int NL, int NX>
__device__ __attribute__((always_inline)) inline void route_tokens(const void *__restrict__ logits,
                                                                   const float *__restrict__ bias,
                                                                   int32_t *__restrict__ ids,
                                                                   float *__restrict__ weights, const RouteParams &p,
                                                                   int64_t t0, int lane, double *lds)
{
    const int l = lane % LPT;
    const int64_t t = t0 + lane / LPT;
    const bool here = t < p.T;
    int id = -1;
    float top = 0.0f;
    double sum = 1.0;
    bool sure = false;
    // the fast path's lanes hold one pick more than k
    const int size = p.E / p.n_group, lanes = size / NL;
    if (p.k < LPT && (p.n_group == 1 || (size % NL == 0 && (lanes & (lanes - 1)) == 0)))
        sure = route_fast<DT, LPT, NL>(logits, bias, p, t, here, l, id, top);
    else {
        top = -__builtin_inff();
        for (int e = l; e < p.E; e += LPT)
            top = fmaxf(top, load_value<DT>(logits, (here ? t : 0) * p.E + e));         // skips NaN
        for (int d = 1; d < LPT; d *= 2)
            top = fmaxf(top, __shfl_xor(top, d));
    }
    // softmax weights that are not renormalised need the float64 sum over all
    // experts, and infinite logits their own rule
    sure = sure && top < __builtin_inff() && (p.score == NVFP4_SCORE_SIGMOID || p.renormalize);
    uint64_t again = __ballot(here && !sure && l == 0);
    while (again) {
        const int at = __ffsll((unsigned long long)again) - 1;
        again &= again - 1;
        int got = -1;
        const double s = route_exact<DT, NX>(logits, bias, t0 + at / LPT, p, at, &got, lds);
        if (lane / LPT == at / LPT) {
            id = got;
            sum = s;
        }
    }
    double w = 0.0;
    if (here && id >= 0) {                                      // lanes without a token carry token 0's picks
        const float v = load_value<DT>(logits, t * p.E + id);
        if (p.score == NVFP4_SCORE_SIGMOID)
            w = 1.0 / (1.0 + exp(-(double)v));
        else                                                    // renormalised: the sum cancels
            w = (v == top ? 1.0 : exp((double)v - (double)top)) / (p.renormalize ? 1.0 : sum);
    }
    if (p.renormalize) {
        double total = w;
#pragma unroll
        for (int d = 1; d < LPT; d *= 2)
            total += __shfl_xor(total, d);
        w = total > 0.0 ? w / total : 0.0;
    }
    if (here && l < p.k) {
        ids[t * p.k + l] = id;
        weights[t * p.k + l] = (float)(w * (double)p.scaling);
    }
}

template <int DT, int LPT, int NL, int NX>
__global__ __launch_bounds__(64 * kRouteWaves) void nvfp4_route_kernel(const void *__restrict__ logits,
                                                                       const float *__restrict__ bias,
                                                                       int32_t *__restrict__ ids,
                                                                       float *__restrict__ weights, RouteParams p)
{
    __shared__ double lds[kRouteWaves][64 * NX];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int64_t t = ((int64_t)blockIdx.x * kRouteWaves + wave) * (64 / LPT);
    if (t < p.T)
        route_tokens<DT, LPT, NL, NX>(logits, bias, ids, weights, p, t, lane, lds[wave]);
}

// ------------------------------------------------------------------ lists

// Lanes of the wave with the same key (bits key bits wide).
__device__ __attribute__((always_inline)) inline uint64_t same_lanes(uint32_t key, int bits)
{
    uint64_t m = kAllLanes;
    for (int b = 0; b < bits; ++b) {
        const bool one = key >> b & 1u;
        const uint64_t v = __ballot(one);
        m &= one ? v : ~v;
    }
    return m;
}

// Inclusive sums over a workgroup's threads (THREADS of them, `part` holds one
// value per wave).
template <int THREADS>
__device__ __attribute__((always_inline)) inline int32_t sum_upto(int32_t v, int32_t *part)
{
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int32_t o = __shfl_up(v, d);
        v += lane >= d ? o : 0;
    }
    if (lane == 63)
        part[wave] = v;
    __syncthreads();
    int32_t before = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w)
        before += w < wave ? part[w] : 0;
    __syncthreads();
    return v + before;
}

// One workgroup counts a chunk of slots: counts[c][e].
__global__ __launch_bounds__(kListThreads) void nvfp4_count_kernel(const int32_t *__restrict__ ids,
                                                                   int32_t *__restrict__ counts, int32_t S, int32_t E,
                                                                   int32_t chunk)
{
    __shared__ int32_t n[kMaxExperts];
    for (int e = threadIdx.x; e < E; e += kListThreads)
        n[e] = 0;
    __syncthreads();
    const int32_t from = blockIdx.x * chunk, to = min(S, from + chunk);
    for (int32_t s = from + (int32_t)threadIdx.x; s < to; s += kListThreads) {
        const int32_t e = ids[s];
        if (e >= 0 && e < E)
            atomicAdd(&n[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kListThreads)
        counts[(int64_t)blockIdx.x * E + e] = n[e];
}

// A workgroup of THREADS places the slots [from, to) in order; base[e] is
// where expert e's slots of this chunk start. at: LDS [waves][E] (per wave).
template <int THREADS>
__device__ __attribute__((always_inline)) inline void place_slots(const int32_t *__restrict__ ids,
                                                                  int32_t *__restrict__ order, int32_t *at,
                                                                  const int32_t *base, int32_t from, int32_t to,
                                                                  int32_t E, int32_t bits)
{
    constexpr int W = THREADS / 64;
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    // each wave a run of whole groups of 64 slots
    const int32_t run = ((to - from + 64 * W - 1) / (64 * W)) * 64;
    const int32_t a = from + wave * run, z = min(to, a + run);
    int32_t *mine = at + wave * E;
    for (int e = threadIdx.x; e < W * E; e += THREADS)
        at[e] = 0;
    __syncthreads();
    for (int32_t s = a + lane; s < z; s += 64) {
        const int32_t e = ids[s];
        if (e >= 0 && e < E)
            atomicAdd(&mine[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += THREADS) {
        int32_t sum = base[e];
        for (int w = 0; w < W; ++w) {
            const int32_t v = at[w * E + e];
            at[w * E + e] = sum;
            sum += v;
        }
    }
    __syncthreads();
    for (int32_t s0 = a; s0 < z; s0 += 64) {
        const int32_t s = s0 + lane;
        int32_t e = s < z ? ids[s] : -1;
        const bool in = e >= 0 && e < E;
        e = in ? e : E;                                         // one key for those in no list
        const uint64_t same = same_lanes((uint32_t)e, bits);
        const int before = __popcll(same & ((1ull << lane) - 1ull));
        const int32_t first = in ? mine[e] : 0;
        wave_sync();
        if (in) {
            order[first + before] = s;
            if (before == 0)
                mine[e] = first + __popcll(same);
        }
        wave_sync();
    }
}

// Every workgroup sums the counts of all chunks (and of those before its own)
// for itself: one launch fewer than a kernel for the sums, and the counts come
// from L2. The last workgroup done with them (by ticket) clears them, as every
// call leaves its workspace's counters.
__global__ __launch_bounds__(kListThreads) void nvfp4_place_kernel(const int32_t *__restrict__ ids,
                                                                   int32_t *counts, uint32_t *ticket,
                                                                   int32_t *__restrict__ offsets,
                                                                   int32_t *__restrict__ order, int32_t S, int32_t E,
                                                                   int32_t chunk, int32_t nc, int32_t bits)
{
    __shared__ uint32_t taken;
    extern __shared__ int32_t list_lds[];                       // base[E], at[waves][E]
    __shared__ int32_t part[kListThreads / 64];
    __shared__ int32_t s_all[kListThreads], s_before[kListThreads];
    int32_t *base = list_lds, *at = list_lds + E;
    // kListThreads / width threads per expert, each every so many chunks
    int width = 64;
    while (width < E)
        width *= 2;
    const int e = threadIdx.x % width, share = threadIdx.x / width, shares = kListThreads / width;
    int32_t all = 0, before = 0;
    if (e < E) {
#pragma unroll 16
        for (int c = share; c < nc; c += shares) {
            const int32_t v = counts[(int64_t)c * E + e];
            all += v;
            before += c < (int)blockIdx.x ? v : 0;
        }
    }
    s_all[threadIdx.x] = all;
    s_before[threadIdx.x] = before;
    __syncthreads();
    all = before = 0;
    if (share == 0)
        for (int h = 0; h < shares; ++h) {
            all += s_all[h * width + e];
            before += s_before[h * width + e];
        }
    const int32_t upto = sum_upto<kListThreads>(all, part);
    if (share == 0 && e < E) {
        base[e] = upto - all + before;
        if (blockIdx.x == 0) {
            offsets[e + 1] = upto;
            if (e == 0)
                offsets[0] = 0;
        }
    }
    __syncthreads();
    // every thread's counts have arrived (the barriers above follow their sums)
    if (threadIdx.x == 0)
        taken = __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const int32_t from = blockIdx.x * chunk;
    place_slots<kListThreads>(ids, order, at, base, from, min(S, from + chunk), E, bits);
    if (taken != (uint32_t)nc - 1)                              // place_slots has barriers of its own
        return;
    for (int64_t i = threadIdx.x; i < (int64_t)nc * E; i += kListThreads)
        counts[i] = 0;
    if (threadIdx.x == 0)
        *ticket = 0u;
}

// Few tokens: the whole router in one workgroup of 16 waves.
template <int DT, int LPT, int NL, int NX>
__global__ __launch_bounds__(kSmallThreads) void nvfp4_route_small_kernel(
    const void *__restrict__ logits, const float *__restrict__ bias, int32_t *__restrict__ ids,
    float *__restrict__ weights, int32_t *__restrict__ offsets, int32_t *__restrict__ order, RouteParams p, int32_t bits)
{
    extern __shared__ int32_t list_lds[];                       // route: the waves' picks; lists: base[E], at[waves][E]
    __shared__ int32_t part[kSmallThreads / 64];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    double *picks = (double *)list_lds + wave * (64 * NX);
    for (int t = wave * (64 / LPT); t < p.T; t += kSmallThreads / LPT)
        route_tokens<DT, LPT, NL, NX>(logits, bias, ids, weights, p, t, lane, picks);
    __syncthreads();                                            // this workgroup's ids are in its reach
    int32_t *base = list_lds, *at = list_lds + p.E;
    const int e = threadIdx.x;
    const int32_t S = p.T * p.k;
    if (e < p.E)
        base[e] = 0;
    __syncthreads();
    for (int s = threadIdx.x; s < S; s += kSmallThreads)
        if (ids[s] >= 0)
            atomicAdd(&base[ids[s]], 1);
    __syncthreads();
    const int32_t n = e < p.E ? base[e] : 0;
    const int32_t upto = sum_upto<kSmallThreads>(n, part);
    if (e < p.E) {
        base[e] = upto - n;
        offsets[e + 1] = upto;
        if (e == 0)
            offsets[0] = 0;
    }
    place_slots<kSmallThreads>(ids, order, at, base, 0, S, p.E, bits);
}

// ------------------------------------------------------------------ combine

template <int DT>
struct Piece {                                                  // 16 bytes of columns
    static constexpr int kN = DT == NVFP4_F32 ? 4 : 8;
};

template <int DT>
__device__ __attribute__((always_inline)) inline float to_float(const uint32_t (&w)[4], int i)
{
    if constexpr (DT == NVFP4_F32)
        return __builtin_bit_cast(float, w[i]);
    else if constexpr (DT == NVFP4_BF16)
        return __builtin_bit_cast(float, i % 2 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    else
        return i % 2 ? (float)as_h2(w[i / 2]).y : (float)as_h2(w[i / 2]).x;
}

template <int DT>
__device__ __attribute__((always_inline)) inline uint32_t value_bits(float v)
{
    if constexpr (DT == NVFP4_F32)
        return __builtin_bit_cast(uint32_t, v);
    else if constexpr (DT == NVFP4_BF16)
        return bf16_bits(v);
    else
        return f16_bits(v);
}

// One thread per 16 bytes of a token's columns; the last piece of a row may be
// partial. Rows have their type's alignment only. Eight slots at a time: their
// ids and weights first, then all their values, so that the loads of a round
// wait for one another once and not per slot.
template <int DT>
__global__ __launch_bounds__(256) void nvfp4_combine_kernel(const uint8_t *__restrict__ y,
                                                            const int32_t *__restrict__ ids,
                                                            const float *__restrict__ weights,
                                                            uint8_t *__restrict__ out, int64_t pieces, int32_t k,
                                                            int32_t M, int32_t per_row)
{
    constexpr int N = Piece<DT>::kN, SZ = DT == NVFP4_F32 ? 4 : 2, R = 8;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= pieces)
        return;
    const int64_t t = pieces < INT32_MAX ? (int64_t)((uint32_t)i / (uint32_t)per_row) : i / per_row;
    const int32_t m = (int32_t)(i - t * per_row) * N;
    float sum[N];
#pragma unroll
    for (int c = 0; c < N; ++c)
        sum[c] = 0.0f;
    const bool whole = m + N <= M;
    const uint8_t *row = y + (t * k * M + m) * SZ;
    for (int32_t j0 = 0; j0 < k; j0 += R) {
        float w[R];
        uint32_t used = 0u, v[R][4];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const int64_t s = t * k + min(j0 + j, k - 1);
            w[j] = weights[s];
            used |= (uint32_t)(j0 + j < k && ids[s] >= 0) << j;
        }
#pragma unroll
        for (int j = 0; j < R; ++j) {
            v[j][0] = v[j][1] = v[j][2] = v[j][3] = 0u;
            if (!(used >> j & 1u))
                continue;
            const uint8_t *p = row + (int64_t)(j0 + j) * M * SZ;
            if (whole) {
                __builtin_memcpy(v[j], p, 16);
            } else if constexpr (SZ == 4) {
#pragma unroll
                for (int c = 0; c < 3; ++c)
                    if (c < M - m)
                        v[j][c] = ((const uint32_t *)p)[c];
            } else {
#pragma unroll
                for (int c = 0; c < 7; ++c)
                    if (c < M - m)
                        v[j][c / 2] |= (uint32_t)((const uint16_t *)p)[c] << (16 * (c % 2));
            }
        }
#pragma unroll
        for (int j = 0; j < R; ++j) {
            if (!(used >> j & 1u))
                continue;
#pragma unroll
            for (int c = 0; c < N; ++c)
                sum[c] = fmaf(w[j], to_float<DT>(v[j], c), sum[c]);
        }
    }
    uint8_t *o = out + (t * M + m) * SZ;
    if (whole) {
        uint32_t v[4];
        if constexpr (SZ == 4) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
                v[c] = value_bits<DT>(sum[c]);
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c)
                v[c] = value_bits<DT>(sum[2 * c]) | (value_bits<DT>(sum[2 * c + 1]) << 16);
        }
        __builtin_memcpy(o, v, 16);
    } else {
#pragma unroll
        for (int c = 0; c < N; ++c) {
            if (c >= M - m)
                break;
            if constexpr (SZ == 4)
                ((uint32_t *)o)[c] = value_bits<DT>(sum[c]);
            else
                ((uint16_t *)o)[c] = (uint16_t)value_bits<DT>(sum[c]);
        }
    }
}

// ------------------------------------------------------------------ host

bool known_type(int dtype) { return dtype == NVFP4_F16 || dtype == NVFP4_BF16 || dtype == NVFP4_F32; }
int64_t type_size(int dtype) { return dtype == NVFP4_F32 ? 4 : 2; }
bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

nvfp4_status_t finish()
{
    const hipError_t e = hipGetLastError();
    if (e == hipSuccess)
        return NVFP4_OK;
    nvfp4_record_hip_error((int)e);
    return NVFP4_ERR_HIP;
}

template <typename F>
void by_type(int dtype, F f)
{
    if (dtype == NVFP4_F16)
        f(std::integral_constant<int, NVFP4_F16>{});
    else if (dtype == NVFP4_BF16)
        f(std::integral_constant<int, NVFP4_BF16>{});
    else
        f(std::integral_constant<int, NVFP4_F32>{});
}

bool route_shape(int64_t T, int64_t E, int64_t k)
{
    return T >= 1 && E >= 1 && E <= kMaxExperts && k >= 1 && k <= E && k <= kMaxTopK && T <= (INT64_C(1) << 30) / k;
}

// Few tokens run in one workgroup: at most 4 tokens per wave, and LDS for the lists.
bool route_small(int64_t T, int64_t E, int64_t k) { return T <= 64 && T * k <= 2048 && E <= kSmallThreads; }

// slots per workgroup of the lists' kernels: at most kMaxChunks chunks, of at least 512
constexpr int64_t kMaxChunks = 128;
int64_t list_chunk(int64_t S) { return std::max<int64_t>(512, (S + kMaxChunks - 1) / kMaxChunks); }
static_assert(kTicketBytes + kMaxChunks * kMaxExperts * 4 <= NVFP4_WORKSPACE_MAX_BYTES);

} // namespace

extern "C" {

size_t nvfp4_moe_route_workspace_bytes(int64_t T, int64_t E, int64_t k)
{
    if (!route_shape(T, E, k) || route_small(T, E, k))
        return 0;
    const int64_t S = T * k, chunk = list_chunk(S);
    return (size_t)(kTicketBytes + (((S + chunk - 1) / chunk) * E * 4 + 255) / 256 * 256);
}

nvfp4_status_t nvfp4_moe_route(const void *logits, int dtype, const float *bias, int32_t *ids, float *weights,
                               int32_t *offsets, int32_t *order, int64_t T, int64_t E, int64_t k,
                               const nvfp4_routing_t *routing, void *workspace, size_t workspace_bytes, void *stream)
{
    if (!logits || !ids || !weights || !offsets || !order || !routing)
        return NVFP4_ERR_NULL_POINTER;
    if (!known_type(dtype))
        return NVFP4_ERR_INVALID_TYPE;
    if (!route_shape(T, E, k))
        return NVFP4_ERR_INVALID_SHAPE;
    const nvfp4_routing_t &r = *routing;
    if ((r.score != NVFP4_SCORE_SOFTMAX && r.score != NVFP4_SCORE_SIGMOID) || r.n_group < 1 ||
        r.n_group > kMaxGroups || E % r.n_group != 0 || r.topk_group < 1 || r.topk_group > r.n_group ||
        r.group_top < 1 || r.group_top > 2 || r.group_top > E / r.n_group || (r.renormalize != 0 && r.renormalize != 1))
        return NVFP4_ERR_INVALID_ROUTING;
    if (!std::isfinite(r.scaling))
        return NVFP4_ERR_INVALID_SCALE;
    if (!aligned(logits, type_size(dtype)) || (bias && !aligned(bias, 4)) || !aligned(ids, 4) || !aligned(weights, 4) ||
        !aligned(offsets, 4) || !aligned(order, 4))
        return NVFP4_ERR_MISALIGNED;
    const size_t need = nvfp4_moe_route_workspace_bytes(T, E, k);
    if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
        return NVFP4_ERR_WORKSPACE;
    // 16 lanes per token where they hold its picks and at most 16 experts each,
    // and where a wave per token would not do at once (a single token)
    const bool narrow = k < 16 && E <= 256 && T > kSmallThreads / 64;
    const int64_t per_wg = kRouteWaves * (narrow ? 4 : 1), grid = (T + per_wg - 1) / per_wg;
    if (grid > kMaxGrid)
        return NVFP4_ERR_INVALID_SHAPE;
    const hipStream_t st = (hipStream_t)stream;
    RouteParams p{(int32_t)T, (int32_t)E, (int32_t)k, r.score, r.n_group, r.topk_group, r.group_top, r.renormalize,
                  r.scaling};
    const int32_t S = (int32_t)(T * k);
    int32_t bits = 1;
    while ((E >> bits) != 0)
        ++bits;                                                 // E itself is a key too
    const bool small = route_small(T, E, k);
    by_type(dtype, [&](auto dt) {
        auto go = [&](auto lpt, auto nl, auto nx) {
            if (small) {
                const size_t lds = std::max<size_t>(kSmallThreads / 64 * 64 * nx() * 8, (1 + kSmallThreads / 64) * E * 4);
                hipLaunchKernelGGL((nvfp4_route_small_kernel<dt(), lpt(), nl(), nx()>), dim3(1), dim3(kSmallThreads), lds,
                                   st, logits, bias, ids, weights, offsets, order, p, bits);
            } else {
                hipLaunchKernelGGL((nvfp4_route_kernel<dt(), lpt(), nl(), nx()>), dim3((uint32_t)grid),
                                   dim3(64 * kRouteWaves), 0, st, logits, bias, ids, weights, p);
            }
        };
        auto n = [](auto v) { return v; };
#define NVFP4_N(v) n(std::integral_constant<int, v>{})
        if (narrow && E <= 64)
            go(NVFP4_N(16), NVFP4_N(4), NVFP4_N(1));
        else if (narrow && E <= 128)
            go(NVFP4_N(16), NVFP4_N(8), NVFP4_N(2));
        else if (narrow)
            go(NVFP4_N(16), NVFP4_N(16), NVFP4_N(4));
        else if (E <= 256)
            go(NVFP4_N(64), NVFP4_N(4), NVFP4_N(4));
        else if (E <= 512)
            go(NVFP4_N(64), NVFP4_N(8), NVFP4_N(8));
        else
            go(NVFP4_N(64), NVFP4_N(16), NVFP4_N(16));
#undef NVFP4_N
    });
    if (!small) {
        // The router does not count its picks as it goes. By atomics (10 us for the
        // lists against 5 + 9, 131072 slots) the counts would have to be zero before
        // the call, and partial sums of a product may stand there in a shared
        // workspace; counts per chunk in LDS, stored as this kernel stores them, would
        // need no zero and are not built.
        const int32_t chunk = (int32_t)list_chunk(S), nc = (S + chunk - 1) / chunk;
        int32_t *counts = (int32_t *)((uint8_t *)workspace + kTicketBytes);
        hipLaunchKernelGGL(nvfp4_count_kernel, dim3(nc), dim3(kListThreads), 0, st, (const int32_t *)ids, counts, S,
                           (int32_t)E, chunk);
        hipLaunchKernelGGL(nvfp4_place_kernel, dim3(nc), dim3(kListThreads), (1 + kListThreads / 64) * E * 4, st,
                           (const int32_t *)ids, counts, (uint32_t *)workspace, offsets, order, S, (int32_t)E, chunk, nc, bits);
    }
    return finish();
}

nvfp4_status_t nvfp4_moe_combine(const void *y, int dtype, const int32_t *ids, const float *weights, void *out,
                                 int64_t T, int64_t k, int64_t M, void *stream)
{
    if (!y || !ids || !weights || !out)
        return NVFP4_ERR_NULL_POINTER;
    if (!known_type(dtype))
        return NVFP4_ERR_INVALID_TYPE;
    if (T < 1 || k < 1 || M < 1 || k > kMaxTopK || T > (INT64_C(1) << 30) / k || M > (INT64_C(1) << 30))
        return NVFP4_ERR_INVALID_SHAPE;
    if (!aligned(y, type_size(dtype)) || !aligned(out, type_size(dtype)) || !aligned(ids, 4) || !aligned(weights, 4))
        return NVFP4_ERR_MISALIGNED;
    const int64_t n = dtype == NVFP4_F32 ? 4 : 8, per_row = (M + n - 1) / n, pieces = T * per_row;
    const int64_t grid = (pieces + 255) / 256;
    if (grid > kMaxGrid)
        return NVFP4_ERR_INVALID_SHAPE;
    by_type(dtype, [&](auto dt) {
        hipLaunchKernelGGL((nvfp4_combine_kernel<dt()>), dim3((uint32_t)grid), dim3(256), 0, (hipStream_t)stream,
                           (const uint8_t *)y, ids, weights, (uint8_t *)out, pieces, (int32_t)k, (int32_t)M,
                           (int32_t)per_row);
    });
    return finish();
}

} // extern "C"
