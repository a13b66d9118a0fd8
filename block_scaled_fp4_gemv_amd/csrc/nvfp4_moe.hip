// Router and combine of a mixture of experts on MI355X (gfx950).
//
// Router. One wave per token: lane i holds the experts i, i + 64, ... . The
// picks are the largest of the wave one after the other, ties to the lower index.
//   Picks are compared in float64 by definition. Almost always float32 scores
// with a bound on their error tell the same: the fast path takes the picks in
// float32 and gives up where two neighbours in the ranking (or the last group
// kept and the first one left) are closer than the bound, unless they are the
// same number computed from the same logit and bias. Then the wave repeats the
// token in float64. The weights are float64 in both.
// Lists. A stable counting sort of the slots by expert: counts per chunk of
// slots, then each chunk's places from the counts of the chunks before it. Every
// rank is counted, no atomic's order enters: the lists are the same each time.
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
constexpr int kSimds = 1024;                   // of the GPU: 256 CUs of 4
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

// Largest value over the wave, the same in every lane: rows of 16 lanes by
// shifts, then across the rows; the last lane holds the result.
template <int CTRL, int ROWS>
__device__ __attribute__((always_inline)) inline float max_step(float v)
{
    return fmaxf(v, as_f32(__builtin_amdgcn_update_dpp(as_i32(v), as_i32(v), CTRL, ROWS, 0xF, false)));
}
__device__ __attribute__((always_inline)) inline float wave_max(float v)
{
    v = max_step<0x111, 0xF>(v);                                // row_shr:1, 2, 4, 8
    v = max_step<0x112, 0xF>(v);
    v = max_step<0x114, 0xF>(v);
    v = max_step<0x118, 0xF>(v);
    v = max_step<0x142, 0xA>(v);                                // row_bcast:15, 31
    v = max_step<0x143, 0xC>(v);
    return as_f32(__builtin_amdgcn_readlane(as_i32(v), 63));
}

struct RouteParams {
    int32_t T, E, k, score, n_group, topk_group, group_top, renormalize;
    float scaling;
    uint64_t group_magic;                                       // ceil(2^32 / group size): e / size = e * magic >> 32
};

constexpr uint64_t kAllLanes = ~0ull;

// lowest value over the wave
__device__ __attribute__((always_inline)) inline int wave_min(int v)
{
#pragma unroll
    for (int d = 32; d; d >>= 1)
        v = min(v, __shfl_xor(v, d));
    return v;
}

// The k picks of a token from the wave's picks (float or double), largest first:
// lane at + j gets the j-th's expert in `id`; lanes past the last keep theirs.
// Each lane's picks are sorted first, so that a round looks at one per lane.
// `close(m, e, last, last_e)` sees each pick before it is taken, beside the one
// before it, and also the first that is left out; where it says false, so does this.
template <int NL, typename V, typename Close>
__device__ __attribute__((always_inline)) inline bool pick_k(V (&v)[NL], int k, int lane, int at, int &id, Close close)
{
    const V none = -(V)__builtin_inff();
    int of[NL];                                                 // v[i] is expert lane + 64 * of[i]
#pragma unroll
    for (int i = 0; i < NL; ++i)
        of[i] = i;
#pragma unroll
    for (int n = NL - 1; n > 0; --n)
#pragma unroll
        for (int i = 0; i < n; ++i) {                           // equal picks keep their order
            const bool swap = v[i + 1] > v[i];
            const V hi = swap ? v[i + 1] : v[i], lo = swap ? v[i] : v[i + 1];
            const int a = swap ? of[i + 1] : of[i], b = swap ? of[i] : of[i + 1];
            v[i] = hi, v[i + 1] = lo;
            of[i] = a, of[i + 1] = b;
        }
    V last = (V)__builtin_inff();
    int last_e = -1;
    for (int j = 0; j <= k; ++j) {                              // one more: the first that is left out
        const V m = wave_max(v[0]);
        if (!(m > none))
            return true;
        const uint64_t best = __ballot(v[0] == m);
        int e;
        if (best & (best - 1))                                  // the same pick in several lanes: the lowest expert
            e = __builtin_amdgcn_readfirstlane(wave_min(v[0] == m ? lane + 64 * of[0] : kMaxExperts));
        else {
            const int l = __ffsll((unsigned long long)best) - 1;
            e = l + 64 * __builtin_amdgcn_readlane(of[0], l);
        }
        if (!close(m, e, last, last_e))
            return false;
        if (j == k)
            return true;
        if (lane == at + j)
            id = e;
        if (lane == e % 64) {
#pragma unroll
            for (int i = 0; i + 1 < NL; ++i)
                v[i] = v[i + 1], of[i] = of[i + 1];
            v[NL - 1] = none;
        }
        last = m, last_e = e;
    }
    return true;
}

// Masks the picks outside of the best groups. `picks`: the wave's picks in LDS.
// Returns false where the border between kept and left groups is closer than `margin`.
template <int NL, typename V>
__device__ __attribute__((always_inline)) inline bool mask_groups(V (&pick)[NL], const V *picks, const RouteParams &p,
                                                                  int lane, V margin)
{
    const V none = -(V)__builtin_inff();
    const int size = p.E / p.n_group;
    // lanes per group: the largest power of two that gives every group as many
    int per = 1, shift = 0;
    while (2 * per * p.n_group <= 64 && per < size)
        per *= 2, ++shift;
    const int g = lane >> shift, sub = lane & (per - 1);
    V a = none, b = none;                                       // the two largest
    if (g < p.n_group)
        for (int j = sub; j < size; j += per) {
            const V v = picks[g * size + j];
            b = v > a ? a : (v > b ? v : b);
            a = v > a ? v : a;
        }
    for (int d = 1; d < per; d *= 2) {
        const V oa = __shfl_xor(a, d), ob = __shfl_xor(b, d);
        const V low = oa > a ? a : oa, high = ob > b ? ob : b;
        a = oa > a ? oa : a;
        b = low > high ? low : high;
    }
    V value = p.group_top > 1 && b > none ? a + b : a;
    if (g >= p.n_group || sub != 0)
        value = none;
    uint64_t keep = 0;
    V last = none;
    bool sure = true;
    for (int j = 0; j <= p.topk_group; ++j) {
        const V m = wave_max(value);
        if (!(m > none))
            break;                                              // groups without an expert left: nothing in them to mask
        if (j == p.topk_group) {
            sure = last - m > margin;
            break;
        }
        last = m;
        const int at = __ffsll((unsigned long long)__ballot(value == m)) - 1;
        keep |= 1ull << (at >> shift);
        if (lane == at)
            value = none;
    }
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        const uint32_t e = (uint32_t)(lane + 64 * i);
        const uint32_t of = min((uint32_t)((e * p.group_magic) >> 32), 63u);
        if (!(keep >> of & 1ull))
            pick[i] = none;
    }
    return sure;
}

// float32 path: x (masked: -inf), bias b -> the picks in lanes at, at + 1, ..
// False: not certain. `same(e, f)`: whether two experts have equal logits and biases.
template <int NL, typename Same>
__device__ __attribute__((always_inline)) inline bool route_fast(const float (&x)[NL], const float (&b)[NL],
                                                                 bool with_bias, float top, const RouteParams &p,
                                                                 int lane, int at, float *lds, int &id, Same same)
{
    const float none = -__builtin_inff();
    float pick[NL], largest = none;
    float score_top = 1.0f;
    if (p.score == NVFP4_SCORE_SOFTMAX) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            pick[i] = __expf(x[i] - top);
            sum += pick[i];
        }
#pragma unroll
        for (int d = 32; d; d >>= 1)
            sum += __shfl_xor(sum, d);
        score_top = 1.0f / sum;                                 // the largest score: exp(0) / sum
#pragma unroll
        for (int i = 0; i < NL; ++i)
            pick[i] *= score_top;
    } else {
#pragma unroll
        for (int i = 0; i < NL; ++i)
            pick[i] = __builtin_amdgcn_rcpf(1.0f + __expf(-x[i]));
    }
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        const float v = pick[i] + b[i];
        pick[i] = x[i] > none && v == v ? v : none;
        largest = pick[i] > none ? fmaxf(largest, fabsf(pick[i])) : largest;
    }
    // exp(-d) is off by at most (d + 2) 2^-23 of itself, so a softmax numerator (d e^-d
    // <= 0.37) or a sigmoid by less than 2^-20 of the largest score. The softmax's sum
    // scales every score alike and matters beside a bias only: it is off by at most
    // (0.37 E + 16) 2^-23 of itself. The pick's own rounding is 2^-24 of the pick.
    const float part = p.score == NVFP4_SCORE_SOFTMAX && with_bias ? (p.E > 64 ? 0x1p-13f : 0x1p-17f) : 0x1p-20f;
    const float margin = 2.0f * (score_top * part + wave_max(largest) * 0x1p-23f);
    if (!(margin < 1.0f))
        return false;                                           // infinite picks: float64 sorts them out
    if (p.n_group > 1) {
#pragma unroll
        for (int i = 0; i < NL; ++i)
            lds[lane + 64 * i] = pick[i];
        wave_sync();
        const bool sure = mask_groups<NL, float>(pick, lds, p, lane, 2.0f * margin);
        wave_sync();
        if (!sure)
            return false;
    }
    return pick_k<NL, float>(pick, p.k, lane, at, id, [&](float m, int e, float last, int last_e) {
        return last - m > margin || same(e, last_e);
    });
}

// An expert's logit and bias for lane `lane` of the i-th 64; masked and past the end: -inf.
template <int DT, int NL>
__device__ __attribute__((always_inline)) inline void load_token(const void *__restrict__ logits,
                                                                 const float *__restrict__ bias, int64_t t, int32_t E,
                                                                 int lane, float (&x)[NL], float (&b)[NL])
{
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        const int e = lane + 64 * i;
        const float v = e < E ? load_value<DT>(logits, t * E + e) : -__builtin_inff();
        b[i] = bias && e < E ? bias[e] : 0.0f;
        x[i] = v == v ? v : -__builtin_inff();
    }
}

// float64 path, the definition itself: the picks in lanes at, at + 1, .. of
// *picked; returns the softmax's sum. Not inlined: it is rarely taken, and its
// registers would cost the fast path waves. It loads the token again.
template <int DT, int NL>
__device__ __attribute__((noinline)) double route_exact(const void *__restrict__ logits, const float *__restrict__ bias,
                                                       int64_t t, RouteParams p, int at, int *picked, double *lds)
{
    const double none = -__builtin_inf();
    const int lane = threadIdx.x % 64;
    float x[NL], b[NL];
    load_token<DT, NL>(logits, bias, t, p.E, lane, x, b);
    double pick[NL], top = none, score_sum = 1.0;
#pragma unroll
    for (int i = 0; i < NL; ++i)
        top = fmax(top, (double)x[i]);
    if (p.score == NVFP4_SCORE_SOFTMAX) {
        top = wave_max(top);
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
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
        mask_groups<NL, double>(pick, lds, p, lane, 0.0);
        wave_sync();
    }
    int id = -1;
    pick_k<NL, double>(pick, p.k, lane, at, id, [](double, int, double, int) { return true; });
    *picked = id;
    return score_sum;
}

// Lanes that hold one token's picks: the power of two from k on.
__device__ __attribute__((always_inline)) inline int pick_lanes(int k)
{
    return k <= 1 ? 1 : 1 << (32 - __builtin_clz(k - 1));
}

// `n` tokens from t on by one wave (n * pick_lanes(k) <= 64): the picks of one
// after the other, then the float64 weights of all at once. `lds`: 64 * NL
// doubles of the wave's own.
template <int DT, int NL>
__device__ __attribute__((always_inline)) inline void route_tokens(const void *__restrict__ logits,
                                                                   const float *__restrict__ bias,
                                                                   int32_t *__restrict__ ids,
                                                                   float *__restrict__ weights, const RouteParams &p,
                                                                   int64_t t, int n, int lane, double *lds)
{
    const int width = pick_lanes(p.k), mine = lane / width;    // the token whose pick this lane holds
    int id = -1;
    float my_top = 0.0f;
    double my_sum = 1.0;
    for (int q = 0; q < n; ++q) {
        const int at = q * width;
        float x[NL], b[NL], top = -__builtin_inff();
        load_token<DT, NL>(logits, bias, t + q, p.E, lane, x, b);
#pragma unroll
        for (int i = 0; i < NL; ++i)
            top = fmaxf(top, x[i]);
        top = wave_max(top);
        // softmax weights that are not renormalised need the float64 sum over all
        // experts, and infinite logits their own rule
        const bool plain = top < __builtin_inff() && (p.score == NVFP4_SCORE_SIGMOID || p.renormalize);
        int got = -1;
        double sum = 1.0;
        auto same = [&](int e, int f) {
            const int64_t row = (t + q) * p.E;
            return f >= 0 && load_value<DT>(logits, row + e) == load_value<DT>(logits, row + f) &&
                   (!bias || bias[e] == bias[f]);
        };
        if (!plain || !route_fast<NL>(x, b, bias != nullptr, top, p, lane, at, (float *)lds, got, same))
            sum = route_exact<DT, NL>(logits, bias, t + q, p, at, &got, lds);
        if (mine == q) {
            id = got;
            my_top = top;
            my_sum = sum;
        }
    }
    const int64_t token = t + mine;
    double w = 0.0;
    if (id >= 0) {
        const float v = load_value<DT>(logits, token * p.E + id);
        if (p.score == NVFP4_SCORE_SIGMOID)
            w = 1.0 / (1.0 + exp(-(double)v));
        else                                                    // renormalised: the sum cancels
            w = (v == my_top ? 1.0 : exp((double)v - (double)my_top)) / (p.renormalize ? 1.0 : my_sum);
    }
    if (p.renormalize) {
        double total = w;
        for (int d = 1; d < width; d *= 2)
            total += __shfl_xor(total, d);
        w = total > 0.0 ? w / total : 0.0;
    }
    const int j = lane % width;
    if (mine < n && j < p.k) {
        ids[token * p.k + j] = id;
        weights[token * p.k + j] = (float)(w * (double)p.scaling);
    }
}

// per_wave tokens per wave.
template <int DT, int NL>
__global__ __launch_bounds__(64 * kRouteWaves) void nvfp4_route_kernel(const void *__restrict__ logits,
                                                                       const float *__restrict__ bias,
                                                                       int32_t *__restrict__ ids,
                                                                       float *__restrict__ weights, RouteParams p,
                                                                       int32_t per_wave)
{
    __shared__ double lds[kRouteWaves][64 * NL];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int64_t t = ((int64_t)blockIdx.x * kRouteWaves + wave) * per_wave;
    if (t < p.T)
        route_tokens<DT, NL>(logits, bias, ids, weights, p, t, (int)min((int64_t)per_wave, p.T - t), lane, lds[wave]);
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
template <int DT, int NL>
__global__ __launch_bounds__(kSmallThreads) void nvfp4_route_small_kernel(
    const void *__restrict__ logits, const float *__restrict__ bias, int32_t *__restrict__ ids,
    float *__restrict__ weights, int32_t *__restrict__ offsets, int32_t *__restrict__ order, RouteParams p, int32_t bits)
{
    extern __shared__ int32_t list_lds[];                       // route: the waves' picks; lists: base[E], at[waves][E]
    __shared__ int32_t part[kSmallThreads / 64];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    double *picks = (double *)list_lds + wave * (64 * NL);
    for (int t = wave; t < p.T; t += kSmallThreads / 64)
        route_tokens<DT, NL>(logits, bias, ids, weights, p, t, 1, lane, picks);
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

// slots per workgroup of the lists' kernels: at most 128 chunks of at least 512
int64_t list_chunk(int64_t S) { return std::max<int64_t>(512, (S + 127) / 128); }

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
    // tokens per wave: as many as its lanes hold picks for, but 4 waves per SIMD
    int64_t width = 1;
    while (width < k)
        width *= 2;
    const int64_t per_wave = std::max<int64_t>(1, std::min<int64_t>(64 / width, T / (4 * kSimds)));
    const int64_t per_wg = per_wave * kRouteWaves, grid = (T + per_wg - 1) / per_wg;
    if (grid > kMaxGrid)
        return NVFP4_ERR_INVALID_SHAPE;
    const hipStream_t st = (hipStream_t)stream;
    const int64_t size = E / r.n_group;
    RouteParams p{(int32_t)T, (int32_t)E, (int32_t)k, r.score, r.n_group, r.topk_group, r.group_top, r.renormalize,
                  r.scaling, (uint64_t)(((INT64_C(1) << 32) + size - 1) / size)};
    const int32_t S = (int32_t)(T * k);
    int32_t bits = 1;
    while ((E >> bits) != 0)
        ++bits;                                                 // E itself is a key too
    const bool small = route_small(T, E, k);
    by_type(dtype, [&](auto dt) {
        auto go = [&](auto nl) {
            if (small) {
                const size_t lds = std::max<size_t>(kSmallThreads / 64 * 64 * nl() * 8, (1 + kSmallThreads / 64) * E * 4);
                hipLaunchKernelGGL((nvfp4_route_small_kernel<dt(), nl()>), dim3(1), dim3(kSmallThreads), lds, st, logits,
                                   bias, ids, weights, offsets, order, p, bits);
            } else {
                hipLaunchKernelGGL((nvfp4_route_kernel<dt(), nl()>), dim3((uint32_t)grid), dim3(64 * kRouteWaves), 0, st,
                                   logits, bias, ids, weights, p, (int32_t)per_wave);
            }
        };
        if (E <= 64)
            go(std::integral_constant<int, 1>{});
        else if (E <= 128)
            go(std::integral_constant<int, 2>{});
        else if (E <= 256)
            go(std::integral_constant<int, 4>{});
        else if (E <= 512)
            go(std::integral_constant<int, 8>{});
        else
            go(std::integral_constant<int, 16>{});
    });
    if (!small) {
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
