// Router and combine of a mixture of experts on MI355X (gfx950).
//
// Router. One wave per token: lane i holds the experts i, i + 64, ... . Scores
// are float64 (64-bit exponentials cost less than a wrong pick: float32
// scores of neighbouring experts collide or swap at their last bits); the k
// picks are k argmaxima over the wave, ties to the lower index.
// Lists. A stable counting sort of the slots by expert in three launches:
// counts per chunk of slots, prefix sums, placement. Every rank is counted,
// no atomic's order enters, so the lists are the same each time.
// Combine. One thread per 8 (4 for float32) columns of a token, float32 sums.
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
constexpr int kChunkMin = 256;                 // slots a wave counts and places
constexpr int kScanThreads = 1024;
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
// largest value and its lowest index over the wave, in every lane
__device__ __attribute__((always_inline)) inline void wave_argmax(double &v, int &i)
{
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        const double ov = __shfl_xor(v, d);
        const int oi = __shfl_xor(i, d);
        if (ov > v || (ov == v && oi < i)) {
            v = ov;
            i = oi;
        }
    }
}

struct RouteParams {
    int32_t T, E, k, score, n_group, topk_group, group_top, renormalize;
    float scaling;
};

// NL experts per lane (E <= 64 * NL).
template <int DT, int NL>
__global__ __launch_bounds__(64 * kRouteWaves) void nvfp4_route_kernel(const void *__restrict__ logits,
                                                                       const float *__restrict__ bias,
                                                                       int32_t *__restrict__ ids,
                                                                       float *__restrict__ weights, RouteParams p)
{
    __shared__ double s_score[kRouteWaves][64 * NL];
    __shared__ double s_pick[kRouteWaves][64 * NL];
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
    if (t >= p.T)
        return;
    const double none = -__builtin_inf();
    double score[NL], pick[NL];
    double top = none;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        const int e = lane + 64 * i;
        const float x = e < p.E ? load_value<DT>(logits, t * p.E + e) : -__builtin_inff();
        score[i] = x == x ? (double)x : none;
        top = fmax(top, score[i]);
    }
    if (p.score == NVFP4_SCORE_SOFTMAX) {
        top = wave_max(top);
        double sum = 0.0;
        uint32_t masked = 0u;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            masked |= (uint32_t)(score[i] == none) << i;
            // +inf: those logits share, the others get nothing
            score[i] = (masked >> i & 1u) ? 0.0 : score[i] == top ? 1.0 : exp(score[i] - top);
            sum += score[i];
        }
        sum = wave_sum(sum);
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            score[i] = sum > 0.0 ? score[i] / sum : 0.0;
            pick[i] = (masked >> i & 1u) ? none : score[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const bool masked = score[i] == none;
            score[i] = masked ? 0.0 : 1.0 / (1.0 + exp(-score[i]));
            pick[i] = masked ? none : score[i];
        }
    }
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        const int e = lane + 64 * i;
        if (bias && e < p.E) {
            const double v = pick[i] + (double)bias[e];
            pick[i] = v == v ? v : none;
        }
        s_score[wave][e] = score[i];
        s_pick[wave][e] = pick[i];
    }
    wave_sync();
    if (p.n_group > 1) {
        const int size = p.E / p.n_group;
        double value = none;
        if (lane < p.n_group) {
            double a = none, b = none;                          // the two largest
            for (int j = 0; j < size; ++j) {
                const double v = s_pick[wave][lane * size + j];
                b = v > a ? a : fmax(b, v);
                a = fmax(a, v);
            }
            value = p.group_top > 1 && b > none ? a + b : a;
        }
        uint64_t keep = 0;
        for (int j = 0; j < p.topk_group; ++j) {
            const bool left = lane < p.n_group && !(keep >> lane & 1ull);
            double v = left ? value : none;
            int g = left ? lane : 64;
            wave_argmax(v, g);
            if (g < 64)
                keep |= 1ull << g;
        }
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const int g = min((lane + 64 * i) / size, 63);
            if (!(keep >> g & 1ull))
                pick[i] = none;
        }
    }
    int mine = -1;
    double w = 0.0;
    for (int j = 0; j < p.k; ++j) {
        double v = none;
        int e = kMaxExperts;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            if (pick[i] > v) {
                v = pick[i];
                e = lane + 64 * i;
            }
        }
        wave_argmax(v, e);
        if (e >= p.E)
            break;                                              // none left, in every lane
#pragma unroll
        for (int i = 0; i < NL; ++i)
            if (e == lane + 64 * i)
                pick[i] = none;
        if (lane == j) {
            mine = e;
            w = s_score[wave][e];
        }
    }
    if (p.renormalize) {
        const double sum = wave_sum(w);
        w = sum > 0.0 ? w / sum : 0.0;
    }
    if (lane < p.k) {
        ids[t * p.k + lane] = mine;
        weights[t * p.k + lane] = (float)(w * (double)p.scaling);
    }
}

// ------------------------------------------------------------------ lists

// One wave counts `chunk` slots: counts[c][e].
__global__ __launch_bounds__(64) void nvfp4_count_kernel(const int32_t *__restrict__ ids, int32_t *__restrict__ counts,
                                                         int32_t S, int32_t E, int32_t chunk)
{
    __shared__ int32_t n[kMaxExperts];
    const int lane = threadIdx.x;
    for (int e = lane; e < E; e += 64)
        n[e] = 0;
    wave_sync();
    const int32_t from = blockIdx.x * chunk, to = min(S, from + chunk);
    for (int32_t s = from + lane; s < to; s += 64) {
        const int32_t e = ids[s];
        if (e >= 0 && e < E)
            atomicAdd(&n[e], 1);
    }
    wave_sync();
    for (int e = lane; e < E; e += 64)
        counts[(int64_t)blockIdx.x * E + e] = n[e];
}

// Exclusive sums over the chunks of each expert (in place) and over the experts.
__global__ __launch_bounds__(kScanThreads) void nvfp4_scan_kernel(int32_t *__restrict__ counts,
                                                                  int32_t *__restrict__ offsets, int32_t nc,
                                                                  int32_t E)
{
    __shared__ int32_t total[kScanThreads];
    const int e = threadIdx.x;
    int32_t sum = 0;
    if (e < E)
        for (int c = 0; c < nc; ++c) {
            const int32_t v = counts[(int64_t)c * E + e];
            counts[(int64_t)c * E + e] = sum;
            sum += v;
        }
    total[e] = sum;
    __syncthreads();
    for (int d = 1; d < kScanThreads; d <<= 1) {
        const int32_t v = e >= d ? total[e - d] : 0;
        __syncthreads();
        total[e] += v;
        __syncthreads();
    }
    if (e < E)
        offsets[e + 1] = total[e];
    if (e == 0)
        offsets[0] = 0;
}

// Lanes of the wave with the same key (bits key bits wide).
__device__ inline uint64_t same_lanes(uint32_t key, int bits)
{
    uint64_t m = ~0ull;
    for (int b = 0; b < bits; ++b) {
        const bool one = key >> b & 1u;
        const uint64_t v = __ballot(one);
        m &= one ? v : ~v;
    }
    return m;
}

// One wave places its chunk's slots in order, and leaves its counts zero (the
// workspace may hold another call's counters there).
__global__ __launch_bounds__(64) void nvfp4_place_kernel(const int32_t *__restrict__ ids,
                                                         int32_t *__restrict__ counts,
                                                         const int32_t *__restrict__ offsets,
                                                         int32_t *__restrict__ order, int32_t S, int32_t E,
                                                         int32_t chunk, int32_t bits)
{
    __shared__ int32_t at[kMaxExperts + 1];
    const int lane = threadIdx.x;
    for (int e = lane; e < E; e += 64) {
        at[e] = counts[(int64_t)blockIdx.x * E + e] + offsets[e];
        counts[(int64_t)blockIdx.x * E + e] = 0;
    }
    wave_sync();
    const int32_t from = blockIdx.x * chunk, to = min(S, from + chunk);
    for (int32_t s0 = from; s0 < to; s0 += 64) {
        const int32_t s = s0 + lane;
        int32_t e = s < to ? ids[s] : -1;
        const bool in = e >= 0 && e < E;
        e = in ? e : E;                                         // one key for those in no list
        const uint64_t same = same_lanes((uint32_t)e, bits);
        const int before = __popcll(same & ((1ull << lane) - 1ull));
        const int32_t base = in ? at[e] : 0;
        wave_sync();
        if (in) {
            order[base + before] = s;
            if (before == 0)
                at[e] = base + __popcll(same);
        }
        wave_sync();
    }
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
// partial. Rows have their type's alignment only.
template <int DT>
__global__ __launch_bounds__(256) void nvfp4_combine_kernel(const uint8_t *__restrict__ y,
                                                            const int32_t *__restrict__ ids,
                                                            const float *__restrict__ weights,
                                                            uint8_t *__restrict__ out, int64_t pieces, int32_t k,
                                                            int32_t M, int32_t per_row)
{
    constexpr int N = Piece<DT>::kN, SZ = DT == NVFP4_F32 ? 4 : 2;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= pieces)
        return;
    const int64_t t = i / per_row;
    const int32_t m = (int32_t)(i - t * per_row) * N;
    float sum[N];
#pragma unroll
    for (int c = 0; c < N; ++c)
        sum[c] = 0.0f;
    const bool whole = m + N <= M;
    for (int32_t j = 0; j < k; ++j) {
        const int64_t s = t * k + j;
        if (ids[s] < 0)
            continue;
        const float w = weights[s];
        const uint8_t *p = y + (s * M + m) * SZ;
        uint32_t v[4] = {0u, 0u, 0u, 0u};
        if (whole) {
            __builtin_memcpy(v, p, 16);
        } else if constexpr (SZ == 4) {
            for (int c = 0; c < M - m; ++c)
                v[c] = ((const uint32_t *)p)[c];
        } else {
            for (int c = 0; c < M - m; ++c)
                v[c / 2] |= (uint32_t)((const uint16_t *)p)[c] << (16 * (c % 2));
        }
#pragma unroll
        for (int c = 0; c < N; ++c)
            sum[c] = fmaf(w, to_float<DT>(v, c), sum[c]);
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

// slots per wave of the lists' kernels: at most about 256 chunks
int64_t list_chunk(int64_t S)
{
    int64_t chunk = kChunkMin;
    while (S > chunk * 256)
        chunk *= 2;
    return chunk;
}

} // namespace

extern "C" {

size_t nvfp4_moe_route_workspace_bytes(int64_t T, int64_t E, int64_t k)
{
    if (!route_shape(T, E, k))
        return 0;
    const int64_t S = T * k, chunk = list_chunk(S);
    return (size_t)((((S + chunk - 1) / chunk) * E * 4 + 255) / 256 * 256);
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
    if (!workspace || workspace_bytes < nvfp4_moe_route_workspace_bytes(T, E, k) || !aligned(workspace, 256))
        return NVFP4_ERR_WORKSPACE;
    const hipStream_t st = (hipStream_t)stream;
    RouteParams p{(int32_t)T, (int32_t)E, (int32_t)k, r.score, r.n_group, r.topk_group, r.group_top, r.renormalize,
                  r.scaling};
    const int64_t grid = (T + kRouteWaves - 1) / kRouteWaves;
    if (grid > kMaxGrid)
        return NVFP4_ERR_INVALID_SHAPE;
    by_type(dtype, [&](auto dt) {
        auto go = [&](auto kern) {
            hipLaunchKernelGGL(kern, dim3((uint32_t)grid), dim3(64 * kRouteWaves), 0, st, logits, bias, ids, weights, p);
        };
        if (E <= 64)
            go(nvfp4_route_kernel<dt(), 1>);
        else if (E <= 128)
            go(nvfp4_route_kernel<dt(), 2>);
        else if (E <= 256)
            go(nvfp4_route_kernel<dt(), 4>);
        else if (E <= 512)
            go(nvfp4_route_kernel<dt(), 8>);
        else
            go(nvfp4_route_kernel<dt(), 16>);
    });
    const int32_t S = (int32_t)(T * k), chunk = (int32_t)list_chunk(S), nc = (S + chunk - 1) / chunk;
    int32_t bits = 1;
    while ((E >> bits) != 0)
        ++bits;                                                 // E itself is a key too
    int32_t *counts = (int32_t *)workspace;
    hipLaunchKernelGGL(nvfp4_count_kernel, dim3(nc), dim3(64), 0, st, (const int32_t *)ids, counts, S, (int32_t)E, chunk);
    hipLaunchKernelGGL(nvfp4_scan_kernel, dim3(1), dim3(kScanThreads), 0, st, counts, offsets, nc, (int32_t)E);
    hipLaunchKernelGGL(nvfp4_place_kernel, dim3(nc), dim3(64), 0, st, (const int32_t *)ids, counts,
                       (const int32_t *)offsets, order, S, (int32_t)E, chunk, bits);
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
