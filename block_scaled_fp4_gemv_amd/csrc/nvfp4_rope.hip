// Rotary positions on MI355X (gfx950): each pair of a head's values is turned by
// the angle position * frequency of its pair.
//
//   y0 = c (x0 cos a - x1 sin a),   y1 = c (x0 sin a + x1 cos a),   a = p f
//
// The gradient is the same map with -a (its matrix transposed).
//
// Angles. p f is taken in float64 with its rounding error (a fused multiply-add
// gives it), less the nearest multiple n of pi / 2, whose 106 bits are subtracted
// in two fused steps; the rest, at most pi / 4, is rounded to float32. sin and cos
// of the rest are Taylor's sums in float32 (x^11 / 11! < 2^-28 x: cut off there),
// n mod 4 says which is which. So an angle is as exact at position 2^30 as at 1.
//
// A workgroup takes a few tokens, computes their angles once into LDS and turns
// all its heads with them: the angles cost R / 2 per token, whatever the heads.
// What bounds it: HBM, every value read and written once. 8192 tokens of 40 heads of 128 in float16: 36 us, 4.7 TB/s
// (42 with one unit a thread at a time and divisions in place of multiplications); small calls the launch.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "nvfp4_device.h"
#include "nvfp4_gemv.h"
#include "nvfp4_internal.h"

namespace {

constexpr int kThreads = 256, U = 4;             // units that a thread loads together
constexpr int kMaxAngles = 1024;                // of a workgroup, 8 KiB of LDS
constexpr int kMaxR = 2 * kMaxAngles;
constexpr int64_t kMaxGrid = 0xFFFFFF;          // workgroups of 256 threads in 2^32 work items
constexpr int64_t kMaxStride = INT64_C(1) << 40;

struct RopeParams {
    const uint8_t *x;
    uint8_t *out;
    const int64_t *positions;
    const double *frequencies;
    int64_t T, x_token, x_head, out_token, out_head;    // strides in bytes
    int32_t H, D, half;                                 // half: R / 2
    int32_t tokens_per_wg, heads_per_wg, head_runs;
    Divisor units, pairs;                               // units of a row, R / 2
    int32_t turned;                                     // the first `turned` units are pairs
    float factor, sign;
};

// cos and sin of position * frequency
__device__ __attribute__((always_inline)) inline void cos_sin(double p, double f, float &c, float &s)
{
    const double a = p * f, low = fma(p, f, -a);
    const double n = rint(a * 0.63661977236758134308);          // 2 / pi
    double r = fma(-n, 1.57079632679489655800, a);              // pi / 2 in two float64
    r = fma(-n, 6.12323399573676603587e-17, r);
    const float x = (float)(r + low), x2 = x * x;
    float ps = fmaf(x2, 1.0f / 362880.0f, -1.0f / 5040.0f);
    ps = fmaf(x2, ps, 1.0f / 120.0f);
    ps = fmaf(x2, ps, -1.0f / 6.0f);
    ps = fmaf(x2 * x, ps, x);
    float pc = fmaf(x2, -1.0f / 3628800.0f, 1.0f / 40320.0f);
    pc = fmaf(x2, pc, -1.0f / 720.0f);
    pc = fmaf(x2, pc, 1.0f / 24.0f);
    pc = fmaf(x2, pc, -0.5f);
    pc = fmaf(x2, pc, 1.0f);
    // n mod 4, also where n is past every integer type (the angle then means nothing)
    const int q = (int)(n - 4.0 * floor(0.25 * n));
    const float sw = q & 1 ? pc : ps, cw = q & 1 ? ps : pc;
    s = q & 2 ? -sw : sw;
    c = (q + 1) & 2 ? -cw : cw;
}

template <int DT>
using Raw = std::conditional_t<DT == NVFP4_F32, uint32_t, uint16_t>;

template <int DT>
__device__ __attribute__((always_inline)) inline float to_float(Raw<DT> v)
{
    if constexpr (DT == NVFP4_F32)
        return __builtin_bit_cast(float, v);
    else if constexpr (DT == NVFP4_BF16)
        return __builtin_bit_cast(float, (uint32_t)v << 16);
    else
        return (float)__builtin_bit_cast(_Float16, v);
}

template <int DT>
__device__ __attribute__((always_inline)) inline Raw<DT> from_float(float v)
{
    if constexpr (DT == NVFP4_F32)
        return __builtin_bit_cast(uint32_t, v);
    else if constexpr (DT == NVFP4_BF16)
        return (uint16_t)bf16_bits(v);
    else
        return f16_bits(v);
}

template <int DT, int V>
struct __attribute__((aligned(V == 1 ? sizeof(Raw<DT>) : 16))) Piece {
    Raw<DT> v[V];
};

// A unit is what one thread takes at a time. V > 1: 16 bytes of neighbouring
// values (V of them), twice for halves, whose pairs stand R / 2 apart; V == 1:
// one pair. Behind the pairs come units of V values (of one) that are copied.
template <int DT, bool HALVES, int V>
__global__ __launch_bounds__(kThreads) void nvfp4_rope_kernel(RopeParams p)
{
    __shared__ __attribute__((aligned(16))) float s_cos[kMaxAngles];
    __shared__ __attribute__((aligned(16))) float s_sin[kMaxAngles];
    const int64_t t0 = (int64_t)(blockIdx.x / (uint32_t)p.head_runs) * p.tokens_per_wg;
    const int h0 = (int)(blockIdx.x % (uint32_t)p.head_runs) * p.heads_per_wg;
    const int tokens = (int)min((int64_t)p.tokens_per_wg, p.T - t0), heads = min(p.heads_per_wg, p.H - h0);
    for (uint32_t i = threadIdx.x; i < (uint32_t)(tokens * p.half); i += kThreads) {
        const uint32_t t = divided(i, p.pairs), j = i - t * p.pairs.d;
        float c, s;
        cos_sin((double)p.positions[t0 + t], p.frequencies[j], c, s);
        s_cos[i] = c * p.factor;
        s_sin[i] = s * p.factor * p.sign;
    }
    __syncthreads();
    constexpr int S = sizeof(Raw<DT>);
    using P = Piece<DT, V>;
    // A unit's two parts: pairs' first and second values (halves, and pairs one by one), or none.
    constexpr bool TWO = HALVES || V == 1;
    const uint32_t n = (uint32_t)tokens * (uint32_t)heads * p.units.d;
    for (uint32_t i0 = threadIdx.x; i0 < n; i0 += U * kThreads) {
        P a[U], b[U];
        uint8_t *y[U];
        uint32_t t[U], u[U];
        // all loads, then all stores: a unit's values are no other's, also in place
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const uint32_t i = min(i0 + k * kThreads, n - 1);
            const uint32_t row = divided(i, p.units);
            u[k] = i - row * p.units.d;
            t[k] = heads == 1 ? row : row / (uint32_t)heads;
            const uint32_t h = row - t[k] * (uint32_t)heads;
            const uint8_t *x = p.x + (t0 + t[k]) * p.x_token + (int64_t)(h0 + h) * p.x_head;
            y[k] = p.out + (t0 + t[k]) * p.out_token + (int64_t)(h0 + h) * p.out_head;
            if ((int)u[k] >= p.turned) {
                a[k] = *(const P *)(x + ((u[k] - p.turned) * V + 2 * p.half) * S);
            } else {
                const uint32_t at = u[k] * (HALVES || V > 1 ? V : 2);
                a[k] = *(const P *)(x + at * S);
                if constexpr (TWO)
                    b[k] = *(const P *)(x + (at + (HALVES ? p.half : 1)) * S);
            }
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (i0 + k * kThreads >= n)
                continue;
            if ((int)u[k] >= p.turned) {
                *(P *)(y[k] + ((u[k] - p.turned) * V + 2 * p.half) * S) = a[k];
                continue;
            }
            const float *cs = s_cos + t[k] * p.half, *sn = s_sin + t[k] * p.half;
            const uint32_t at = u[k] * (HALVES || V > 1 ? V : 2);
            if constexpr (TWO) {
                const uint32_t j = HALVES ? at : u[k];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float x0 = to_float<DT>(a[k].v[e]), x1 = to_float<DT>(b[k].v[e]), c = cs[j + e], s = sn[j + e];
                    a[k].v[e] = from_float<DT>(fmaf(-x1, s, x0 * c));
                    b[k].v[e] = from_float<DT>(fmaf(x1, c, x0 * s));
                }
                *(P *)(y[k] + at * S) = a[k];
                *(P *)(y[k] + (at + (HALVES ? p.half : 1)) * S) = b[k];
            } else {
#pragma unroll
                for (int e = 0; e + 1 < V; e += 2) {
                    const float x0 = to_float<DT>(a[k].v[e]), x1 = to_float<DT>(a[k].v[e + 1]), c = cs[(at + e) / 2], s = sn[(at + e) / 2];
                    a[k].v[e] = from_float<DT>(fmaf(-x1, s, x0 * c));
                    a[k].v[e + 1] = from_float<DT>(fmaf(x1, c, x0 * s));
                }
                *(P *)(y[k] + at * S) = a[k];
            }
        }
    }
}

// ------------------------------------------------------------------ host

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

template <int DT>
void launch(const RopeParams &p, bool halves, bool wide, int64_t grid, hipStream_t st)
{
    constexpr int V = DT == NVFP4_F32 ? 4 : 8;
    auto go = [&](auto kern) { hipLaunchKernelGGL(kern, dim3((uint32_t)grid), dim3(kThreads), 0, st, p); };
    if (halves)
        wide ? go(nvfp4_rope_kernel<DT, true, V>) : go(nvfp4_rope_kernel<DT, true, 1>);
    else
        wide ? go(nvfp4_rope_kernel<DT, false, V>) : go(nvfp4_rope_kernel<DT, false, 1>);
}

// Rows [T][H] of D values at these strides do not overlap.
bool apart(int64_t T, int64_t H, int64_t D, int64_t token, int64_t head)
{
    if (token < 0 || head < 0 || token >= kMaxStride || head >= kMaxStride)
        return false;
    if (H == 1)
        return T == 1 || token >= D;
    if (T == 1)
        return head >= D;
    return (head >= D && token >= (H - 1) * head + D) || (token >= D && head >= (T - 1) * token + D);
}

} // namespace

extern "C" {

nvfp4_status_t nvfp4_rope_frequencies(double *frequencies, int64_t R, double base, const nvfp4_rope_scaling_t *scaling)
{
    if (!frequencies)
        return NVFP4_ERR_NULL_POINTER;
    if (R < 2 || R % 2 || R > kMaxR)
        return NVFP4_ERR_INVALID_SHAPE;
    if (!(base > 1.0) || !std::isfinite(base))
        return NVFP4_ERR_INVALID_SCALE;
    const int method = scaling ? scaling->method : NVFP4_ROPE_UNSCALED;
    if (method < NVFP4_ROPE_UNSCALED || method > NVFP4_ROPE_RAMP)
        return NVFP4_ERR_INVALID_ROTATION;
    const double two_pi = 6.28318530717958647693;
    if (method != NVFP4_ROPE_UNSCALED && (!(scaling->factor >= 1.0) || !std::isfinite(scaling->factor)))
        return NVFP4_ERR_INVALID_SCALE;
    if (method == NVFP4_ROPE_BASE && R == 2)        // its one pair has frequency 1 for every base
        return NVFP4_ERR_INVALID_ROTATION;
    const bool parts = method == NVFP4_ROPE_BANDS || method == NVFP4_ROPE_RAMP;
    if (parts && (!(scaling->low > 0.0) || !(scaling->high > scaling->low) || !std::isfinite(scaling->high) ||
                  !(scaling->length > 0.0) || !std::isfinite(scaling->length)))
        return NVFP4_ERR_INVALID_ROTATION;
    if (method == NVFP4_ROPE_BASE)
        base *= std::pow(scaling->factor, (double)R / (double)(R - 2));
    // RAMP: the pairs whose waves turn `high` and `low` times in `length` positions
    double first = 0.0, last = 0.0;
    if (method == NVFP4_ROPE_RAMP) {
        auto pair_of = [&](double turns) { return R * std::log(scaling->length / (turns * two_pi)) / (2.0 * std::log(base)); };
        first = std::max(0.0, std::floor(pair_of(scaling->high)));
        last = std::min((double)(R - 1), std::ceil(pair_of(scaling->low)));
        if (last <= first)
            last = first + 0.001;
    }
    for (int64_t j = 0; j < R / 2; ++j) {
        const double f = std::pow(base, -2.0 * (double)j / (double)R);
        double keep = 1.0;                      // how much of f stays; the rest is f / factor
        if (method == NVFP4_ROPE_LINEAR)
            keep = 0.0;
        else if (method == NVFP4_ROPE_BANDS)
            keep = (scaling->length * f / two_pi - scaling->low) / (scaling->high - scaling->low);
        else if (method == NVFP4_ROPE_RAMP)
            keep = 1.0 - ((double)j - first) / (last - first);
        keep = std::min(1.0, std::max(0.0, keep));
        frequencies[j] = method == NVFP4_ROPE_UNSCALED || method == NVFP4_ROPE_BASE
                             ? f : f * keep + f / scaling->factor * (1.0 - keep);
    }
    return NVFP4_OK;
}

nvfp4_status_t nvfp4_rope(const void *x, int dtype, void *out, const int64_t *positions, const double *frequencies,
                          int64_t T, int64_t H, int64_t D, int64_t R, int64_t x_token_stride, int64_t x_head_stride,
                          int64_t out_token_stride, int64_t out_head_stride, int layout, float factor, int transpose,
                          void *stream)
{
    if (!x || !out || !positions || !frequencies)
        return NVFP4_ERR_NULL_POINTER;
    if (dtype != NVFP4_F16 && dtype != NVFP4_BF16 && dtype != NVFP4_F32)
        return NVFP4_ERR_INVALID_TYPE;
    if (T < 1 || H < 1 || D < 2 || R < 2 || R % 2 || R > D || R > kMaxR || H > (1 << 20) || D > (1 << 20) ||
        T > (INT64_C(1) << 40))
        return NVFP4_ERR_INVALID_SHAPE;
    if (layout != NVFP4_ROPE_HALF && layout != NVFP4_ROPE_INTERLEAVED)
        return NVFP4_ERR_INVALID_ROTATION;
    if (transpose != 0 && transpose != 1)
        return NVFP4_ERR_INVALID_ROTATION;
    if (!std::isfinite(factor))
        return NVFP4_ERR_INVALID_SCALE;
    if (x_token_stride < 0 || x_head_stride < 0 || x_token_stride >= kMaxStride || x_head_stride >= kMaxStride ||
        !apart(T, H, D, out_token_stride, out_head_stride) ||
        (x == out && ((T > 1 && x_token_stride != out_token_stride) || (H > 1 && x_head_stride != out_head_stride))))
        return NVFP4_ERR_INVALID_STRIDE;
    const int64_t size = dtype == NVFP4_F32 ? 4 : 2;
    if (!aligned(x, size) || !aligned(out, size) || !aligned(positions, 8) || !aligned(frequencies, 8))
        return NVFP4_ERR_MISALIGNED;
    const bool halves = layout == NVFP4_ROPE_HALF;
    const int64_t V = 16 / size, half = R / 2;
    // 16 bytes at a time where every row, both halves of its pairs and its rest start at multiples of that
    auto whole = [&](int64_t stride, int64_t n) { return n == 1 || stride % V == 0; };
    const bool wide = aligned(x, 16) && aligned(out, 16) && whole(x_token_stride, T) && whole(out_token_stride, T) &&
                      whole(x_head_stride, H) && whole(out_head_stride, H) && (halves ? half : R) % V == 0 && (D - R) % V == 0;
    RopeParams p{};
    p.x = (const uint8_t *)x, p.out = (uint8_t *)out;
    p.positions = positions, p.frequencies = frequencies;
    p.T = T, p.H = (int32_t)H, p.D = (int32_t)D, p.half = (int32_t)half;
    p.x_token = x_token_stride * size, p.x_head = x_head_stride * size;
    p.out_token = out_token_stride * size, p.out_head = out_head_stride * size;
    p.factor = factor, p.sign = transpose ? -1.0f : 1.0f;
    p.turned = (int32_t)(wide ? (halves ? half : R) / V : half);
    const int64_t units = p.turned + (x == out ? 0 : wide ? (D - R) / V : D - R);      // in place the rest stays
    p.units = divisor_of((uint32_t)units), p.pairs = divisor_of((uint32_t)half);
    // tokens whose angles fill two rounds of the threads; fewer, then heads apart, while there is not a
    // workgroup for every place (1024 of them are four on each CU)
    int64_t tokens = std::max<int64_t>(1, std::min<int64_t>(T, 2 * kThreads / half)), heads = H;
    while (tokens > 1 && (T + tokens - 1) / tokens < 1024)
        tokens = (tokens + 1) / 2;
    while (heads > 1 && (T + tokens - 1) / tokens * ((H + heads - 1) / heads) < 1024 && tokens * heads * units > kThreads)
        heads = (heads + 1) / 2;
    while (heads > 1 && tokens * heads * units > (1 << 20))        // units of a workgroup are counted in 32 bits
        heads = (heads + 1) / 2;
    p.tokens_per_wg = (int32_t)tokens, p.heads_per_wg = (int32_t)heads;
    p.head_runs = (int32_t)((H + heads - 1) / heads);
    const int64_t runs = (T + tokens - 1) / tokens;
    if (runs > kMaxGrid / p.head_runs)
        return NVFP4_ERR_INVALID_SHAPE;
    const int64_t grid = runs * p.head_runs;
    const hipStream_t st = (hipStream_t)stream;
    if (dtype == NVFP4_F16)
        launch<NVFP4_F16>(p, halves, wide, grid, st);
    else if (dtype == NVFP4_BF16)
        launch<NVFP4_BF16>(p, halves, wide, grid, st);
    else
        launch<NVFP4_F32>(p, halves, wide, grid, st);
    const hipError_t e = hipGetLastError();
    if (e == hipSuccess)
        return NVFP4_OK;
    nvfp4_record_hip_error((int)e);
    return NVFP4_ERR_HIP;
}

} // extern "C"
