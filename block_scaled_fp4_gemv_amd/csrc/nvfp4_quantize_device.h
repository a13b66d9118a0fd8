// Blocks of 16 values to NVFP4 codes and a scale, and 16 values back to memory:
// shared by the quantisation of activations and the key/value cache's writes, so
// that both give the same codes. Internal header.
//
//   s = E4M3 nearest to max |x| / (6 g),   q[k] = E2M1 nearest to x[k] / (s g)
//
// Exactness. Both roundings are those of the exact quotients. A code is decided
// by comparing |x| with a midpoint of two codes times s and g: midpoint * s
// has at most 7 significant bits (an exact float32), and the sign of
// fma(midpoint * s, -g, |x|) is the sign of the exact difference, since the
// fused multiply-add rounds once and to the nearest, and a nonzero difference
// of these operands stays nonzero (g >= 2^-100, so the midpoints are at least
// 2^-111 and a difference at least 2^-142). The same test with 6 * (midpoint
// of two E4M3 values), at most 7 bits, decides the scale. No division's
// rounding enters.
#ifndef NVFP4_QUANTIZE_DEVICE_H
#define NVFP4_QUANTIZE_DEVICE_H

#include <hip/hip_runtime.h>

#include <cstdint>

#include "nvfp4_device.h"
#include "nvfp4_gemv.h"

namespace {

constexpr float kMinScale = 7.8886091e-31f;     // 2^-100

// ------------------------------------------------------------------ loads

// 16 consecutive elements, as loaded. The address has the type's own alignment
// only: gfx950 takes 16-byte global loads at any.
template <int DT>
struct Block {
    uint32_t w[DT == NVFP4_F32 ? 16 : 8];
};

template <int DT>
__device__ __attribute__((always_inline)) inline Block<DT> load_block(const uint8_t *p)
{
    Block<DT> b;
    __builtin_memcpy(&b, p, sizeof(b));
    return b;
}

// the i-th element from memory again
template <int DT>
__device__ __attribute__((always_inline)) inline float load_element(const uint8_t *p, int i)
{
    if constexpr (DT == NVFP4_F32)
        return ((const float *)p)[i];
    else if constexpr (DT == NVFP4_BF16)
        return __builtin_bit_cast(float, (uint32_t)((const uint16_t *)p)[i] << 16);
    else
        return (float)((const _Float16 *)p)[i];
}

// element i as float32 (exact for every type)
template <int DT>
__device__ __attribute__((always_inline)) inline float element(const Block<DT> &b, int i)
{
    if constexpr (DT == NVFP4_F32)
        return __builtin_bit_cast(float, b.w[i]);
    else if constexpr (DT == NVFP4_BF16)
        return __builtin_bit_cast(float, i % 2 ? b.w[i / 2] & 0xFFFF0000u : b.w[i / 2] << 16);
    else
        return i % 2 ? (float)as_h2(b.w[i / 2]).y : (float)as_h2(b.w[i / 2]).x;
}

template <int DT>
constexpr int kSize = DT == NVFP4_F32 ? 4 : 2;

// ------------------------------------------------------------------ sizes

typedef uint16_t ushort2_t __attribute__((ext_vector_type(2)));

// Largest size in `top`: 16-bit types two at a time, their sizes being ordered
// as integers. Infinities and NaN are the largest integers and win.
template <int DT>
__device__ __attribute__((always_inline)) inline uint32_t max_size(uint32_t top, uint32_t w)
{
    if constexpr (DT == NVFP4_F32)
        return max(top, w & 0x7FFFFFFFu);
    const ushort2_t m = __builtin_elementwise_max(__builtin_bit_cast(ushort2_t, top),
                                                  __builtin_bit_cast(ushort2_t, w & 0x7FFF7FFFu));
    return __builtin_bit_cast(uint32_t, m);
}

// A size as max_size leaves it (16-bit types: the larger half) -> float32 bits
template <int DT>
__device__ __attribute__((always_inline)) inline uint32_t size_bits(uint32_t top)
{
    if constexpr (DT == NVFP4_BF16)
        return max(top & 0xFFFFu, top >> 16) << 16;
    else if constexpr (DT == NVFP4_F16)
        return __builtin_bit_cast(uint32_t, (float)__builtin_bit_cast(_Float16, (uint16_t)max(top & 0xFFFFu, top >> 16)));
    else
        return top;
}

// ------------------------------------------------------------------ quantise

__device__ __attribute__((always_inline)) inline float e4m3_value(uint32_t code)
{
    return __builtin_amdgcn_cvt_f32_fp8((int)code, 0);
}

// What the blocks need of the global scale.
struct Global {
    float g, per_g;                             // g and about 1 / (6 g), 0 where that is no normal number
    bool good;
};

__device__ __attribute__((always_inline)) inline Global global_of(const float *gp)
{
    const float g = gp ? *gp : 1.0f;
    return {g, g < 0x1p100f ? __builtin_amdgcn_rcpf(g) * (1.0f / 6.0f) : 0.0f, g >= kMinScale && g < __builtin_inff()};
}

// E4M3 code of the exact quotient amax / (6 g), amax finite or infinite, >= 0.
// The float32 quotient is within a few units of its last place, so its code is
// the right one or a neighbour; the two midpoints around it decide.
__device__ __attribute__((always_inline)) inline uint32_t scale_code(float amax, const Global &gl)
{
    const float g = gl.g;
    const float v = fminf(gl.per_g != 0.0f ? amax * gl.per_g : (amax / g) * (1.0f / 6.0f), 448.0f);
    uint32_t c = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v, v, 0, false) & 0xFFu;
    const float here = e4m3_value(c);
    const float above = e4m3_value(c < 126u ? c + 1 : c), below = e4m3_value(c > 0u ? c - 1 : c);
    const float up = fmaf(3.0f * (here + above), -g, amax);     // 6 * midpoint
    const float down = fmaf(3.0f * (here + below), -g, amax);
    const bool odd = c & 1u;
    if (c < 126u && (up > 0.0f || (up == 0.0f && odd)))
        return c + 1;
    if (c > 0u && (down < 0.0f || (down == 0.0f && odd)))
        return c - 1;
    return c;
}

// E2M1 code (sign included) of the exact quotient x / (s g), s > 0.
__device__ __attribute__((always_inline)) inline uint32_t value_code(float x, float s, float g)
{
    const float a = fabsf(x);
    // one count per midpoint passed; at a tie the even neighbour's side
    uint32_t n = 0;
    n += fmaf(0.25f * s, -g, a) > 0.0f;
    n += fmaf(0.75f * s, -g, a) >= 0.0f;
    n += fmaf(1.25f * s, -g, a) > 0.0f;
    n += fmaf(1.75f * s, -g, a) >= 0.0f;
    n += fmaf(2.5f * s, -g, a) > 0.0f;
    n += fmaf(3.5f * s, -g, a) >= 0.0f;
    n += fmaf(5.0f * s, -g, a) > 0.0f;
    return n | ((__builtin_bit_cast(uint32_t, x) >> 31) << 3);
}

// 8 values (from element i on) times r -> 8 codes
template <int DT>
__device__ __attribute__((always_inline)) inline uint32_t convert8(const Block<DT> &b, int i, float r)
{
    uint32_t w = 0u;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, element<DT>(b, i) * r, element<DT>(b, i + 1) * r, 1.0f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, element<DT>(b, i + 2) * r, element<DT>(b, i + 3) * r, 1.0f, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, element<DT>(b, i + 4) * r, element<DT>(b, i + 5) * r, 1.0f, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, element<DT>(b, i + 6) * r, element<DT>(b, i + 7) * r, 1.0f, 3);
    return w;
}

// One block of 16 values (at x) -> 8 bytes of codes and the scale code.
template <int DT>
__device__ __attribute__((always_inline)) inline uint2_t quantize_block(const uint8_t *x, const Global &gl,
                                                                        uint32_t &scale)
{
    const Block<DT> b = load_block<DT>(x);
    uint32_t top = 0u;                          // sizes ordered as integers: NaN above infinity
#pragma unroll
    for (int i = 0; i < (DT == NVFP4_F32 ? 16 : 8); ++i)
        top = max_size<DT>(top, b.w[i]);
    const float amax = __builtin_bit_cast(float, size_bits<DT>(top));
    if (!gl.good || amax != amax) {
        scale = 0x7Fu;
        return (uint2_t){0u, 0u};
    }
    scale = scale_code(amax, gl);
    if (scale == 0u)
        return (uint2_t){0u, 0u};
    const float s = e4m3_value(scale);
    // The reciprocal, the products and s * g are off by less than 2^-21 together:
    // the exact quotients lie between the products with r (1 -+ 2^-21). Where the
    // conversion (nearest, ties to even) gives both ends the same code, that is
    // the exact quotient's code; else the two are neighbours and the midpoint
    // between them decides. bfloat16 values have few different sizes, so a
    // quotient stands on a midpoint in most waves: the doubtful values are
    // taken one by one (all 16 anew: 52 us for 8192 x 7168, one by one 29).
    const float u = s * gl.g, r = __builtin_amdgcn_rcpf(u);
    const float r0 = r * (1.0f - 0x1p-21f), r1 = r * (1.0f + 0x1p-21f);
    if (!(u < 0x1p100f) || !(amax < __builtin_inff())) {
        uint32_t w[2] = {0u, 0u};
#pragma unroll
        for (int i = 0; i < 16; ++i)
            w[i / 8] |= value_code(element<DT>(b, i), s, gl.g) << (4 * (i % 8));
        return (uint2_t){w[0], w[1]};
    }
    uint64_t low = (uint64_t)convert8<DT>(b, 8, r0) << 32 | convert8<DT>(b, 0, r0);
    const uint64_t high = (uint64_t)convert8<DT>(b, 8, r1) << 32 | convert8<DT>(b, 0, r1);
    uint64_t differ = low ^ high;
    while (differ) {
        const int at = __builtin_ctzll(differ) / 4;
        const uint64_t nibble = (uint64_t)15 << (4 * at);
        const uint32_t c0 = (uint32_t)(low >> (4 * at)) & 7u, c1 = (uint32_t)(high >> (4 * at)) & 7u;
        const half2_t ends = fp4x2<0>(c0 | c1 << 4);
        const float middle = 0.5f * ((float)ends.x + (float)ends.y);
        const float d = fmaf(middle * s, -gl.g, fabsf(load_element<DT>(x, at)));
        if (d > 0.0f || (d == 0.0f && (c0 & 1u)))
            low ^= differ & nibble;
        differ &= ~nibble;
    }
    return (uint2_t){(uint32_t)low, (uint32_t)(low >> 32)};
}

// ------------------------------------------------------------------ values

template <int DT>
__device__ __attribute__((always_inline)) inline void store16(uint8_t *p, const float (&v)[16])
{
    if constexpr (DT == NVFP4_F32) {
        __builtin_memcpy(p, v, 64);
    } else {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (DT == NVFP4_F16)
                w[i] = (uint32_t)f16_bits(v[2 * i]) | ((uint32_t)f16_bits(v[2 * i + 1]) << 16);
            else
                w[i] = bf16_bits(v[2 * i]) | (bf16_bits(v[2 * i + 1]) << 16);
        }
        __builtin_memcpy(p, w, 32);
    }
}

} // namespace

#endif
