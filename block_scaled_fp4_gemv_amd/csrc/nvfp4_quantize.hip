// Quantisation of activations to NVFP4 on MI355X (gfx950): the global scale,
// codes and block scales, and the way back to values.
//
//   g    = max finite |x| * (1 / 2688)
//   s[b] = E4M3 nearest to max_b |x| / (6 g),   q[k] = E2M1 nearest to x[k] / (s[b] g)
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
//
// What bounds it: HBM. Each kernel reads and writes every byte once. 8192 x 7168
// bf16: global scale 23 us (5.1 TB/s), quantise 28 with x in the last-level cache
// and 34 without (4.5 TB/s), dequantise 28 (5.4 TB/s); with plain scales 31 and 25.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "nvfp4_device.h"
#include "nvfp4_gemv.h"
#include "nvfp4_internal.h"

namespace {

constexpr int kQThreads = 256;
// One workgroup per CU, 16 waves of 4 loads each: the workgroups' maxima meet in
// atomics on one address, and 1024 workgroups of 4 waves took 47 us where these
// take 35 (8192 x 7168 bf16, 117 MB). The loads are non-temporal: 23 us (5.1 TB/s)
// whatever was written before, where ordinary ones took 24, and 29 to 35 after
// a kernel that had filled the cache with its output.
constexpr int kAmaxThreads = 1024;
constexpr int kAmaxMaxGrid = 256;
constexpr float kMinScale = 7.8886091e-31f;     // 2^-100
constexpr int64_t kMaxGrid = 0xFFFFFF;           // workgroups of 256 threads in 2^32 work items

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

// ------------------------------------------------------------------ global scale

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

// The same, values that are not finite passed over.
template <int DT>
__device__ __attribute__((always_inline)) inline uint32_t max_finite(uint32_t top, uint32_t w)
{
    if constexpr (DT == NVFP4_F32)
        return (w & 0x7FFFFFFFu) < 0x7F800000u ? max_size<DT>(top, w) : top;
    constexpr uint32_t inf = DT == NVFP4_BF16 ? 0x7F80u : 0x7C00u;
    w &= 0x7FFF7FFFu;
    w = (w & 0xFFFFu) >= inf ? w & 0xFFFF0000u : w;
    w = (w >> 16) >= inf ? w & 0xFFFFu : w;
    return max_size<DT>(top, w);
}

template <int DT>
__device__ __attribute__((always_inline)) inline bool all_finite(uint32_t top)
{
    if constexpr (DT == NVFP4_F32)
        return top < 0x7F800000u;
    constexpr uint32_t inf = DT == NVFP4_BF16 ? 0x7F80u : 0x7C00u;
    return (top & 0xFFFFu) < inf && (top >> 16) < inf;
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

struct ScanParams {
    int64_t pieces, per_row;                    // whole 16-byte pieces of all rows, of one
    int64_t K, rows, lines;                     // rows per batch, rows of all batches
    int64_t row_bytes, batch_bytes;
};

typedef uint32_t any_uint4_t __attribute__((ext_vector_type(4), aligned(2)));         // at any address of a value

// One thread's share: runs of U * kAmaxThreads pieces per workgroup, U loads in
// flight, without a condition (loads past the end clamped to the last piece
// made every wave of the last round ask for one line); then the pieces that
// fill no run, and the rows' last elements that fill no piece.
// FINITE: passes over what is not finite. FLAT: one row.
template <int DT, bool FINITE, bool FLAT>
__device__ __attribute__((always_inline)) inline uint32_t scan_share(const uint8_t *__restrict__ x, const ScanParams &p)
{
    constexpr int U = 4, N = 16 / kSize<DT>, RUN = U * kAmaxThreads;
    uint32_t top = 0;
    auto take = [&](uint32_t w) { top = FINITE ? max_finite<DT>(top, w) : max_size<DT>(top, w); };
    auto row_at = [&](int64_t r) {
        const int64_t l = r < p.rows ? 0 : r / p.rows;
        return x + l * p.batch_bytes + (r - l * p.rows) * p.row_bytes;
    };
    auto piece_at = [&](int64_t k) -> const uint8_t * {
        if constexpr (FLAT)
            return x + k * 16;
        const int64_t r = p.pieces < INT32_MAX ? (int64_t)((uint32_t)k / (uint32_t)p.per_row) : k / p.per_row;
        return row_at(r) + (k - r * p.per_row) * 16;
    };
    auto take4 = [&](uint4_t v) {
        take(v.x);
        take(v.y);
        take(v.z);
        take(v.w);
    };
    const int64_t runs = p.pieces / RUN;
    for (int64_t run = blockIdx.x; run < runs; run += gridDim.x) {
        uint4_t v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            v[u] = __builtin_nontemporal_load((const any_uint4_t *)piece_at(run * RUN + u * kAmaxThreads + threadIdx.x));
#pragma unroll
        for (int u = 0; u < U; ++u)
            take4(v[u]);
    }
    const int64_t step = (int64_t)gridDim.x * kAmaxThreads, i = (int64_t)blockIdx.x * kAmaxThreads + threadIdx.x;
    for (int64_t k = runs * RUN + i; k < p.pieces; k += step) {
        uint4_t v;
        __builtin_memcpy(&v, piece_at(k), 16);
        take4(v);
    }
    const int64_t rest = p.K - p.per_row * N;
    for (int64_t at = i; at < p.lines * rest; at += step) {
        const int64_t r = at / rest;
        const uint8_t *q = row_at(r) + (p.per_row * N + (at - r * rest)) * kSize<DT>;
        if constexpr (DT == NVFP4_F32)
            take(*(const uint32_t *)q);
        else
            take(*(const uint16_t *)q);
    }
    return top;
}

// A thread that meets a value that is not finite reads its share again.
// Maxima are joined with an atomic maximum (any order gives the same result);
// the last workgroup (by ticket) writes the scale and clears the two counters.
template <int DT, bool FLAT>
__global__ __launch_bounds__(kAmaxThreads) void nvfp4_global_scale_kernel(const uint8_t *__restrict__ x,
                                                                         float *__restrict__ scale,
                                                                         uint32_t *__restrict__ ws, ScanParams p)
{
    uint32_t top = scan_share<DT, false, FLAT>(x, p);
    if (!all_finite<DT>(top))
        top = scan_share<DT, true, FLAT>(x, p);
    top = size_bits<DT>(top);
#pragma unroll
    for (int d = 32; d; d >>= 1)
        top = max(top, (uint32_t)__shfl_xor((int)top, d));
    __shared__ uint32_t wave_top[kAmaxThreads / 64];
    if (threadIdx.x % 64 == 0)
        wave_top[threadIdx.x / 64] = top;
    __syncthreads();
    if (threadIdx.x != 0)
        return;
#pragma unroll
    for (int w = 1; w < kAmaxThreads / 64; ++w)
        top = max(top, wave_top[w]);
    if (gridDim.x > 1) {
        // the maximum has to be in place before the ticket is taken: the
        // returned value is waited for
        const uint32_t was = __hip_atomic_fetch_max(&ws[0], top, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        asm volatile("s_waitcnt vmcnt(0)" : : "v"(was) : "memory");
        const uint32_t before = __hip_atomic_fetch_add(&ws[1], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (before != gridDim.x - 1)
            return;
        top = __hip_atomic_exchange(&ws[0], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __hip_atomic_store(&ws[1], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    // the product with the float32 nearest to 1/2688: within one step of the
    // quotient, and any g near it serves (the codes are exact for the g written)
    *scale = top ? fmaxf(__builtin_bit_cast(float, top) * (1.0f / 2688.0f), kMinScale) : 1.0f;
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

struct QParams {
    int64_t rows, row_bytes, batch_bytes;
    int32_t nkb;                     // 16-element blocks per row
    int32_t wg_per_band;             // workgroups per band of rows (blocked) or batch (plain)
    int32_t bands;                   // bands of rows per batch (blocked)
};

// Plain scales: one thread per block, blocks of a batch in order.
template <int DT>
__global__ __launch_bounds__(kQThreads) void nvfp4_quantize_plain_kernel(
    const uint8_t *__restrict__ x, const float *__restrict__ gp, uint8_t *__restrict__ codes,
    uint8_t *__restrict__ scales, QParams p)
{
    const Global gl = global_of(gp);
    const int64_t l = blockIdx.x / (uint32_t)p.wg_per_band;
    // the grid keeps every index of a block below 2^32
    const uint32_t i = (blockIdx.x % (uint32_t)p.wg_per_band) * kQThreads + threadIdx.x;
    if (i >= p.rows * p.nkb)
        return;
    const int64_t r = i / (uint32_t)p.nkb;
    const uint32_t kb = i % (uint32_t)p.nkb;
    uint32_t s;
    const uint2_t q =
        quantize_block<DT>(x + l * p.batch_bytes + r * p.row_bytes + (int64_t)kb * 16 * kSize<DT>, gl, s);
    const int64_t o = l * p.rows * p.nkb + i;
    *(uint2_t *)(codes + o * 8) = q;
    scales[o] = (uint8_t)s;
}

// Blocked scales: a workgroup takes 16 rows, r32 .. r32+3 of each 32-row
// quarter of a 128-row block, and 16 columns of blocks. Four neighbouring
// threads hold the four scales of a row and 4-column group; one of them
// stores the word. Rows and columns past the matrix write zero scales.
template <int DT>
__global__ __launch_bounds__(kQThreads) void nvfp4_quantize_blocked_kernel(
    const uint8_t *__restrict__ x, const float *__restrict__ gp, uint8_t *__restrict__ codes,
    uint8_t *__restrict__ scales, QParams p)
{
    const Global gl = global_of(gp);
    const int32_t t = threadIdx.x;
    const uint32_t band = blockIdx.x / (uint32_t)p.wg_per_band;            // batch * bands + 16-row band
    const int32_t kb = (int32_t)(blockIdx.x % (uint32_t)p.wg_per_band) * 16 + t % 16;
    const int64_t l = band / (uint32_t)p.bands;
    const int32_t b = (int32_t)(band % (uint32_t)p.bands);
    const int64_t rb = b / 8;
    const int32_t r32 = (b % 8) * 4 + t / 64, quarter = (t / 16) % 4;
    const int64_t r = rb * 128 + quarter * 32 + r32;
    const int32_t ncb = (p.nkb + 3) / 4;
    uint32_t s = 0u;
    if (r < p.rows && kb < p.nkb) {
        const uint2_t q =
            quantize_block<DT>(x + l * p.batch_bytes + r * p.row_bytes + (int64_t)kb * 16 * kSize<DT>, gl, s);
        *(uint2_t *)(codes + ((l * p.rows + r) * p.nkb + kb) * 8) = q;
    }
    // four lanes' scales in one word, lane 0 of the four stores it
    s <<= 8 * (t % 4);
    s |= (uint32_t)__shfl_xor((int)s, 1);
    s |= (uint32_t)__shfl_xor((int)s, 2);
    if (t % 4 == 0 && kb / 4 < ncb) {
        const int64_t nrb = (p.rows + 127) / 128;
        *(uint32_t *)(scales + ((l * nrb + rb) * ncb + kb / 4) * 512 + r32 * 16 + quarter * 4) = s;
    }
}

// ------------------------------------------------------------------ dequantise

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

template <int DT, int LAYOUT>
__global__ __launch_bounds__(kQThreads) void nvfp4_dequantize_kernel(
    const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales, const float *__restrict__ gp,
    uint8_t *__restrict__ out, uint32_t rows, int64_t blocks, uint32_t nkb)
{
    // the grid keeps every index of a block below 2^32
    const uint32_t i = blockIdx.x * kQThreads + threadIdx.x;
    if (i >= blocks)
        return;
    const float g = gp ? *gp : 1.0f;
    const uint32_t lr = i / nkb, kb = i % nkb;
    int64_t at = i;
    if constexpr (LAYOUT == NVFP4_SF_BLOCKED) {
        const uint32_t l = lr / rows, r = lr % rows, ncb = (nkb + 3) / 4;
        const int64_t nrb = (rows + 127) / 128;
        at = ((l * nrb + r / 128) * ncb + kb / 4) * 512 + (r % 32) * 16 + ((r % 128) / 32) * 4 + kb % 4;
    }
    const uint2_t q = *(const uint2_t *)(codes + (int64_t)i * 8);
    const float s = e4m3_value(scales[at]);
    float v[16];
    const uint32_t w[2] = {q.x, q.y};
#pragma unroll
    for (int d = 0; d < 2; ++d) {
        const half2_t h[4] = {fp4x2<0>(w[d]), fp4x2<1>(w[d]), fp4x2<2>(w[d]), fp4x2<3>(w[d])};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[8 * d + 2 * j] = (float)h[j].x * s * g;
            v[8 * d + 2 * j + 1] = (float)h[j].y * s * g;
        }
    }
    store16<DT>(out + (int64_t)i * 16 * kSize<DT>, v);
}

// ------------------------------------------------------------------ host

constexpr int64_t kMaxRows = INT64_C(1) << 40, kMaxStride = INT64_C(1) << 40;

bool known_type(int dtype) { return dtype == NVFP4_F16 || dtype == NVFP4_BF16 || dtype == NVFP4_F32; }
int64_t type_size(int dtype) { return dtype == NVFP4_F32 ? 4 : 2; }
bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

bool good_strides(int64_t rows, int64_t K, int64_t row_stride, int64_t batch_stride)
{
    return row_stride >= (rows > 1 ? K : 0) && row_stride < kMaxStride && batch_stride >= 0 &&
           batch_stride < kMaxStride;
}

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

} // namespace

extern "C" {

size_t nvfp4_global_scale_workspace_bytes(void) { return 256; }

nvfp4_status_t nvfp4_global_scale(const void *x, int dtype, float *scale, int64_t rows, int64_t K, int64_t L,
                                  int64_t row_stride, int64_t batch_stride, void *workspace,
                                  size_t workspace_bytes, void *stream)
{
    if (!x || !scale)
        return NVFP4_ERR_NULL_POINTER;
    if (!known_type(dtype))
        return NVFP4_ERR_INVALID_TYPE;
    if (rows < 1 || K < 1 || L < 1 || rows > kMaxRows || L > kMaxRows || K > INT32_MAX / 2 || rows > kMaxRows / L ||
        rows * L > (INT64_C(1) << 62) / K)
        return NVFP4_ERR_INVALID_SHAPE;
    if (!good_strides(rows, K, row_stride, batch_stride))
        return NVFP4_ERR_INVALID_STRIDE;
    const int64_t size = type_size(dtype);
    if (!aligned(x, size) || !aligned(scale, 4))
        return NVFP4_ERR_MISALIGNED;
    if (!workspace || workspace_bytes < nvfp4_global_scale_workspace_bytes() || !aligned(workspace, 256))
        return NVFP4_ERR_WORKSPACE;
    const int64_t n = 16 / size;
    // a dense tensor is one row
    const bool flat = (rows == 1 || row_stride == K) && (L == 1 || batch_stride == rows * K);
    ScanParams p{};
    p.K = flat ? L * rows * K : K;
    p.rows = flat ? 1 : rows;
    p.lines = flat ? 1 : rows * L;
    p.per_row = p.K / n;
    p.pieces = p.lines * p.per_row;
    p.row_bytes = row_stride * size;
    p.batch_bytes = batch_stride * size;
    const int64_t units = std::max<int64_t>(p.pieces, p.lines);
    const int64_t grid = std::min<int64_t>(kAmaxMaxGrid, (units + kAmaxThreads - 1) / kAmaxThreads);
    by_type(dtype, [&](auto dt) {
        auto go = [&](auto kern) {
            hipLaunchKernelGGL(kern, dim3((uint32_t)grid), dim3(kAmaxThreads), 0, (hipStream_t)stream,
                               (const uint8_t *)x, scale, (uint32_t *)workspace, p);
        };
        flat ? go(nvfp4_global_scale_kernel<dt(), true>) : go(nvfp4_global_scale_kernel<dt(), false>);
    });
    return finish();
}

nvfp4_status_t nvfp4_quantize(const void *x, int dtype, const float *global_scale, void *codes, void *scales,
                              int64_t rows, int64_t K, int64_t L, int64_t row_stride, int64_t batch_stride,
                              int sf_layout, void *stream)
{
    if (!x || !codes || !scales)
        return NVFP4_ERR_NULL_POINTER;
    if (!known_type(dtype))
        return NVFP4_ERR_INVALID_TYPE;
    if (nvfp4_blocked_scales_bytes(rows, K, L) == 0 || rows * L > (INT64_C(1) << 62) / K)
        return NVFP4_ERR_INVALID_SHAPE;
    if (sf_layout != NVFP4_SF_PLAIN && sf_layout != NVFP4_SF_BLOCKED)
        return NVFP4_ERR_INVALID_LAYOUT;
    if (!good_strides(rows, K, row_stride, batch_stride))
        return NVFP4_ERR_INVALID_STRIDE;
    const int64_t size = type_size(dtype);
    const bool blocked = sf_layout == NVFP4_SF_BLOCKED;
    if (!aligned(x, size) || !aligned(codes, 8) || (blocked && !aligned(scales, 4)) ||
        (global_scale && !aligned(global_scale, 4)))
        return NVFP4_ERR_MISALIGNED;
    QParams p{};
    p.rows = rows;
    p.row_bytes = row_stride * size;
    p.batch_bytes = batch_stride * size;
    p.nkb = (int32_t)(K / 16);
    int64_t grid;
    if (blocked) {
        const int64_t bands = (rows + 127) / 128 * 8, per = (p.nkb + 15) / 16;
        if (bands > INT32_MAX || bands > kMaxGrid / per / L)
            return NVFP4_ERR_INVALID_SHAPE;
        p.bands = (int32_t)bands;
        p.wg_per_band = (int32_t)per;
        grid = L * bands * per;
    } else {
        const int64_t per = (rows * p.nkb + kQThreads - 1) / kQThreads;
        if (per > kMaxGrid / L)
            return NVFP4_ERR_INVALID_SHAPE;
        p.wg_per_band = (int32_t)per;
        grid = L * per;
    }
    by_type(dtype, [&](auto dt) {
        auto go = [&](auto kern) {
            hipLaunchKernelGGL(kern, dim3((uint32_t)grid), dim3(kQThreads), 0, (hipStream_t)stream,
                               (const uint8_t *)x, global_scale, (uint8_t *)codes, (uint8_t *)scales, p);
        };
        blocked ? go(nvfp4_quantize_blocked_kernel<dt()>) : go(nvfp4_quantize_plain_kernel<dt()>);
    });
    return finish();
}

nvfp4_status_t nvfp4_dequantize(const void *codes, const void *scales, const float *global_scale, void *out,
                                int dtype, int64_t rows, int64_t K, int64_t L, int sf_layout, void *stream)
{
    if (!codes || !scales || !out)
        return NVFP4_ERR_NULL_POINTER;
    if (!known_type(dtype))
        return NVFP4_ERR_INVALID_TYPE;
    if (nvfp4_blocked_scales_bytes(rows, K, L) == 0 || rows * L > (INT64_C(1) << 62) / K)
        return NVFP4_ERR_INVALID_SHAPE;
    if (sf_layout != NVFP4_SF_PLAIN && sf_layout != NVFP4_SF_BLOCKED)
        return NVFP4_ERR_INVALID_LAYOUT;
    if (!aligned(codes, 8) || !aligned(out, type_size(dtype)) || (global_scale && !aligned(global_scale, 4)))
        return NVFP4_ERR_MISALIGNED;
    const int64_t nkb = K / 16, blocks = L * rows * nkb;
    const int64_t grid = (blocks + kQThreads - 1) / kQThreads;
    if (grid > kMaxGrid)
        return NVFP4_ERR_INVALID_SHAPE;
    by_type(dtype, [&](auto dt) {
        auto go = [&](auto kern) {
            hipLaunchKernelGGL(kern, dim3((uint32_t)grid), dim3(kQThreads), 0, (hipStream_t)stream,
                               (const uint8_t *)codes, (const uint8_t *)scales, global_scale, (uint8_t *)out,
                               (uint32_t)rows, blocks, (uint32_t)nkb);
        };
        sf_layout == NVFP4_SF_BLOCKED ? go(nvfp4_dequantize_kernel<dt(), NVFP4_SF_BLOCKED>)
                                      : go(nvfp4_dequantize_kernel<dt(), NVFP4_SF_PLAIN>);
    });
    return finish();
}

} // extern "C"
