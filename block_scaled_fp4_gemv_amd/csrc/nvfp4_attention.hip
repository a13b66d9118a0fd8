// Attention over a paged NVFP4 key/value cache on MI355X (gfx950).
//
//   out = sum_t p_t V[t],   p = softmax over the visible t of scale * q . K[t]
//
// This form: a wave per query and head, which takes the visible positions one by one
// with a running maximum and sum.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "nvfp4_device.h"
#include "nvfp4_gemv.h"
#include "nvfp4_internal.h"

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
    int64_t code_page, scale_page;
    int32_t T, H, B, width, pages, shift, heads, G, D;
    int32_t max_q, max_length, window, causal, dtype;
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

__device__ __attribute__((always_inline)) inline float load_value(const uint8_t *x, int i, int dtype)
{
    if (dtype == NVFP4_F32)
        return ((const float *)x)[i];
    const uint16_t v = ((const uint16_t *)x)[i];
    return dtype == NVFP4_BF16 ? __builtin_bit_cast(float, (uint32_t)v << 16) : (float)__builtin_bit_cast(_Float16, v);
}

__device__ __attribute__((always_inline)) inline void store_value(uint8_t *c, int64_t i, float v, int dtype)
{
    if (dtype == NVFP4_F32)
        ((float *)c)[i] = v;
    else
        ((uint16_t *)c)[i] = dtype == NVFP4_BF16 ? (uint16_t)bf16_bits(v) : f16_bits(v);
}

__global__ __launch_bounds__(64) void nvfp4_attention_simple_kernel(AttParams p)
{
    const int lane = (int)threadIdx.x;
    const int h = (int)(blockIdx.x % (uint32_t)p.H), i = (int)(blockIdx.x / (uint32_t)p.H % (uint32_t)p.max_q),
              b = (int)(blockIdx.x / (uint32_t)p.H / (uint32_t)p.max_q);
    const Sequence s = sequence_of(p, b);
    if (i >= s.n)
        return;
    const int32_t pos = s.length - s.n + i;
    const int32_t end = p.causal ? min(s.length, pos + 1) : s.length;
    const int32_t begin = p.window ? max(0, pos - p.window + 1) : 0;
    const uint8_t *x = p.q + (int64_t)(s.first + i) * p.q_token + (int64_t)h * p.q_head;
    float q[4], acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    bool finite = true;
    for (int e = 0; e < 4; ++e) {
        const int d = 2 * (lane + e / 2 * 64) + e % 2;
        q[e] = d < p.D ? load_value(x, d, p.dtype) : 0.0f;
        finite &= __builtin_isfinite(q[e]);
    }
    finite = __ballot(finite) == ~0ull;
    const float factor = p.scale * (p.gk ? *p.gk : 1.0f), gv = p.gv ? *p.gv : 1.0f;
    float top = -__builtin_inff(), sum = 0.0f;
    bool any = false;
    for (int32_t t = begin; t < end; ++t) {
        const uint32_t page = (uint32_t)p.table[(int64_t)b * p.width + (t >> p.shift)];
        if (page >= (uint32_t)p.pages)
            continue;
        const int64_t row = ((int64_t)(h / p.G) << p.shift) + (t & ((1 << p.shift) - 1));
        const uint8_t *kc = p.kc + page * p.code_page + row * (p.D / 2), *ks = p.ks + page * p.scale_page + row * (p.D / 16);
        const uint8_t *vc = p.vc + page * p.code_page + row * (p.D / 2), *vs = p.vs + page * p.scale_page + row * (p.D / 16);
        float dot = 0.0f, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int e = 0; e < 2; ++e) {
            const int at = lane + e * 64;
            if (2 * at < p.D) {
                const half2_t k2 = fp4x2<0>(kc[at]), v2 = fp4x2<0>(vc[at]);
                const float sk = __builtin_amdgcn_cvt_f32_fp8((int)ks[at / 8], 0), sv = __builtin_amdgcn_cvt_f32_fp8((int)vs[at / 8], 0);
                dot += q[2 * e] * ((float)k2.x * sk) + q[2 * e + 1] * ((float)k2.y * sk);
                v[2 * e] = (float)v2.x * sv;
                v[2 * e + 1] = (float)v2.y * sv;
            }
        }
        for (int d = 1; d < 64; d <<= 1)
            dot += __shfl_xor(dot, d);
        const float logit = dot * factor, above = fmaxf(top, logit);
        const float keep = any ? expf(top - above) : 0.0f, w = expf(logit - above);
        sum = sum * keep + w;
        for (int e = 0; e < 4; ++e)
            acc[e] = acc[e] * keep + w * v[e];
        top = above;
        any = true;
    }
    const int64_t row = (int64_t)(s.first + i) * p.H + h;
    for (int e = 0; e < 4; ++e) {
        const int d = 2 * (lane + e / 2 * 64) + e % 2;
        if (d < p.D)
            store_value(p.out, row * p.D + d, !any ? 0.0f : finite ? acc[e] / sum * gv : __builtin_nanf(""), p.dtype);
    }
    if (p.lse && lane == 0)
        p.lse[row] = !any ? -__builtin_inff() : finite ? top + logf(sum) : __builtin_nanf("");
}

// ------------------------------------------------------------------ host

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
        a->max_q > T || a->max_q > most / B || a->max_length < 1 || a->max_length > most)
        return NVFP4_ERR_INVALID_SHAPE;
    if (a->window < 0 || a->window > INT32_MAX || (a->causal != 0 && a->causal != 1))
        return NVFP4_ERR_INVALID_CACHE;
    if (!std::isfinite(a->scale))
        return NVFP4_ERR_INVALID_SCALE;
    if (a->q_token_stride < 0 || a->q_head_stride < 0 || a->q_token_stride >= kMaxStride || a->q_head_stride >= kMaxStride)
        return NVFP4_ERR_INVALID_STRIDE;
    return NVFP4_OK;
}

} // namespace

extern "C" {

size_t nvfp4_cache_attention_workspace_bytes(const nvfp4_cache_t *cache, int dtype, int64_t T, int64_t H, int64_t B,
                                             const nvfp4_attention_t *attention)
{
    return 0;
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
    p.code_page = cache->code_page_stride, p.scale_page = cache->scale_page_stride;
    p.T = (int32_t)T, p.H = (int32_t)H, p.B = (int32_t)B, p.width = (int32_t)table_width, p.pages = (int32_t)cache->pages;
    p.shift = __builtin_ctzll((uint64_t)cache->page_size);
    p.heads = (int32_t)cache->heads, p.G = (int32_t)(H / cache->heads), p.D = (int32_t)cache->head_size;
    p.max_q = (int32_t)attention->max_q, p.max_length = (int32_t)attention->max_length;
    p.window = (int32_t)attention->window, p.causal = attention->causal, p.dtype = dtype, p.scale = attention->scale;
    if (B * attention->max_q > kMaxGrid / H)
        return NVFP4_ERR_INVALID_SHAPE;
    hipLaunchKernelGGL(nvfp4_attention_simple_kernel, dim3((uint32_t)(B * attention->max_q * H)), dim3(64), 0,
                       (hipStream_t)stream, p);
    const hipError_t e = hipGetLastError();
    if (e == hipSuccess)
        return NVFP4_OK;
    nvfp4_record_hip_error((int)e);
    return NVFP4_ERR_HIP;
}

} // extern "C"
