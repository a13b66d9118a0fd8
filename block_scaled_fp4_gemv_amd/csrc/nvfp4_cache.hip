// Keys and values of new tokens into the pages of an NVFP4 cache, and rows of the
// cache back as values, on MI355X (gfx950).
//
// A row (one token, one head) is D / 16 blocks of 16 values, quantised exactly as
// nvfp4_quantize does with the cache's global scale (nvfp4_quantize_device.h). A thread
// has one block: 16 values, 8 bytes of codes, 1 byte of scale; neighbours have the
// neighbouring blocks of a row, then the next token of the same head, which mostly lies next in the
// page, for a run of 16 tokens, then the next head: whole lines on both sides, and the rows that
// are at work at once lie together (head by head over all tokens they were 2 KiB apart: 43 us for 38).
// Keys and values in one launch.
// What bounds it: HBM, every byte read and written once; small calls the launch. 8 heads of 128: 16384 tokens
// written from bfloat16 and read back 38 to 43 us (36 at a copy's 4.8 TB/s), 32768 read as float16 46 us, 3.8 TB/s.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <initializer_list>
#include <type_traits>

#include "nvfp4_device.h"
#include "nvfp4_gemv.h"
#include "nvfp4_internal.h"
#include "nvfp4_quantize_device.h"

namespace {

constexpr int kThreads = 256, kBlocks = 4, kRun = 4;
constexpr int64_t kManyBlocks = 1 << 20;         // of keys (of values): 16 waves of single blocks on every CU
constexpr int64_t kMaxStride = INT64_C(1) << 40, kMaxPage = INT64_C(1) << 32;

struct RowParams {
    uint8_t *codes[2], *scales[2];              // keys, values
    const float *global[2];
    const uint8_t *in[2];
    uint8_t *out[2];
    const int64_t *slots;
    int64_t in_token[2], in_head[2];            // bytes
    int64_t code_page, scale_page, all_slots;
    Divisor heads, blocks;                      // blocks of a row
    uint32_t tokens, run;                       // runs of 1 << run tokens
    int32_t shift, nkb;                       // page_size = 1 << shift
    uint32_t wgs;                               // for the keys
};

// A block: 0 keys, 1 values; token, head, block of the row. False past the end.
struct Place {
    uint32_t which, t, h, kb;
    bool real;
};

// The k-th block of a thread of U.
template <int U>
__device__ __attribute__((always_inline)) inline Place place_of(const RowParams &p, int k)
{
    Place at;
    at.which = blockIdx.x >= p.wgs;
    // the grid keeps every index of a block below 2^31
    const uint32_t i = ((blockIdx.x - (at.which ? p.wgs : 0u)) * U + k) * kThreads + threadIdx.x;
    const uint32_t row = divided(i, p.blocks);
    at.kb = i - row * p.blocks.d;
    const uint32_t run = row >> p.run, run_t = divided(run, p.heads);
    at.h = run - run_t * p.heads.d;
    at.t = (run_t << p.run) + (row & ((1u << p.run) - 1u));
    at.real = at.t < p.tokens;
    return at;
}

// Byte offsets of a slot's block in codes and scales; the slot is inside the cache.
__device__ __attribute__((always_inline)) inline void offsets_of(const RowParams &p, int64_t slot, const Place &at,
                                                                 int64_t &code, int64_t &scale)
{
    const int64_t page = slot >> p.shift, in_page = slot & ((1 << p.shift) - 1);
    const int64_t row = ((int64_t)at.h << p.shift) + in_page;
    code = page * p.code_page + (row * p.nkb + at.kb) * 8;
    scale = page * p.scale_page + row * p.nkb + at.kb;
}

// U blocks a thread: their slots are all loaded before the first is used.
template <int DT, int U>
__global__ __launch_bounds__(kThreads) void nvfp4_cache_write_kernel(RowParams p)
{
    Place at[U];
    int64_t slot[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        at[k] = place_of<U>(p, k);
        slot[k] = at[k].real ? p.slots[at[k].t] : -1;
    }
    const uint32_t which = at[0].which;
    const Global gl = global_of(p.global[which]);
#pragma unroll
    for (int k = 0; k < U; ++k) {
        if ((uint64_t)slot[k] >= (uint64_t)p.all_slots)
            continue;
        const uint8_t *x = (which ? p.in[1] + at[k].t * p.in_token[1] + at[k].h * p.in_head[1]
                                  : p.in[0] + at[k].t * p.in_token[0] + at[k].h * p.in_head[0]) + at[k].kb * 16 * kSize<DT>;
        uint32_t s;
        const uint2_t q = quantize_block<DT>(x, gl, s);
        int64_t code, scale;
        offsets_of(p, slot[k], at[k], code, scale);
        *(uint2_t *)(p.codes[which] + code) = q;
        p.scales[which][scale] = (uint8_t)s;
    }
}

// Rows of slots outside the cache are zeros. U blocks a thread, loaded together.
template <int DT, int U>
__global__ __launch_bounds__(kThreads) void nvfp4_cache_read_kernel(RowParams p)
{
    Place at[U];
    int64_t slot[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        at[k] = place_of<U>(p, k);
        slot[k] = at[k].real ? p.slots[at[k].t] : -1;
    }
    const uint32_t which = at[0].which;
    const float *gp = p.global[which];
    const float g = gp ? *gp : 1.0f;
    uint2_t q[U];
    uint32_t scale[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        q[k] = (uint2_t){0u, 0u};
        scale[k] = 0u;
        if ((uint64_t)slot[k] < (uint64_t)p.all_slots) {
            int64_t code, sc;
            offsets_of(p, slot[k], at[k], code, sc);
            q[k] = *(const uint2_t *)(p.codes[which] + code);
            scale[k] = p.scales[which][sc];
        }
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
        // a slot outside: zeros whatever the global scale
        const bool there = (uint64_t)slot[k] < (uint64_t)p.all_slots;
        const float s = e4m3_value(scale[k]), by = there ? g : 0.0f;
        float v[16];
        const uint32_t w[2] = {q[k].x, q[k].y};
#pragma unroll
        for (int d = 0; d < 2; ++d) {
            const half2_t h[4] = {fp4x2<0>(w[d]), fp4x2<1>(w[d]), fp4x2<2>(w[d]), fp4x2<3>(w[d])};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[8 * d + 2 * j] = (float)h[j].x * s * by;
                v[8 * d + 2 * j + 1] = (float)h[j].y * s * by;
            }
        }
        if (at[k].real)
            store16<DT>(p.out[which] + (((int64_t)at[k].t * p.heads.d + at[k].h) * p.nkb + at[k].kb) * 16 * kSize<DT>, v);
    }
}

// ------------------------------------------------------------------ host

bool known_type(int dtype) { return dtype == NVFP4_F16 || dtype == NVFP4_BF16 || dtype == NVFP4_F32; }
bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// What both calls check and fill.
nvfp4_status_t rows_of(const nvfp4_cache_t *cache, const int64_t *slots, int64_t T, RowParams &p)
{
    const nvfp4_status_t st = nvfp4_check_cache(cache);
    if (st != NVFP4_OK)
        return st;
    const int64_t H = cache->heads, nkb = cache->head_size / 16;
    // blocks are counted below 2^31, with the tokens rounded up to runs and the workgroups to threads
    if (T < 1 || T > ((INT64_C(1) << 31) - 2048) / H / nkb - 64)
        return NVFP4_ERR_INVALID_SHAPE;
    if (!aligned(slots, 8))
        return NVFP4_ERR_MISALIGNED;
    p = {};
    p.codes[0] = (uint8_t *)cache->k_codes, p.codes[1] = (uint8_t *)cache->v_codes;
    p.scales[0] = (uint8_t *)cache->k_scales, p.scales[1] = (uint8_t *)cache->v_scales;
    p.global[0] = cache->k_scale, p.global[1] = cache->v_scale;
    p.slots = slots;
    p.code_page = cache->code_page_stride, p.scale_page = cache->scale_page_stride;
    p.all_slots = cache->pages * cache->page_size;
    p.shift = __builtin_ctzll((uint64_t)cache->page_size);
    p.nkb = (int32_t)nkb;
    p.tokens = (uint32_t)T, p.run = T >= 16 ? kRun : 0;
    p.heads = divisor_of((uint32_t)H), p.blocks = divisor_of((uint32_t)nkb);
    return NVFP4_OK;
}

nvfp4_status_t finish()
{
    const hipError_t e = hipGetLastError();
    if (e == hipSuccess)
        return NVFP4_OK;
    nvfp4_record_hip_error((int)e);
    return NVFP4_ERR_HIP;
}

// One block a thread where that does not fill the card, else kBlocks.
template <typename K>
void launch(K one, K several, RowParams &p, hipStream_t st)
{
    const int64_t runs = ((int64_t)p.tokens + (1 << p.run) - 1) >> p.run, blocks = ((runs * p.heads.d) << p.run) * p.nkb;
    const int each = blocks >= kManyBlocks ? kBlocks : 1;
    p.wgs = (uint32_t)((blocks + each * kThreads - 1) / (each * kThreads));
    hipLaunchKernelGGL((each == 1 ? one : several), dim3(2 * p.wgs), dim3(kThreads), 0, st, p);
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

nvfp4_status_t nvfp4_check_cache(const nvfp4_cache_t *c)
{
    if (!c || !c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales)
        return NVFP4_ERR_NULL_POINTER;
    const int64_t D = c->head_size, ps = c->page_size;
    if (c->pages < 1 || c->pages > INT32_MAX || c->heads < 1 || c->heads > 4096 || D < 32 || D > 256 || D % 32 || ps < 16 ||
        ps > 4096 || (ps & (ps - 1)))
        return NVFP4_ERR_INVALID_CACHE;
    const int64_t rows = c->heads * ps;                 // of a page; offsets in it are below 2^31
    if (rows * (D / 2) > INT32_MAX)
        return NVFP4_ERR_INVALID_CACHE;
    if (c->code_page_stride < rows * (D / 2) || c->scale_page_stride < rows * (D / 16) || c->code_page_stride % 16 ||
        c->scale_page_stride % 16 || c->code_page_stride >= kMaxPage || c->scale_page_stride >= kMaxPage)
        return NVFP4_ERR_INVALID_STRIDE;
    if (!aligned(c->k_codes, 16) || !aligned(c->k_scales, 16) || !aligned(c->v_codes, 16) || !aligned(c->v_scales, 16) ||
        (c->k_scale && !aligned(c->k_scale, 4)) || (c->v_scale && !aligned(c->v_scale, 4)))
        return NVFP4_ERR_MISALIGNED;
    return NVFP4_OK;
}

extern "C" {

nvfp4_status_t nvfp4_cache_write(const nvfp4_cache_t *cache, const void *k, const void *v, int dtype,
                                 const int64_t *slots, int64_t T, int64_t k_token_stride, int64_t k_head_stride,
                                 int64_t v_token_stride, int64_t v_head_stride, void *stream)
{
    if (!k || !v || !slots)
        return NVFP4_ERR_NULL_POINTER;
    if (!known_type(dtype))
        return NVFP4_ERR_INVALID_TYPE;
    RowParams p;
    const nvfp4_status_t st = rows_of(cache, slots, T, p);
    if (st != NVFP4_OK)
        return st;
    for (int64_t s : {k_token_stride, k_head_stride, v_token_stride, v_head_stride})
        if (s < 0 || s >= kMaxStride)
            return NVFP4_ERR_INVALID_STRIDE;
    const int64_t size = dtype == NVFP4_F32 ? 4 : 2;
    if (!aligned(k, size) || !aligned(v, size))
        return NVFP4_ERR_MISALIGNED;
    p.in[0] = (const uint8_t *)k, p.in[1] = (const uint8_t *)v;
    p.in_token[0] = k_token_stride * size, p.in_token[1] = v_token_stride * size;
    p.in_head[0] = k_head_stride * size, p.in_head[1] = v_head_stride * size;
    by_type(dtype, [&](auto dt) {
        launch(nvfp4_cache_write_kernel<dt(), 1>, nvfp4_cache_write_kernel<dt(), kBlocks>, p, (hipStream_t)stream);
    });
    return finish();
}

nvfp4_status_t nvfp4_cache_read(const nvfp4_cache_t *cache, void *k, void *v, int dtype, const int64_t *slots, int64_t T,
                                void *stream)
{
    if (!k || !v || !slots)
        return NVFP4_ERR_NULL_POINTER;
    if (!known_type(dtype))
        return NVFP4_ERR_INVALID_TYPE;
    RowParams p;
    const nvfp4_status_t st = rows_of(cache, slots, T, p);
    if (st != NVFP4_OK)
        return st;
    const int64_t size = dtype == NVFP4_F32 ? 4 : 2;
    if (!aligned(k, size) || !aligned(v, size))
        return NVFP4_ERR_MISALIGNED;
    p.out[0] = (uint8_t *)k, p.out[1] = (uint8_t *)v;
    by_type(dtype, [&](auto dt) {
        launch(nvfp4_cache_read_kernel<dt(), 1>, nvfp4_cache_read_kernel<dt(), kBlocks>, p, (hipStream_t)stream);
    });
    return finish();
}

} // extern "C"
