// Copies from global memory straight into LDS, and packed codes to float16: shared by
// the products and attention. Internal header.
#ifndef NVFP4_LDS_H
#define NVFP4_LDS_H

#include <hip/hip_runtime.h>

#include <cstdint>

#include "nvfp4_device.h"

namespace {

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));

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
// count the copies: the kernels wait for them themselves. The forms with _s take
// a base that the compiler has in scalar registers, so lanes may be left out.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __attribute__((always_inline)) inline void copy16_s(const uint8_t *base, uint32_t off, uint32_t dst)
{
    asm volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_dwordx4 %0, %1" : : "v"(off), "s"(base), "s"(dst) : "memory", "m0");
}
__device__ __attribute__((always_inline)) inline void copy4_s(const uint8_t *base, uint32_t off, uint32_t dst)
{
    asm volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_dword %0, %1" : : "v"(off), "s"(base), "s"(dst) : "memory", "m0");
}
__device__ __attribute__((always_inline)) inline void copy16(const uint8_t *base, uint32_t off, uint32_t dst)
{
    copy16_s(uniform_ptr(base), off, dst);
}
__device__ __attribute__((always_inline)) inline void copy4(const uint8_t *base, uint32_t off, uint32_t dst)
{
    copy4_s(uniform_ptr(base), off, dst);
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

// 8 codes (a dword) times a scale -> 8 float16
__device__ __attribute__((always_inline)) inline half8_t decode8(uint32_t w, half2_t s)
{
    const half2_t v0 = fp4x2<0>(w) * s, v1 = fp4x2<1>(w) * s, v2 = fp4x2<2>(w) * s, v3 = fp4x2<3>(w) * s;
    return (half8_t){v0.x, v0.y, v1.x, v1.y, v2.x, v2.y, v3.x, v3.y};
}


// The same with a scale for each pair of neighbours: 4 half2 in `s`
__device__ __attribute__((always_inline)) inline half8_t decode8_by(uint32_t w, uint4_t s)
{
    const half2_t v0 = fp4x2<0>(w) * as_h2(s.x), v1 = fp4x2<1>(w) * as_h2(s.y), v2 = fp4x2<2>(w) * as_h2(s.z),
                  v3 = fp4x2<3>(w) * as_h2(s.w);
    return (half8_t){v0.x, v0.y, v1.x, v1.y, v2.x, v2.y, v3.x, v3.y};
}

// Transposed reads from LDS among 16 lanes. Each gives the address of 8 bytes: 16 codes, of
// which lane i gets code i of every lane in order; or 4 float16, of which lane i gets value
// i % 4 of lanes i / 4, 4 + i / 4, 8 + i / 4, 12 + i / 4 (so 4 rows of 16 become 16 columns of 4).
#define NVFP4_LDS __attribute__((address_space(3)))
typedef int int2_t __attribute__((ext_vector_type(2)));
typedef short short4_t __attribute__((ext_vector_type(4)));

__device__ __attribute__((always_inline)) inline uint2_t read_transposed4(const uint8_t *p)
{
    return __builtin_bit_cast(uint2_t, __builtin_amdgcn_ds_read_tr4_b64_v2i32((NVFP4_LDS int2_t *)p));
}
__device__ __attribute__((always_inline)) inline uint2_t read_transposed16(const uint8_t *p)
{
    return __builtin_bit_cast(uint2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((NVFP4_LDS short4_t *)p));
}

} // namespace

#endif
