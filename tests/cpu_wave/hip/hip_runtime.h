// The part of HIP that the kernels of nvfp4_moe.hip, nvfp4_quantize.hip,
// nvfp4_gemm.hip, nvfp4_rope.hip, nvfp4_cache.hip and nvfp4_attention.hip use, on the CPU, so that a test runs the sources themselves,
// launches included, on memory whose ends it guards.
// One workgroup at a time; each thread is a coroutine with a stack of its own.
// Cross-lane operations and barriers switch to the next thread until all of the
// wave (the workgroup) are there; threads that wait for one that has returned end
// the program with an error. Of inline assembly, the copies from global memory to
// LDS and the waits for them are carried out: a copy lands at once (`lazy` false) or
// not before a wait asks for it. With `lockstep` assembly is a meeting of the wave
// too, for sources whose lanes read what others have copied.
#ifndef CPU_WAVE_HIP_RUNTIME_H
#define CPU_WAVE_HIP_RUNTIME_H

#include <setjmp.h>
#include <sys/mman.h>
#include <ucontext.h>

#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <functional>
#include <type_traits>
#include <vector>

#define __device__
#define __global__
#define __launch_bounds__(...)
#define __shared__ thread_local     // static, and one OS thread runs all
// asm(..): register constraints only. asm volatile(..): its text, and the operands
// of a copy by the names that the copies have
#define asm(...)
#define volatile(...) (""); cpu_wave::assembly(#__VA_ARGS__, base, off, dst)
inline const int base = 0, off = 0, dst = 0;

struct dim3 {
    uint32_t x;
    dim3(int64_t n) : x((uint32_t)n) {}
};
typedef void *hipStream_t;
typedef int hipError_t;
constexpr hipError_t hipSuccess = 0;
inline hipError_t hipGetLastError() { return hipSuccess; }

// ------------------------------------------------------------------ threads

struct CpuWaveIndex {
    uint32_t x;
};
inline CpuWaveIndex threadIdx, blockIdx, gridDim;

namespace cpu_wave {

constexpr int kMaxThreads = 1024;
constexpr size_t kStack = 256 << 10;

// Arrivals at cross-lane operations of a wave, or at barriers of the workgroup:
// n threads pass the i-th when i * n have arrived.
struct Meeting {
    uint64_t arrived;
    uint64_t slots[2][64];
};
struct Thread {
    ucontext_t context;                 // its start; then its place (no system call to change to it)
    jmp_buf place;
    bool started, done;
    uint64_t wave_ops, barriers;        // how many this thread has arrived at
    const Meeting *at;                  // waits there until `until` have arrived
    uint64_t until;
    std::vector<struct Copy> copies;    // not landed yet, in order
};
// One lane's part of a copy from global memory to LDS.
struct Copy {
    uint8_t bytes[16], *to;
    size_t n;
};
inline Thread threads[kMaxThreads];
inline Meeting waves[kMaxThreads / 64], workgroup;
inline ucontext_t scheduler_start;
inline jmp_buf scheduler;
inline int threads_n;
inline uint8_t *stacks;
inline const std::function<void()> *body;
inline bool lazy, lockstep;
inline uint8_t *lds_start;              // dynamic LDS of the launches: set by the program
inline size_t lds_bytes;
inline std::vector<const char *> launched;      // kernels, in order

inline void yield()
{
    if (!_setjmp(threads[threadIdx.x].place))
        _longjmp(scheduler, 1);
}
inline void resume(Thread &t)
{
    if (_setjmp(scheduler))
        return;
    if (t.started)
        _longjmp(t.place, 1);
    t.started = true;
    swapcontext(&scheduler_start, &t.context);
}

inline void meet(Meeting &m, uint64_t &count, int n)
{
    Thread &t = threads[threadIdx.x];
    ++m.arrived;
    t.until = ++count * n;
    t.at = &m;
    if (m.arrived < t.until)
        yield();
}

// Every lane's value of 8 bytes or less; index i of the result is lane i's. Two
// buffers in turn: a lane arrives at the next operation when it has read this one's.
inline const uint64_t *exchange(uint64_t v)
{
    Thread &t = threads[threadIdx.x];
    Meeting &m = waves[threadIdx.x / 64];
    uint64_t *buffer = m.slots[t.wave_ops % 2];
    buffer[threadIdx.x % 64] = v;
    meet(m, t.wave_ops, 64);
    return buffer;
}

template <typename T>
T from(T v, int lane)
{
    uint64_t bits = 0;
    memcpy(&bits, &v, sizeof v);
    const uint64_t *all = exchange(bits);
    memcpy(&v, &all[lane & 63], sizeof v);
    return v;
}

[[noreturn]] inline void fail(const char *what)
{
    fprintf(stderr, "%s (workgroup %u, thread %u)\n", what, blockIdx.x, threadIdx.x);
    exit(3);
}

// Lets copies land until at most n are out.
inline void wait_copies(size_t n)
{
    std::vector<Copy> &c = threads[threadIdx.x].copies;
    size_t landed = 0;
    for (; c.size() - landed > n; ++landed)
        memcpy(c[landed].to, c[landed].bytes, c[landed].n);
    c.erase(c.begin(), c.begin() + landed);
}

template <typename A, typename B, typename C>
void assembly(const char *text, A from, B offset, C to)
{
    if (lockstep)
        exchange(0);
    if (const char *w = strstr(text, "vmcnt("))
        wait_copies((size_t)atoi(w + 6));
    if constexpr (std::is_same_v<A, const uint8_t *>) {
        const char *name = strstr(text, "global_load_lds_");
        if (!name)
            fail("assembly that is not known");
        Copy c{};
        const size_t lane = threadIdx.x % 64;
        c.n = !strncmp(name + 16, "dwordx4", 7) ? 16 : !strncmp(name + 16, "ushort", 6) ? 2 : 4;
        const size_t at = (uint32_t)(to - (uint32_t)(uintptr_t)lds_start) + lane * (c.n == 16 ? 16 : 4);
        if (at + c.n > lds_bytes)
            fail("a copy outside of LDS");
        memcpy(c.bytes, from + offset, c.n);
        c.to = lds_start + at;
        threads[threadIdx.x].copies.push_back(c);
        if (!lazy)
            wait_copies(0);
    }
}

inline void entry()
{
    (*body)();
    if (!threads[threadIdx.x].copies.empty())
        fail("a thread ended before its copies landed");
    threads[threadIdx.x].done = true;
    for (;;)
        yield();
}

inline void run_workgroup(int n, const std::function<void()> &f)
{
    if (!stacks)
        stacks = (uint8_t *)mmap(nullptr, kMaxThreads * kStack, PROT_READ | PROT_WRITE, MAP_PRIVATE | MAP_ANONYMOUS, -1, 0);
    body = &f;
    threads_n = n;
    workgroup = {};
    for (int t = 0; t < n; ++t) {
        Thread &th = threads[t];
        if (t % 64 == 0)
            waves[t / 64] = {};
        th.copies.clear();
        th.started = th.done = false;
        th.wave_ops = th.barriers = th.until = 0;
        th.at = &workgroup;
        getcontext(&th.context);
        th.context.uc_stack.ss_sp = stacks + t * kStack;
        th.context.uc_stack.ss_size = kStack;
        th.context.uc_link = nullptr;
        makecontext(&th.context, entry, 0);
    }
    for (int left = n; left;) {
        bool any = false;
        for (int t = 0; t < n; ++t) {
            if (threads[t].done || threads[t].at->arrived < threads[t].until)
                continue;
            any = true;
            threadIdx.x = (uint32_t)t;
            resume(threads[t]);
            left -= threads[t].done;
        }
        if (!any) {
            fprintf(stderr, "%d threads wait for ones that have returned\n", left);
            exit(3);
        }
    }
}

// The kernel's dynamic LDS holds NaN codes and scales (0x7F) where a workgroup starts.
template <typename K, typename... A>
void launch(K kernel, const char *name, dim3 grid, dim3 block, size_t lds, A... args)
{
    launched.push_back(name);
    gridDim.x = grid.x;
    lds_bytes = lds;
    const std::function<void()> f = [&] { kernel(args...); };
    for (uint32_t b = 0; b < grid.x; ++b) {
        blockIdx.x = b;
        if (lds_start)
            memset(lds_start, 0x7F, lds);
        run_workgroup((int)block.x, f);
    }
}

} // namespace cpu_wave

#define hipLaunchKernelGGL(kernel, grid, block, lds, stream, ...) \
    ((void)(stream), cpu_wave::launch(kernel, __PRETTY_FUNCTION__, grid, block, lds, __VA_ARGS__))

// ------------------------------------------------------------------ device functions

inline void __syncthreads()
{
    cpu_wave::meet(cpu_wave::workgroup, cpu_wave::threads[threadIdx.x].barriers, cpu_wave::threads_n);
}

template <typename T>
T __shfl_xor(T v, int d) { return cpu_wave::from(v, (int)(threadIdx.x % 64) ^ d); }
template <typename T>
T __shfl(T v, int lane) { return cpu_wave::from(v, lane); }
template <typename T>
T __shfl_up(T v, int d)
{
    const int lane = (int)(threadIdx.x % 64);
    return cpu_wave::from(v, lane >= d ? lane - d : lane);
}
template <typename T>
T __shfl_down(T v, int d)
{
    const int lane = (int)(threadIdx.x % 64);
    return cpu_wave::from(v, lane + d < 64 ? lane + d : lane);
}
inline uint64_t __ballot(bool one)
{
    const uint64_t *all = cpu_wave::exchange(one);
    uint64_t m = 0;
    for (int i = 0; i < 64; ++i)
        m |= all[i] << i;
    return m;
}
inline int __ffsll(unsigned long long v) { return __builtin_ffsll((long long)v); }
inline int __popcll(unsigned long long v) { return __builtin_popcountll(v); }
inline int atomicAdd(int *p, int v) { return (*p += v) - v; }
inline uint32_t atomicOr(uint32_t *p, uint32_t v)
{
    const uint32_t was = *p;
    *p |= v;
    return was;
}
inline float __expf(float v) { return expf(v); }

template <typename A, typename B>
std::common_type_t<A, B> min(A a, B b) { return b < a ? b : a; }
template <typename A, typename B>
std::common_type_t<A, B> max(A a, B b) { return a < b ? b : a; }

// the controls that the sources use; all rows and banks on, no lane reads outside its 16
inline int cpu_wave_dpp(int, int v, int ctrl, int, int, bool)
{
    const int lane = (int)(threadIdx.x % 64), row = lane & ~15, l = lane & 15;
    int src = -1;
    if (ctrl >= 0x121 && ctrl <= 0x12F)         // row_ror
        src = (l - (ctrl - 0x120)) & 15;
    else if (ctrl < 0x100)                      // quad_perm
        src = (l & ~3) | (ctrl >> (2 * (l & 3)) & 3);
    else if (ctrl >= 0x101 && ctrl <= 0x10F)    // row_shl: from the lane above
        src = l + (ctrl - 0x100) < 16 ? l + (ctrl - 0x100) : -1;
    else if (ctrl >= 0x111 && ctrl <= 0x11F)    // row_shr
        src = l - (ctrl - 0x110);
    else if (ctrl == 0x140)                     // row_mirror
        src = 15 - l;
    else if (ctrl == 0x141)                     // row_half_mirror
        src = (l & 8) | (7 - (l & 7));
    else {
        fprintf(stderr, "DPP control %#x\n", ctrl);
        exit(3);
    }
    const int got = cpu_wave::from(v, row | (src < 0 ? 0 : src));
    return src < 0 ? 0 : got;
}
inline int cpu_wave_first(int v) { return cpu_wave::from(v, 0); }

// ------------------------------------------------------------------ formats and the matrix instruction

typedef _Float16 cpu_wave_half2 __attribute__((ext_vector_type(2)));
typedef _Float16 cpu_wave_half8 __attribute__((ext_vector_type(8)));
typedef float cpu_wave_float16 __attribute__((ext_vector_type(16)));

inline float cpu_wave_fp4(uint32_t code)
{
    const float size[8] = {0.0f, 0.5f, 1.0f, 1.5f, 2.0f, 3.0f, 4.0f, 6.0f};
    return code & 8 ? -size[code & 7] : size[code & 7];
}
inline float cpu_wave_fp8(uint32_t code)
{
    const int e = (int)(code >> 3) & 15, m = (int)code & 7;
    const float size = e == 15 && m == 7 ? NAN : e ? ldexpf(8 + m, e - 10) : ldexpf(m, -9);
    return code & 0x80 ? -size : size;
}
// nearest code of a table that rises, ties to the even one
template <typename F>
uint32_t cpu_wave_nearest(float size, uint32_t n, F value)
{
    for (uint32_t c = 0; c + 1 < n; ++c) {
        const float middle = 0.5f * (value(c) + value(c + 1));
        if (size < middle || (size == middle && c % 2 == 0))
            return c;
    }
    return n - 1;
}
inline uint32_t cpu_wave_to_fp8(float v)
{
    return v != v ? 0x7Fu : (cpu_wave_nearest(fabsf(v), 127, cpu_wave_fp8) | (std::signbit(v) ? 0x80u : 0u));
}
inline uint32_t cpu_wave_to_fp4(float v)
{
    return cpu_wave_nearest(fabsf(v), 8, cpu_wave_fp4) | (std::signbit(v) ? 8u : 0u);
}
inline cpu_wave_half2 cpu_wave_h2_of_fp4(uint32_t w, float, int byte)
{
    return {(_Float16)cpu_wave_fp4(w >> (8 * byte) & 15), (_Float16)cpu_wave_fp4(w >> (8 * byte + 4) & 15)};
}
inline cpu_wave_half2 cpu_wave_h2_of_fp8(uint32_t w, float, bool high)
{
    w >>= high ? 16 : 0;
    return {(_Float16)cpu_wave_fp8(w & 255), (_Float16)cpu_wave_fp8(w >> 8 & 255)};
}
inline int cpu_wave_fp8_of_f32(float a, float b, int old, bool high)
{
    const uint32_t both = cpu_wave_to_fp8(a) | cpu_wave_to_fp8(b) << 8;
    return (int)(high ? ((uint32_t)old & 0xFFFFu) | both << 16 : ((uint32_t)old & 0xFFFF0000u) | both);
}
inline uint32_t cpu_wave_fp4_of_f32(uint32_t old, float a, float b, float, int byte)
{
    return (old & ~(255u << (8 * byte))) | (cpu_wave_to_fp4(a) | cpu_wave_to_fp4(b) << 4) << (8 * byte);
}
inline int cpu_wave_frexp_exp(float v)
{
    int e = 0;
    if (std::isfinite(v))
        frexpf(v, &e);
    return e;
}
inline float cpu_wave_frexp_mant(float v)
{
    int e;
    return std::isfinite(v) ? frexpf(v, &e) : v;
}

// 32 x 32 x 16: lane l holds row (column) l % 32, k 8 (l / 32) .. + 7 of each operand;
// register r of its result is row 8 (r / 4) + 4 (l / 32) + r % 4 of column l % 32
inline cpu_wave_float16 cpu_wave_mfma(cpu_wave_half8 a, cpu_wave_half8 b, cpu_wave_float16 c, int, int, int)
{
    static float rows[cpu_wave::kMaxThreads / 64][2][64][8], columns[cpu_wave::kMaxThreads / 64][2][64][8];
    const uint32_t wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    const uint32_t turn = cpu_wave::threads[threadIdx.x].wave_ops % 2;
    for (int k = 0; k < 8; ++k) {
        rows[wave][turn][lane][k] = a[k];
        columns[wave][turn][lane][k] = b[k];
    }
    cpu_wave::exchange(0);
    for (uint32_t r = 0; r < 16; ++r) {
        double sum = 0.0;
        for (uint32_t k = 0; k < 16; ++k)
            sum += (double)rows[wave][turn][8 * (r / 4) + 4 * (lane / 32) + r % 4 + 32 * (k / 8)][k % 8] *
                   (double)columns[wave][turn][lane % 32 + 32 * (k / 8)][k % 8];
        c[r] = (float)(c[r] + sum);
    }
    return c;
}

// 16 x 16 x 32: lane l holds row (column) l % 16, k 8 (l / 16) .. + 7 of each operand;
// register r of its result is row 4 (l / 16) + r of column l % 16
typedef float cpu_wave_float4 __attribute__((ext_vector_type(4)));
inline cpu_wave_float4 cpu_wave_mfma16(cpu_wave_half8 a, cpu_wave_half8 b, cpu_wave_float4 c, int, int, int)
{
    static float rows[cpu_wave::kMaxThreads / 64][2][64][8], columns[cpu_wave::kMaxThreads / 64][2][64][8];
    const uint32_t wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    const uint32_t turn = cpu_wave::threads[threadIdx.x].wave_ops % 2;
    for (int k = 0; k < 8; ++k) {
        rows[wave][turn][lane][k] = a[k];
        columns[wave][turn][lane][k] = b[k];
    }
    cpu_wave::exchange(0);
    for (uint32_t r = 0; r < 4; ++r) {
        double sum = 0.0;
        for (uint32_t k = 0; k < 32; ++k)
            sum += (double)rows[wave][turn][4 * (lane / 16) + r + 16 * (k / 8)][k % 8] *
                   (double)columns[wave][turn][lane % 16 + 16 * (k / 8)][k % 8];
        c[r] = (float)(c[r] + sum);
    }
    return c;
}

// halves (odd and even rows of 16) of two registers exchanged
typedef uint32_t cpu_wave_uint2 __attribute__((ext_vector_type(2)));
inline cpu_wave_uint2 cpu_wave_swap(uint32_t a, uint32_t b, uint32_t step)
{
    const uint32_t lane = threadIdx.x % 64;
    const bool low = !(lane & step);
    const uint32_t other = (uint32_t)cpu_wave::from(low ? b : a, (int)(lane ^ step));
    return low ? (cpu_wave_uint2){a, other} : (cpu_wave_uint2){other, b};
}

// Transposed reads of 8 bytes per lane among 16 lanes: 16 codes, of which lane i gets the i-th of
// each lane; 4 float16, of which lane i gets the (i % 4)-th of lanes i / 4 + 0, 4, 8, 12
typedef int cpu_wave_int2 __attribute__((ext_vector_type(2)));
typedef short cpu_wave_short4 __attribute__((ext_vector_type(4)));
template <typename P>
uint64_t cpu_wave_8_bytes(P p)
{
    uint64_t v;
    memcpy(&v, (const void *)(uintptr_t)p, 8);
    return v;
}
template <typename P>
cpu_wave_int2 cpu_wave_tr4(P p)
{
    const uint64_t *all = cpu_wave::exchange(cpu_wave_8_bytes(p));
    const uint32_t lane = threadIdx.x % 64, i = lane % 16;
    uint64_t v = 0;
    for (uint32_t n = 0; n < 16; ++n)
        v |= (all[lane - i + n] >> (4 * i) & 15) << (4 * n);
    return {(int)(uint32_t)v, (int)(uint32_t)(v >> 32)};
}
template <typename P>
cpu_wave_short4 cpu_wave_tr16(P p)
{
    const uint64_t *all = cpu_wave::exchange(cpu_wave_8_bytes(p));
    const uint32_t lane = threadIdx.x % 64, i = lane % 16;
    cpu_wave_short4 v;
    for (uint32_t n = 0; n < 4; ++n)
        v[n] = (short)(all[lane - i + 4 * n + i / 4] >> (16 * (i % 4)));
    return v;
}

inline void cpu_wave_s_waitcnt(int imm)
{
    cpu_wave::exchange(0);
    cpu_wave::wait_copies((size_t)((imm & 15) | (imm >> 14 & 3) << 4));
}

#define __builtin_amdgcn_update_dpp cpu_wave_dpp
#define __builtin_amdgcn_readlane(v, lane) cpu_wave::from((int)(v), lane)
#define __builtin_amdgcn_readfirstlane(v) cpu_wave_first((int)(v))
#define __builtin_amdgcn_fence(...) ((void)0)
#define __builtin_amdgcn_wave_barrier() ((void)cpu_wave::exchange(0))
#define __builtin_amdgcn_s_setprio(priority) ((void)0)
#define __builtin_amdgcn_rcpf(v) (1.0f / (v))
#define __builtin_amdgcn_cvt_scalef32_pk_f16_fp4 cpu_wave_h2_of_fp4
#define __builtin_amdgcn_cvt_scalef32_pk_f16_fp8 cpu_wave_h2_of_fp8
#define __builtin_amdgcn_cvt_scalef32_pk_fp4_f32 cpu_wave_fp4_of_f32
#define __builtin_amdgcn_cvt_f32_fp8(v, byte) cpu_wave_fp8((uint32_t)(v) >> (8 * (byte)) & 255)
#define __builtin_amdgcn_cvt_pk_fp8_f32 cpu_wave_fp8_of_f32
#define __builtin_amdgcn_frexp_mantf cpu_wave_frexp_mant
#define __builtin_amdgcn_frexp_expf cpu_wave_frexp_exp
#define __builtin_amdgcn_mfma_f32_32x32x16_f16 cpu_wave_mfma
#define __builtin_amdgcn_mfma_f32_16x16x32_f16 cpu_wave_mfma16
#define __builtin_amdgcn_ds_read_tr4_b64_v2i32 cpu_wave_tr4
#define __builtin_amdgcn_ds_read_tr16_b64_v4i16 cpu_wave_tr16
#define __builtin_amdgcn_permlane32_swap(a, b, f, c) cpu_wave_swap(a, b, 32)
#define __builtin_amdgcn_permlane16_swap(a, b, f, c) cpu_wave_swap(a, b, 16)
#define __builtin_amdgcn_exp2f(v) exp2f(v)
#define __builtin_amdgcn_logf(v) log2f(v)
#define __builtin_amdgcn_s_waitcnt cpu_wave_s_waitcnt
#define __builtin_amdgcn_s_barrier __syncthreads

// one thread runs at a time
#define __HIP_MEMORY_SCOPE_AGENT 0
#define __hip_atomic_fetch_add(p, v, order, scope) ((*(p) += (v)) - (v))
#define __hip_atomic_store(p, v, order, scope) ((void)(*(p) = (v)))
#define __hip_atomic_load(p, order, scope) (*(p))
template <typename T>
T cpu_wave_replace(T *p, T v)
{
    const T was = *p;
    *p = v;
    return was;
}
#define __hip_atomic_exchange(p, v, order, scope) cpu_wave_replace(p, v)
#define __hip_atomic_fetch_max(p, v, order, scope) cpu_wave_replace(p, max(*(p), v))

// float32 -> bfloat16, nearest, ties to even (the C library here has none)
extern "C" inline __bf16 __truncsfbf2(float v)
{
    uint32_t w;
    memcpy(&w, &v, 4);
    const uint16_t h = v != v ? (uint16_t)(w >> 16 | 0x40) : (uint16_t)((w + 0x7FFF + (w >> 16 & 1)) >> 16);
    __bf16 r;
    memcpy(&r, &h, 2);
    return r;
}

#endif
