// The part of HIP that the kernels of nvfp4_moe.hip use, on the CPU, so that a
// test runs the source itself, launches included, on memory whose ends it guards.
// One workgroup at a time; each thread is a coroutine with a stack of its own.
// Cross-lane operations and barriers switch to the next thread until all of the
// wave (the workgroup) are there; threads that wait for one that has returned end
// the program with an error.
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

#define __device__
#define __global__
#define __launch_bounds__(...)
#define __shared__ thread_local     // static, and one OS thread runs all
#define asm(...)                    // register constraints only

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
};
inline Thread threads[kMaxThreads];
inline Meeting waves[kMaxThreads / 64], workgroup;
inline ucontext_t scheduler_start;
inline jmp_buf scheduler;
inline int threads_n;
inline uint8_t *stacks;
inline const std::function<void()> *body;

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

inline void entry()
{
    (*body)();
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

template <typename K, typename... A>
void launch(K kernel, dim3 grid, dim3 block, A... args)
{
    gridDim.x = grid.x;
    const std::function<void()> f = [&] { kernel(args...); };
    for (uint32_t b = 0; b < grid.x; ++b) {
        blockIdx.x = b;
        run_workgroup((int)block.x, f);
    }
}

} // namespace cpu_wave

#define hipLaunchKernelGGL(kernel, grid, block, lds, stream, ...) \
    ((void)(lds), (void)(stream), cpu_wave::launch(kernel, grid, block, __VA_ARGS__))

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

template <int N>
using cpu_wave_halves = _Float16 __attribute__((ext_vector_type(N)));
inline cpu_wave_halves<2> cpu_wave_no_conversion(uint32_t, float, int)
{
    fprintf(stderr, "conversion not written here\n");
    exit(3);
}

#define __builtin_amdgcn_update_dpp cpu_wave_dpp
#define __builtin_amdgcn_readlane(v, lane) cpu_wave::from((int)(v), lane)
#define __builtin_amdgcn_readfirstlane(v) cpu_wave_first((int)(v))
#define __builtin_amdgcn_fence(...) ((void)0)
#define __builtin_amdgcn_wave_barrier() ((void)cpu_wave::exchange(0))
#define __builtin_amdgcn_rcpf(v) (1.0f / (v))
#define __builtin_amdgcn_cvt_scalef32_pk_f16_fp4 cpu_wave_no_conversion
#define __builtin_amdgcn_cvt_scalef32_pk_f16_fp8 cpu_wave_no_conversion
#define __HIP_MEMORY_SCOPE_AGENT 0
#define __hip_atomic_fetch_add(p, v, order, scope) ((*(p) += (v)) - (v))

#endif
