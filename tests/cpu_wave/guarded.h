// Memory whose end, or start, is where its mapping ends; a program's input and output.
#ifndef CPU_WAVE_GUARDED_H
#define CPU_WAVE_GUARDED_H

#include <sys/mman.h>

#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

namespace guarded {

// n bytes aligned to `align`; behind them (less than `align` further on), or before
// them with `at_start`, a page that is not mapped.
inline uint8_t *make(size_t n, size_t align, bool at_start)
{
    const size_t page = 4096, size = (n + page - 1) / page * page;
    uint8_t *p = (uint8_t *)mmap(nullptr, size + 2 * page, PROT_NONE, MAP_PRIVATE | MAP_ANONYMOUS, -1, 0);
    if (p == MAP_FAILED || mprotect(p + page, size, PROT_READ | PROT_WRITE))
        exit(4);
    return p + page + (at_start ? 0 : (size - n) / align * align);
}

struct Input {
    FILE *f;
    explicit Input(const char *name) : f(fopen(name, "rb"))
    {
        if (!f)
            exit(5);
    }
    void read(void *to, size_t n)
    {
        if (fread(to, 1, n, f) != n)
            exit(5);
    }
    template <typename T>
    T word()
    {
        T v;
        read(&v, sizeof v);
        return v;
    }
    std::vector<uint8_t> bytes(size_t n)
    {
        std::vector<uint8_t> v(n);
        read(v.data(), n);
        return v;
    }
};

// The bytes in guarded memory (null for none).
inline uint8_t *copy(const std::vector<uint8_t> &v, size_t align, bool at_start)
{
    if (v.empty())
        return nullptr;
    uint8_t *p = make(v.size(), align, at_start);
    memcpy(p, v.data(), v.size());
    return p;
}

} // namespace guarded

#endif
