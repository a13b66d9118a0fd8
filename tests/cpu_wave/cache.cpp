// Runs the library's cache write and read (source and launches) on the CPU, on guarded memory.
//   cache <in> <out>
// in, 4-byte words: dtype T pages page_size heads D token_stride head_stride, code_gap scale_gap
// (bytes between pages), k_scale, v_scale (float32); then slots (int64 [T]), k, v: as many elements
// as the strides reach
// out: the four arrays of the cache with their gaps (0xA5 where nothing was written), k and v read back
#include "nvfp4_cache.hip"

#include "guarded.h"

void nvfp4_record_hip_error(int) {}

int main(int argc, char **argv)
{
    if (argc != 3)
        return 5;
    guarded::Input in(argv[1]);
    FILE *out = fopen(argv[2], "wb");
    int32_t w[10];
    in.read(w, sizeof w);
    float g[2];
    in.read(g, sizeof g);
    const int dtype = w[0];
    const int64_t T = w[1], pages = w[2], ps = w[3], H = w[4], D = w[5];
    const size_t size = dtype == NVFP4_F32 ? 4 : 2;
    const auto slots = in.bytes(8 * T);
    const size_t reach = (size_t)((T - 1) * w[6] + (H - 1) * w[7] + D) * size;
    const auto k = in.bytes(reach), v = in.bytes(reach);
    const int64_t code = H * ps * D / 2 + w[8], scale = H * ps * D / 16 + w[9];
    std::vector<uint8_t> first;
    for (int turn = 0; turn < 2; ++turn) {
        const bool at_start = turn;
        auto room = [&](size_t n, size_t align) {
            uint8_t *p = guarded::make(n, align, at_start);
            memset(p, 0xA5, n);
            return p;
        };
        const size_t codes_n = (pages - 1) * code + H * ps * D / 2, scales_n = (pages - 1) * scale + H * ps * D / 16;
        uint8_t *a[4] = {room(codes_n, 16), room(scales_n, 16), room(codes_n, 16), room(scales_n, 16)};
        float *gs[2];
        for (int i = 0; i < 2; ++i)
            *(gs[i] = (float *)guarded::make(4, 4, at_start)) = g[i];
        const nvfp4_cache_t cache = {a[0], a[1], a[2], a[3], gs[0], gs[1], pages, ps, H, D, code, scale};
        const int64_t *at = (const int64_t *)guarded::copy(slots, 8, at_start);
        uint8_t *ko = room(T * H * D * size, size), *vo = room(T * H * D * size, size);
        if (nvfp4_cache_write(&cache, guarded::copy(k, size, at_start), guarded::copy(v, size, at_start), dtype, at, T, w[6], w[7], w[6],
                              w[7], nullptr) != NVFP4_OK ||
            nvfp4_cache_read(&cache, ko, vo, dtype, at, T, nullptr) != NVFP4_OK)
            return 6;
        std::vector<uint8_t> got;
        for (int i = 0; i < 4; ++i)
            got.insert(got.end(), a[i], a[i] + (i % 2 ? scales_n : codes_n));
        got.insert(got.end(), ko, ko + T * H * D * size);
        got.insert(got.end(), vo, vo + T * H * D * size);
        if (turn && got != first)
            return 8;
        first = got;
    }
    fwrite(first.data(), 1, first.size(), out);
    return fclose(out) ? 5 : 0;
}
