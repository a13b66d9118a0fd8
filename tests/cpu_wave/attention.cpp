// Runs the library's attention over a paged cache (source and launches) on the CPU,
// on guarded memory.
//   attention <in> <out>
// in, 4-byte words: dtype T H B max_q max_length width pages page_size heads D window causal,
// scale, k_scale, v_scale (float32); then the cache's four arrays, q, offsets, lengths, table
// out: out (0xA5 where nothing was written), lse; stdout: the kernels launched
#include "nvfp4_attention.hip"

#include "guarded.h"

namespace {
thread_local __attribute__((aligned(16))) uint8_t lds[160 << 10];
}

void nvfp4_record_hip_error(int) {}
nvfp4_status_t nvfp4_check_cache(const nvfp4_cache_t *) { return NVFP4_OK; }

int main(int argc, char **argv)
{
    if (argc != 3)
        return 5;
    guarded::Input in(argv[1]);
    FILE *out = fopen(argv[2], "wb");
    int32_t w[13];
    in.read(w, sizeof w);
    float f[3];
    in.read(f, sizeof f);
    const int dtype = w[0];
    const int64_t T = w[1], H = w[2], B = w[3], width = w[6], pages = w[7], ps = w[8], heads = w[9], D = w[10];
    const size_t size = dtype == NVFP4_F32 ? 4 : 2, rows = pages * heads * ps;
    const auto kc = in.bytes(rows * D / 2), ks = in.bytes(rows * D / 16), vc = in.bytes(rows * D / 2), vs = in.bytes(rows * D / 16),
               q = in.bytes(T * H * D * size), offsets = in.bytes(4 * (B + 1)), lengths = in.bytes(4 * B), table = in.bytes(4 * B * width);
    std::vector<uint8_t> first;
    cpu_wave::lds_start = lds;
    // the ends of every buffer, with copies to LDS that land at once; their starts, with
    // copies that land as late as the waits let them
    for (int turn = 0; turn < 2; ++turn) {
        const bool at_start = turn;
        cpu_wave::lazy = turn;
        auto here = [&](const std::vector<uint8_t> &v, size_t align) { return guarded::copy(v, align, at_start); };
        float *g[2];
        for (int i = 0; i < 2; ++i)
            *(g[i] = (float *)guarded::make(4, 4, at_start)) = f[1 + i];
        const nvfp4_cache_t cache = {here(kc, 16), here(ks, 16), here(vc, 16), here(vs, 16), g[0], g[1], pages, ps, heads, D,
                                     heads * ps * D / 2, heads * ps * D / 16};
        const nvfp4_attention_t a = {H * D, D, w[4], w[5], w[11], f[0], w[12]};
        const size_t need = nvfp4_cache_attention_workspace_bytes(&cache, dtype, T, H, B, &a);
        uint8_t *o = guarded::make(T * H * D * size, size, at_start), *lse = guarded::make(T * H * 4, 4, at_start),
                *ws = need ? guarded::make(need, 256, at_start) : nullptr;
        memset(o, 0xA5, T * H * D * size);
        memset(lse, 0xA5, T * H * 4);
        if (nvfp4_cache_attention(&cache, here(q, size), dtype, o, (float *)lse, (const int32_t *)here(offsets, 4),
                                  (const int32_t *)here(lengths, 4), (const int32_t *)here(table, 4), T, H, B, width, &a, ws, need,
                                  nullptr) != NVFP4_OK)
            return 6;
        for (size_t i = 0; i < std::min<size_t>(need, kTicketBytes); ++i)
            if (ws[i])
                return 7;
        std::vector<uint8_t> got(o, o + T * H * D * size);
        got.insert(got.end(), lse, lse + T * H * 4);
        if (turn && got != first)
            return 8;
        first = got;
    }
    for (const char *name : cpu_wave::launched)
        puts(name);
    fwrite(first.data(), 1, first.size(), out);
    return fclose(out) ? 5 : 0;
}
