// Runs the library's router (source and launches) on the CPU: every buffer ends
// where its mapping ends, so a read or write past one is a segmentation fault.
//   route <in> <out>, 4-byte words (in): dtype T E k score n_group topk_group
//   group_top renormalize has_bias, scaling (float32), logits, bias
//   out: ids, weights, offsets, order
#include "nvfp4_moe.hip"

#include <cstdio>
#include <vector>

namespace {
thread_local int32_t list_lds[40960];           // the launches' dynamic LDS

// n bytes, the page behind them not mapped; `at_start`: the page before them instead
uint8_t *guarded(size_t n, bool at_start)
{
    const size_t page = 4096, size = (n + page - 1) / page * page;
    uint8_t *p = (uint8_t *)mmap(nullptr, size + 2 * page, PROT_NONE, MAP_PRIVATE | MAP_ANONYMOUS, -1, 0);
    if (p == MAP_FAILED || mprotect(p + page, size, PROT_READ | PROT_WRITE))
        exit(4);
    return p + page + (at_start ? 0 : size - n);
}
} // namespace

void nvfp4_record_hip_error(int) {}

int main(int argc, char **argv)
{
    if (argc != 3)
        return 5;
    FILE *in = fopen(argv[1], "rb"), *out = fopen(argv[2], "wb");
    int32_t w[10];
    float scaling;
    if (!in || !out || fread(w, 4, 10, in) != 10 || fread(&scaling, 4, 1, in) != 1)
        return 5;
    const int dtype = w[0], T = w[1], E = w[2], k = w[3], S = T * k;
    const size_t size = dtype == NVFP4_F32 ? 4 : 2;
    std::vector<uint8_t> logits_in((size_t)T * E * size), bias_in((size_t)E * 4);
    if (fread(logits_in.data(), 1, logits_in.size(), in) != logits_in.size() || fread(bias_in.data(), 4, E, in) != (size_t)E)
        return 5;
    const nvfp4_routing_t routing{w[4], w[5], w[6], w[7], w[8], scaling};
    for (int at_start = 0; at_start < 2; ++at_start) {
        auto make = [&](size_t n) { return guarded(n, at_start); };
        uint8_t *logits = make(logits_in.size()), *bias = make(bias_in.size());
        memcpy(logits, logits_in.data(), logits_in.size());
        memcpy(bias, bias_in.data(), bias_in.size());
        int32_t *ids = (int32_t *)make(4 * S), *offsets = (int32_t *)make(4 * (E + 1)), *order = (int32_t *)make(4 * S);
        float *weights = (float *)make(4 * S);
        const size_t need = nvfp4_moe_route_workspace_bytes(T, E, k);
        uint8_t *ws = guarded(need + 1, true);  // the entry point wants 256-byte alignment; zero-filled
        const nvfp4_status_t st = nvfp4_moe_route(logits, dtype, w[9] ? (const float *)bias : nullptr, ids, weights, offsets,
                                                  order, T, E, k, &routing, ws, need, nullptr);
        if (st != NVFP4_OK)
            return 6;
        for (size_t i = 0; i < need; ++i)
            if (ws[i])
                return 7;
        if (at_start)
            continue;
        fwrite(ids, 4, S, out);
        fwrite(weights, 4, S, out);
        fwrite(offsets, 4, E + 1, out);
        fwrite(order, 4, S, out);
    }
    return fclose(out) ? 5 : 0;
}
