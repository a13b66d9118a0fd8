// Runs the library's router and combine (source and launches) on the CPU, on
// guarded memory: an access outside of a buffer is a segmentation fault.
//   route <in> <out>
// in, 4-byte words: 0, dtype T E k score n_group topk_group group_top renormalize
// has_bias, scaling (float32), logits, bias; out: ids, weights, offsets, order
// in: 1, dtype T k M, y, ids, weights; out: out
#include "nvfp4_moe.hip"

#include "guarded.h"

namespace {
thread_local int32_t list_lds[40960];

int route(guarded::Input &in, FILE *out)
{
    int32_t w[10];
    in.read(w, sizeof w);
    const float scaling = in.word<float>();
    const int dtype = w[0], T = w[1], E = w[2], k = w[3], S = T * k;
    const auto logits = in.bytes((size_t)T * E * (dtype == NVFP4_F32 ? 4 : 2)), bias = in.bytes(w[9] ? 4 * E : 0);
    const nvfp4_routing_t routing{w[4], w[5], w[6], w[7], w[8], scaling};
    for (int at_start = 0; at_start < 2; ++at_start) {
        auto make = [&](size_t n) { return guarded::make(n, 4, at_start); };
        int32_t *ids = (int32_t *)make(4 * S), *offsets = (int32_t *)make(4 * (E + 1)), *order = (int32_t *)make(4 * S);
        float *weights = (float *)make(4 * S);
        const size_t need = nvfp4_moe_route_workspace_bytes(T, E, k);
        uint8_t *ws = need ? guarded::make(need, 256, at_start) : nullptr;
        if (nvfp4_moe_route(guarded::copy(logits, dtype == NVFP4_F32 ? 4 : 2, at_start), dtype,
                            (const float *)guarded::copy(bias, 4, at_start), ids, weights, offsets, order, T, E, k, &routing, ws,
                            need, nullptr) != NVFP4_OK)
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
    return 0;
}

int combine(guarded::Input &in, FILE *out)
{
    int32_t w[4];
    in.read(w, sizeof w);
    const int dtype = w[0], T = w[1], k = w[2], M = w[3];
    const size_t size = dtype == NVFP4_F32 ? 4 : 2, n = (size_t)T * M * size;
    const auto y = in.bytes(n * k), ids = in.bytes(4 * T * k), weights = in.bytes(4 * T * k);
    for (int at_start = 0; at_start < 2; ++at_start) {
        uint8_t *o = guarded::make(n, size, at_start);
        if (nvfp4_moe_combine(guarded::copy(y, size, at_start), dtype, (const int32_t *)guarded::copy(ids, 4, at_start),
                              (const float *)guarded::copy(weights, 4, at_start), o, T, k, M, nullptr) != NVFP4_OK)
            return 6;
        if (at_start)
            fwrite(o, 1, n, out);
    }
    return 0;
}
} // namespace

void nvfp4_record_hip_error(int) {}

int main(int argc, char **argv)
{
    if (argc != 3)
        return 5;
    guarded::Input in(argv[1]);
    FILE *out = fopen(argv[2], "wb");
    const int status = in.word<int32_t>() ? combine(in, out) : route(in, out);
    return fclose(out) ? 5 : status;
}
