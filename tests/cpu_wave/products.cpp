// Runs the library's products (source and launches) on the CPU, on guarded memory.
//   products <in> <out>
// in, 4-byte words: experts (0, 1), kind (-1: the plan's own), slices of K, dtype, M, N
// (experts: slots), K, L (experts), slots_per_row, layout, alpha (float32),
// has scale_a, has scale_b; then a, b, sfa, sfb, offsets and order (experts),
// scale_a, scale_b
// out: c (0xA5 where nothing was written); stdout: the kernels launched
//   products, with lines "experts M N K L" on stdin: each shape's kind and slices;
// first the kinds that are built: kind, uses (1 dense, 2 experts), most slices
#include "nvfp4_gemm.hip"

#include "guarded.h"

namespace {
thread_local __attribute__((aligned(16))) uint8_t lds[kLdsBytes];

// The plan's count of tiles and slices for a shape that is given.
Plan forced(int kind, int64_t splits, int64_t M, int64_t N, int64_t K, int64_t L, bool experts)
{
    Plan p{};
    for (const Shape &s : kShapes) {
        if (s.kind != (Kind)kind)
            continue;
        p.kind = s.kind, p.bm = s.bm, p.bn = s.bn;
        p.stages = (int32_t)ceil_div(K, kStageK);
        p.tiles_m = ceil_div(M, s.bm);
        p.tiles_n = experts ? std::min<int64_t>(N, N / s.bn + std::min(L, N)) : ceil_div(N, s.bn);
        p.tiles = p.tiles_m * p.tiles_n * (experts ? 1 : L);
        p.per_split = (int32_t)ceil_div(p.stages, splits);
        p.splits = (int32_t)ceil_div(p.stages, p.per_split);
    }
    return p;
}
} // namespace

void nvfp4_record_hip_error(int) {}

int main(int argc, char **argv)
{
    if (argc == 1) {
        for (const Shape &s : kShapes)
            printf("built %d %d %d\n", (int)s.kind, s.uses, s.max_splits);
        long long experts, M, N, K, L;
        while (scanf("%lld %lld %lld %lld %lld", &experts, &M, &N, &K, &L) == 5) {
            const Plan p = experts ? experts_plan(M, K, L, N) : dense_plan(M, N, K, L);
            printf("%d %d\n", (int)p.kind, p.splits);
        }
        return 0;
    }
    if (argc != 3)
        return 5;
    guarded::Input in(argv[1]);
    FILE *out = fopen(argv[2], "wb");
    int32_t w[10];
    in.read(w, sizeof w);
    const float alpha = in.word<float>();
    const int32_t has_ga = in.word<int32_t>(), has_gb = in.word<int32_t>();
    const bool experts = w[0];
    const int64_t M = w[4], N = w[5], K = w[6], L = w[7], per = w[8];
    const int dtype = w[3], layout = w[9];
    const int64_t rows = experts ? N / per : N, b_batches = experts ? 1 : L, ncb = (K / 16 + 3) / 4;
    auto scale_bytes = [&](int64_t r, int64_t batches) {
        return (size_t)(batches * (layout == NVFP4_SF_BLOCKED ? (r + 127) / 128 * ncb * 512 : r * (K / 16)));
    };
    const auto a = in.bytes(L * M * K / 2), b = in.bytes(b_batches * rows * K / 2), sfa = in.bytes(scale_bytes(M, L)),
               sfb = in.bytes(scale_bytes(rows, b_batches)), offsets = in.bytes(experts ? 4 * (L + 1) : 0),
               order = in.bytes(experts ? 4 * N : 0), ga = in.bytes(has_ga ? (experts ? 4 * L : 4) : 0),
               gb = in.bytes(has_gb ? 4 : 0);
    const Plan plan = w[1] < 0 ? (experts ? experts_plan(M, K, L, N) : dense_plan(M, N, K, L))
                               : forced(w[1], w[2], M, N, K, L, experts);
    const size_t size = dtype == NVFP4_F32 ? 4 : 2, rows_c = (experts ? 1 : L) * N, bytes_c = rows_c * M * size;
    const size_t need = plan_workspace(plan, (int64_t)rows_c, M);
    std::vector<uint8_t> first;
    cpu_wave::lds_start = lds;
    cpu_wave::lockstep = true;
    // the ends of every buffer, with copies to LDS that land at once; their starts, with
    // copies that land as late as the waits let them
    for (int turn = 0; turn < 2; ++turn) {
        const bool at_start = turn;
        cpu_wave::lazy = turn;
        auto here = [&](const std::vector<uint8_t> &v, size_t align) { return guarded::copy(v, align, at_start); };
        uint8_t *c = guarded::make(bytes_c, size, at_start), *ws = need ? guarded::make(need, 256, at_start) : nullptr;
        memset(c, 0xA5, bytes_c);
        GemmParams p = fill(plan, here(a, 16), here(b, 16), here(sfa, 16), here(sfb, 16), c, dtype, M, N, K, L, layout, alpha,
                            (const float *)here(ga, 4), (const float *)here(gb, 4), ws);
        nvfp4_status_t st;
        if (experts) {
            p.offsets = (const int32_t *)here(offsets, 4), p.order = (const int32_t *)here(order, 4);
            p.slots_per_row = (int32_t)per;
            st = run<true>(plan, p, nullptr);
        } else {
            st = run<false>(plan, p, nullptr);
        }
        if (st != NVFP4_OK)
            return 6;
        for (size_t i = 0; i < std::min<size_t>(need, kTicketBytes); ++i)
            if (ws[i])
                return 7;
        const std::vector<uint8_t> got(c, c + bytes_c);
        if (turn && got != first)
            return 8;
        first = got;
    }
    for (const char *name : cpu_wave::launched)
        puts(name);
    fwrite(first.data(), 1, first.size(), out);
    return fclose(out) ? 5 : 0;
}
