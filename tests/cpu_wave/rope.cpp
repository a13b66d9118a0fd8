// Runs the library's rope (source and launch) on the CPU, on guarded memory.
//   rope <in> <out>
// in, 4-byte words: dtype T H D R x_token x_head out_token out_head layout transpose in_place,
// factor (float32), a word; then positions (int64 [T]), frequencies (float64 [R / 2]), x: as many
// elements as its strides reach
// out: out, as many elements as its strides reach (0xA5 where nothing was written; in place: x)
#include "nvfp4_rope.hip"

#include "guarded.h"

void nvfp4_record_hip_error(int) {}

int main(int argc, char **argv)
{
    if (argc != 3)
        return 5;
    guarded::Input in(argv[1]);
    FILE *out = fopen(argv[2], "wb");
    int32_t w[12];
    in.read(w, sizeof w);
    const float factor = in.word<float>();
    in.word<int32_t>();
    const int dtype = w[0];
    const int64_t T = w[1], H = w[2], D = w[3], R = w[4];
    const size_t size = dtype == NVFP4_F32 ? 4 : 2;
    auto reach = [&](int64_t token, int64_t head) { return (size_t)((T - 1) * token + (H - 1) * head + D) * size; };
    const auto positions = in.bytes(8 * T), frequencies = in.bytes(4 * R), x = in.bytes(reach(w[5], w[6]));
    const size_t n = reach(w[7], w[8]);
    std::vector<uint8_t> first;
    for (int turn = 0; turn < 2; ++turn) {
        const bool at_start = turn;
        uint8_t *px = guarded::copy(x, size, at_start), *po = w[11] ? px : guarded::make(n, size, at_start);
        if (!w[11])
            memset(po, 0xA5, n);
        if (nvfp4_rope(px, dtype, po, (const int64_t *)guarded::copy(positions, 8, at_start),
                       (const double *)guarded::copy(frequencies, 8, at_start), T, H, D, R, w[5], w[6], w[7], w[8], w[9], factor, w[10],
                       nullptr) != NVFP4_OK)
            return 6;
        const std::vector<uint8_t> got(po, po + n);
        // the ends and the starts have other alignments, so other kernels: the same results
        if (turn && got != first)
            return 8;
        first = got;
    }
    fwrite(first.data(), 1, first.size(), out);
    return fclose(out) ? 5 : 0;
}
