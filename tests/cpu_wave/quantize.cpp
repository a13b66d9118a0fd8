// Runs the library's global scale, quantise and dequantise (source and launches)
// on the CPU, on guarded memory.
//   quantize <in> <out>
// in, 4-byte words: dtype rows K L row_stride batch_stride layout given, scale
// (float32, used where given), x: as many elements as the strides reach
// out: the global scale, the scale that was used, codes, scales, values
#include "nvfp4_quantize.hip"

#include "guarded.h"

void nvfp4_record_hip_error(int) {}
extern "C" size_t nvfp4_blocked_scales_bytes(int64_t rows, int64_t K, int64_t L)
{
    return (size_t)(K % 32 ? 0 : L * ((rows + 127) / 128) * ((K + 63) / 64) * 512);
}

int main(int argc, char **argv)
{
    if (argc != 3)
        return 5;
    guarded::Input in(argv[1]);
    FILE *out = fopen(argv[2], "wb");
    int32_t w[8];
    in.read(w, sizeof w);
    const float given = in.word<float>();
    const int dtype = w[0], layout = w[6];
    const int64_t rows = w[1], K = w[2], L = w[3], rs = w[4], bs = w[5];
    const size_t size = dtype == NVFP4_F32 ? 4 : 2;
    const auto x = in.bytes((size_t)((L - 1) * bs + (rows - 1) * rs + K) * size);
    const size_t codes_n = L * rows * K / 2, n = L * rows * K * size,
                 scales_n = layout == NVFP4_SF_BLOCKED ? nvfp4_blocked_scales_bytes(rows, K, L) : L * rows * (K / 16);
    for (int at_start = 0; at_start < 2; ++at_start) {
        uint8_t *px = guarded::copy(x, size, at_start), *ws = guarded::make(256, 256, at_start);
        float *g = (float *)guarded::make(4, 4, at_start), *used = (float *)guarded::make(4, 4, at_start);
        if (nvfp4_global_scale(px, dtype, g, rows, K, L, rs, bs, ws, 256, nullptr) != NVFP4_OK)
            return 6;
        for (int i = 0; i < 256; ++i)
            if (ws[i])
                return 7;
        *used = w[7] ? given : *g;
        uint8_t *codes = guarded::make(codes_n, 8, at_start), *scales = guarded::make(scales_n, 4, at_start),
                *values = guarded::make(n, size, at_start);
        if (nvfp4_quantize(px, dtype, used, codes, scales, rows, K, L, rs, bs, layout, nullptr) != NVFP4_OK ||
            nvfp4_dequantize(codes, scales, used, values, dtype, rows, K, L, layout, nullptr) != NVFP4_OK)
            return 6;
        if (!at_start)
            continue;
        fwrite(g, 4, 1, out);
        fwrite(used, 4, 1, out);
        fwrite(codes, 1, codes_n, out);
        fwrite(scales, 1, scales_n, out);
        fwrite(values, 1, n, out);
    }
    return fclose(out) ? 5 : 0;
}
