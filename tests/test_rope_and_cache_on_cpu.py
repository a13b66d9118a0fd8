"""CPU run of the sources of rotary positions (nvfp4_rope.hip) and of the paged cache's
write and read (nvfp4_cache.hip), launches included, compiled for the host
(tests/cpu_wave): buffers end, and once more start, at a page that is not mapped; slots lead
outside the cache; what is written is the definition's, and nothing else is."""
import numpy as np
import pytest

import attention_reference as ref
import block_scaled_fp4_gemv_amd as g
import cpu_wave_util as cpu_wave
import fp4_reference as fp4

torch = pytest.importorskip("torch")

DTYPES = [torch.float16, torch.bfloat16, torch.float32]     # by nvfp4_dtype_t


@pytest.fixture(scope="module")
def rope(tmp_path_factory):
    return cpu_wave.build(tmp_path_factory.mktemp("rope"), "rope")


@pytest.fixture(scope="module")
def cache(tmp_path_factory):
    return cpu_wave.build(tmp_path_factory.mktemp("cache"), "cache")


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dt", [0, 1, 2])
@pytest.mark.parametrize("T,H,D,R,gap,kind", [(1, 1, 2, 2, 0, ""), (3, 5, 64, 64, 0, ""), (2, 3, 96, 48, 32, "place"), (5, 1, 33, 32, 1, ""),
                                              (40, 2, 32, 16, 8, "heads"), (2, 600, 16, 16, 0, ""), (7, 3, 80, 64, 3, "place"),
                                              (1, 2, 2048, 2048, 0, "transpose")])
def test_rope(rope, tmp_path, T, H, D, R, gap, kind, dt, layout):
    rng = np.random.default_rng([T, H, D, dt])
    token, head = H * (D + gap) + gap, D + gap
    n = (T - 1) * token + (H - 1) * head + D
    flat = torch.from_numpy(rng.standard_normal(n)).to(DTYPES[dt])
    ot, oh = (token, head) if kind == "place" else (D + gap, T * (D + gap)) if kind == "heads" else (H * D, D)
    positions, f = rng.integers(-1000, 100000, T), np.array(g.nvfp4_rope_frequencies(R, 10000.0))
    back = kind == "transpose"
    head_words = np.array([dt, T, H, D, R, token, head, ot, oh, layout == "interleaved", back, kind == "place"], np.int32)
    got, _ = cpu_wave.run(rope, tmp_path, [head_words, np.float32(1.5), np.int32(0), positions.astype(np.int64), f, flat.view(torch.uint8).numpy()])
    all_out = torch.from_numpy(got.copy()).view(DTYPES[dt])
    out = all_out.as_strided((T, H, D), (ot, oh, 1))
    x = flat.as_strided((T, H, D), (token, head, 1)).double().numpy()
    ref.check_rope(out, x, ref.rope(x, positions, f, R, layout, 1.5, back), R, layout, 1.5, DTYPES[dt])
    other = torch.ones(all_out.shape, dtype=torch.bool)
    other.as_strided((T, H, D), (ot, oh, 1)).fill_(False)
    untouched = flat if kind == "place" else torch.from_numpy(np.full(len(got), 0xA5, np.uint8)).view(DTYPES[dt])
    assert torch.equal(all_out.view(torch.uint8).reshape(len(all_out), -1)[other], untouched.view(torch.uint8).reshape(len(all_out), -1)[other])


@pytest.mark.parametrize("dt", [0, 1, 2])
@pytest.mark.parametrize("T,heads,D,page_size,pages,gap", [(1, 1, 32, 16, 1, 0), (5, 3, 96, 16, 2, 16), (17, 2, 64, 32, 1, 0), (33, 5, 160, 16, 4, 48),
                                                           (70, 1, 256, 16, 5, 0), (16, 7, 128, 64, 1, 32)])
def test_cache(cache, tmp_path, T, heads, D, page_size, pages, gap, dt):
    rng = np.random.default_rng([T, heads, D, dt])
    total = pages * page_size
    slots = rng.permutation(max(total, T))[:T].astype(np.int64)
    slots[rng.random(T) < 0.2] = -3
    if T > 2:
        slots[1], slots[2] = total, 2 ** 62
    kept = (slots >= 0) & (slots < total)
    token, head = heads * (D + 5) + 7, D + 5
    n = (T - 1) * token + (heads - 1) * head + D
    k, v = (torch.from_numpy(rng.standard_normal(n) * 2).to(DTYPES[dt]) for _ in range(2))
    scales = np.array([0.02, 0.3], np.float32)
    head_words = np.array([dt, T, pages, page_size, heads, D, token, head, gap, gap], np.int32)
    got, _ = cpu_wave.run(cache, tmp_path, [head_words, scales, slots, k.view(torch.uint8).numpy(), v.view(torch.uint8).numpy()])
    at = 0
    page, place = slots[kept] // page_size, slots[kept] % page_size
    for i, x in enumerate((k, v)):
        rows = x.as_strided((T, heads, D), (token, head, 1)).double().numpy()[kept]
        want = [np.zeros((0, heads, D // 2), np.uint8), np.zeros((0, heads, D // 16), np.uint8)]
        if len(rows):
            codes, sc = fp4.quantize(rows, float(scales[i]))
            want = [fp4.pack(codes), sc]
        for w, each in zip(want, (D // 2, D // 16)):
            stride = heads * page_size * each + gap
            size = (pages - 1) * stride + heads * page_size * each
            room, expect = got[at:at + size], np.full(size, 0xA5, np.uint8)
            view = np.lib.stride_tricks.as_strided(expect, (pages, heads, page_size, each), (stride, page_size * each, each, 1))
            view[page, :, place] = w
            assert np.array_equal(room, expect)
            at += size
    size = 4 if dt == 2 else 2
    for i, x in enumerate((k, v)):
        back = torch.from_numpy(got[at:at + T * heads * D * size].copy()).view(DTYPES[dt]).reshape(T, heads, D).double().numpy()
        at += T * heads * D * size
        want = np.zeros((T, heads, D))
        rows = x.as_strided((T, heads, D), (token, head, 1)).double().numpy()[kept]
        if len(rows):
            codes, sc = fp4.quantize(rows, float(scales[i]))
            want[kept] = fp4.values(fp4.pack(codes), sc) * np.float64(scales[i])
        assert (np.abs(back - want) <= (2.0 ** -24 + fp4.HALF_STEP[DTYPES[dt]] * (1 + 2.0 ** -10)) * np.abs(want) + fp4.LEAST[DTYPES[dt]]).all()
