"""CPU run of the source of global scale, quantise and dequantise
(nvfp4_quantize.hip), launches included, compiled for the host (tests/cpu_wave):
buffers end, and once more start, at a page that is not mapped, and what is
written is the definition's, bit for bit."""
import numpy as np
import pytest

import block_scaled_fp4_gemv_amd as g
import cpu_wave_util as cpu_wave
import fp4_reference as ref

torch = pytest.importorskip("torch")

DTYPES = {g.NVFP4_F16: torch.float16, g.NVFP4_BF16: torch.bfloat16, g.NVFP4_F32: torch.float32}


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    return cpu_wave.build(tmp_path_factory.mktemp("quantize"), "quantize")


@pytest.mark.parametrize("layout", [0, 1], ids=["plain", "blocked"])
@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("L,rows,K,pad,gap,given", [(1, 1, 32, 0, 0, 0), (2, 3, 96, 0, 0, 0), (1, 5, 160, 7, 0, 0), (3, 17, 288, 1, 9, 0),
                                                    (1, 129, 64, 0, 0, 0.3), (2, 33, 544, 33, 5, 1e-29), (1, 40, 2080, 0, 0, 1e9)])
def test_stays_inside_its_buffers(program, tmp_path, L, rows, K, pad, gap, given, dtype, layout):
    rng = np.random.default_rng([L, rows, K, dtype])
    rs = K + pad
    bs = rows * rs + gap
    n = (L - 1) * bs + (rows - 1) * rs + K
    flat = torch.from_numpy(rng.standard_normal(n) * np.exp(rng.standard_normal(n)) * (given or 1.0)).to(DTYPES[dtype])
    head = np.array([dtype, rows, K, L, rs, bs, layout, given != 0], np.int32)
    out, _ = cpu_wave.run(program, tmp_path, [head, np.float32(given), flat.view(torch.uint8).numpy()])
    x = flat.as_strided((L, rows, K), (bs, rs, 1)).double().numpy()
    scale, used = (float(v) for v in out[:8].view(np.float32))
    assert scale == ref.global_scale(x)
    codes, left = out[8:8 + L * rows * K // 2].reshape(L, rows, K // 2), out[8 + L * rows * K // 2:]
    count = L * (ref.cdiv(rows, 128) * ref.cdiv(K, 64) * 512 if layout else rows * K // 16)
    scales, values = left[:count].reshape(L, -1), left[count:]
    if layout:
        assert not scales[:, ref.blocked_pad_mask(rows, K)].any(), "padding is not zero"
        scales = np.stack([ref.from_blocked(s, rows, K) for s in scales])
    scales = scales.reshape(L, rows, K // 16)
    want, want_s = ref.quantize(x, used)
    assert np.array_equal(scales, want_s) and np.array_equal(ref.unpack(codes), want)
    got = torch.from_numpy(values.copy()).view(DTYPES[dtype]).double().numpy().reshape(L, rows, K)
    exact = ref.values(codes, scales) * used
    top = torch.finfo(DTYPES[dtype]).max
    tol = (2.0 ** -24 + ref.HALF_STEP[DTYPES[dtype]] * (1 + 2.0 ** -10)) * np.abs(exact) + ref.LEAST[DTYPES[dtype]]
    assert (np.abs(got - exact) <= tol)[np.abs(exact) < top].all()
