"""GPU: global scale, quantisation and dequantisation against the 64-bit
definition. Codes and scales have to be equal bit for bit (both sides round the
exact quotients); dequantised values are within their two roundings."""
import numpy as np
import pytest

import fp4_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_gemv_amd as g  # noqa: E402

DTYPES = [torch.float16, torch.bfloat16, torch.float32]
TAIL = 64


def sample(rng, L, rows, K, kind):
    x = rng.standard_normal((L, rows, K)) * np.exp(rng.standard_normal(K))
    if kind == "edge":
        x[rng.random(x.shape) < 0.3] = 0.0
        x[rng.random(x.shape) < 0.05] *= 1e-4
        x[:, :, :16] = 0.0
        x[rng.random(x.shape) < 0.05] = -0.0
    elif kind == "ties":
        # with g = 1 every block's scale is 1 (largest value 6) and every value a midpoint or a code
        x = rng.choice([0, 0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6], (L, rows, K))
        x[..., ::16] = 6.0
        x *= rng.choice([-1.0, 1.0], x.shape)
        x *= np.exp2(rng.integers(-3, 4, (L, rows, 1)))
    elif kind == "special":
        flat = x.reshape(-1)
        at = rng.integers(0, flat.size, max(3, flat.size // 64))
        flat[at] = rng.choice([np.nan, np.inf, -np.inf, 3e38, -1e-38, 1e-44], at.size)
    return x


def run(x, dtype, gs, layout, row_pad=0, rows=None, K=None):
    """Quantises x [L][rows][K] (a torch CPU tensor of dtype); returns codes, plain scale codes, raw scales."""
    L, rows, K = x.shape
    buf = torch.full((L, rows, K + row_pad), float("nan"), dtype=dtype)
    buf[:, :, :K] = x
    dev = buf.cuda()
    codes = torch.full((L * rows * K // 2 + TAIL,), 0xA5, dtype=torch.uint8, device="cuda")
    n = L * ref.cdiv(rows, 128) * ref.cdiv(K, 64) * 512 if layout == "blocked" else L * rows * K // 16
    scales = torch.full((n + TAIL,), 0xA5, dtype=torch.uint8, device="cuda")
    scale = None if gs is None else torch.tensor([gs], dtype=torch.float32, device="cuda")
    g.nvfp4_quantize(dev, codes, scales, rows, K, L, layout, global_scale=scale, row_stride=K + row_pad,
                     batch_stride=rows * (K + row_pad))
    torch.cuda.synchronize()
    c, s = codes.cpu().numpy(), scales.cpu().numpy()
    assert (c[-TAIL:] == 0xA5).all() and (s[-TAIL:] == 0xA5).all(), "write past the end"
    c, s = c[:-TAIL].reshape(L, rows, K // 2), s[:-TAIL]
    if layout == "blocked":
        each = s.reshape(L, -1)
        assert not each[:, ref.blocked_pad_mask(rows, K)].any(), "padding is not zero"
        plain = np.stack([ref.from_blocked(b, rows, K) for b in each])
    else:
        plain = s.reshape(L, rows, K // 16)
    return c, plain, codes[:-TAIL], scales[:-TAIL]


SHAPES = [(1, 1, 32), (1, 1, 7168), (2, 5, 96), (1, 127, 4096), (3, 129, 160), (1, 33, 2080), (1, 300, 1056)]


@pytest.mark.parametrize("layout", ["plain", "blocked"])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("kind,gs", [("normal", 0.0123), ("edge", 3e-4), ("ties", None), ("ties", 0.5), ("special", 0.7),
                                     ("normal", 1e9), ("edge", 1e-29)])
@pytest.mark.parametrize("L,rows,K", SHAPES)
def test_codes_are_the_definitions(L, rows, K, kind, gs, dtype, layout):
    rng = np.random.default_rng([L, rows, K, len(kind)])
    x = torch.from_numpy(sample(rng, L, rows, K, kind) * (gs or 1.0 if kind != "special" else 1.0)).to(dtype)
    want, scale = ref.quantize(x.double().numpy(), float(np.float32(gs)) if gs else 1.0)
    codes, plain, _, _ = run(x, dtype, gs, layout, row_pad=(0, 8, 33)[rows % 3])
    assert np.array_equal(plain, scale), np.argwhere(plain != scale)[:4]
    assert np.array_equal(ref.unpack(codes), want), np.argwhere(ref.unpack(codes) != want)[:4]


@pytest.mark.parametrize("gs", [0.0, -1.0, float("nan"), float("inf"), 1e-35])
def test_bad_global_scale_shows(gs):
    x = torch.randn(1, 4, 64)
    codes, plain, _, _ = run(x, torch.float32, gs, "plain")
    assert (plain == 0x7F).all() and not codes.any()


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("L,rows,K,pad", [(1, 1, 1, 0), (1, 1, 7168, 0), (2, 3, 33, 5), (1, 1000, 4096, 0), (3, 77, 1001, 7),
                                          (1, 4096, 4096, 0)])
def test_global_scale(L, rows, K, pad, dtype):
    gen = torch.Generator().manual_seed(rows + K)
    buf = torch.full((L, rows, K + pad), float("nan"), dtype=dtype)
    buf[:, :, :K] = (torch.randn(L, rows, K, generator=gen) * 3).to(dtype)
    dev = buf.cuda()
    ws = torch.zeros(g.nvfp4_global_scale_workspace_bytes(), dtype=torch.uint8, device="cuda")
    out = torch.zeros(2, device="cuda")
    last = None
    for fill in (None, float("nan"), float("-inf"), 0.0):
        if fill is not None:
            dev[-1, -1, K - 1] = fill
            dev[0, 0, 0] = fill
        if fill == 0.0:
            dev[:, :, :K] = -0.0
        g.nvfp4_global_scale(dev, out, rows, K, L, ws, row_stride=K + pad, batch_stride=rows * (K + pad))
        want = ref.global_scale(dev[:, :, :K].double().cpu().numpy())
        assert out.tolist() == [want, 0.0], fill
        assert not ws.any(), "counters are not cleared"
        last = want
    assert last == 1.0


def test_global_scale_of_tiny_values():
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    out = torch.zeros(1, device="cuda")
    g.nvfp4_global_scale(torch.full((64,), 1e-40, device="cuda"), out, 1, 64, 1, ws)
    assert out.item() == 2.0 ** -100


@pytest.mark.parametrize("layout", ["plain", "blocked"])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("L,rows,K,gs", [(1, 1, 32, None), (2, 129, 96, 0.37), (1, 300, 4096, 1.5e-3)])
def test_dequantize(L, rows, K, gs, dtype, layout):
    rng = np.random.default_rng(rows)
    x = torch.from_numpy(sample(rng, L, rows, K, "normal") * (gs or 1.0)).float()
    codes, plain, dc, ds = run(x, torch.float32, gs, layout)
    n = L * rows * K
    out = torch.full((n + TAIL,), -1.0, dtype=dtype, device="cuda")
    scale = None if gs is None else torch.tensor([gs], dtype=torch.float32, device="cuda")
    g.nvfp4_dequantize(dc, ds, out[:n], rows, K, L, layout, global_scale=scale)
    torch.cuda.synchronize()
    assert (out[n:] == -1).all()
    want = ref.values(codes, plain) * (float(np.float32(gs)) if gs else 1.0)
    got = out[:n].double().cpu().numpy().reshape(want.shape)
    tol = (2.0 ** -24 + ref.HALF_STEP[dtype] * (1 + 2.0 ** -23)) * np.abs(want) + ref.LEAST[dtype]
    assert (np.abs(got - want) <= tol).all()
    # every value within half a step of its code, a sixteenth of the largest of its block for the scale's rounding
    if dtype is torch.float32:
        block = np.abs(x.double().numpy().reshape(L, rows, -1, 16)).max(-1, keepdims=True)
        off = np.abs(got - x.double().numpy()).reshape(L, rows, -1, 16)
        assert (off <= block * (1 / 6 + 1 / 16) + 2.0 ** -10 * 6 * (gs or 1.0)).all()


def test_far_offsets():
    """A batch stride that carries the second batch past 2^32 bytes."""
    rows, K = 3, 64
    stride = (1 << 31) + 64
    big = torch.empty(stride + rows * K, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(2, rows, K).to(torch.bfloat16)
    big[:rows * K] = x[0].reshape(-1).cuda()
    big[stride:] = x[1].reshape(-1).cuda()
    codes = torch.zeros(2 * rows * K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(2 * rows * K // 16, dtype=torch.uint8, device="cuda")
    gs, ws = torch.zeros(1, device="cuda"), torch.zeros(256, dtype=torch.uint8, device="cuda")
    g.nvfp4_global_scale(big, gs, rows, K, 2, ws, row_stride=K, batch_stride=stride)
    g.nvfp4_quantize(big, codes, scales, rows, K, 2, "plain", global_scale=gs, row_stride=K, batch_stride=stride)
    v = x.double().numpy()
    assert gs.item() == ref.global_scale(v)
    want, scale = ref.quantize(v, gs.item())
    assert np.array_equal(scales.cpu().numpy().reshape(scale.shape), scale)
    assert np.array_equal(codes.cpu().numpy().reshape(2, rows, K // 2), ref.pack(want))


def test_on_a_stream_and_in_a_graph():
    """The whole chain on a stream of its own and captured, replayed with eager work between."""
    rows, K = 130, 1056
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(rows, K, device="cuda", generator=gen)
    codes = torch.zeros(rows * K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(ref.cdiv(rows, 128) * ref.cdiv(K, 64) * 512, dtype=torch.uint8, device="cuda")
    gs, ws = torch.zeros(1, device="cuda"), torch.zeros(256, dtype=torch.uint8, device="cuda")
    y = torch.zeros(rows, K, device="cuda")

    def chain():
        g.nvfp4_global_scale(x, gs, rows, K, 1, ws)
        g.nvfp4_quantize(x, codes, scales, rows, K, 1, "blocked", global_scale=gs)
        g.nvfp4_dequantize(codes, scales, y, rows, K, 1, "blocked", global_scale=gs)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        chain()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for i in range(3):
        x.copy_(torch.randn(rows, K, device="cuda", generator=gen) * (i + 1))
        chain()
        torch.cuda.synchronize()
        want = (codes.clone(), scales.clone(), y.clone(), gs.clone())
        for t in (codes, scales, y, gs):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((codes, scales, y, gs), want):
            assert torch.equal(a, b)
