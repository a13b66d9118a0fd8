"""GPU: nvfp4_gemm against the 64-bit product of the operands' exact values,
within the tolerance of float32 accumulation (fp4_reference); plain and blocked
scales give equal bits; nothing outside c is written."""
import numpy as np
import pytest

import fp4_reference as ref
import synth

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_gemv_amd as g  # noqa: E402

DTYPES = [torch.float16, torch.bfloat16, torch.float32]
TAIL = 64
_values = {}


def operand(rng, L, rows, K, dist="uniform"):
    codes = synth.pack_nibbles(synth.e2m1_codes(rng, (L, rows, K), dist))
    return codes, synth.scale_codes(rng, (L, rows, K // 16), dist)


def layout_of(scales, layout):
    return synth.to_blocked(scales) if layout == "blocked" else scales     # blocked padding: NaN codes


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def run(a, sfa, b, sfb, dtype, layout, alpha=1.0, ga=None, gb=None, stream=None):
    L, M, K = a.shape[0], a.shape[1], a.shape[2] * 2
    N = b.shape[1]
    c = torch.full((L * N * M + TAIL,), float("nan"), dtype=dtype, device="cuda")
    ws = torch.zeros(g.nvfp4_gemm_workspace_bytes(M, N, K, L), dtype=torch.uint8, device="cuda")
    scale = lambda v: None if v is None else torch.tensor([v], dtype=torch.float32, device="cuda")  # noqa: E731
    g.nvfp4_gemm(dev(a), dev(b), dev(layout_of(sfa, layout)), dev(layout_of(sfb, layout)), c[:L * N * M], M, N, K, L,
                 layout, alpha=alpha, scale_a=scale(ga), scale_b=scale(gb), workspace=ws if ws.numel() else None)
    torch.cuda.synchronize()
    assert torch.isnan(c[L * N * M:]).all(), "write past the end of c"
    assert not ws[:65536].any(), "tickets are not cleared"
    return c[:L * N * M].reshape(L, N, M)


def reference(a, sfa, b, sfb):
    """The product and the sum of its terms' sizes, float64, on the GPU's 64-bit units (torch)."""
    va, vb = dev(ref.values(a, sfa)), dev(ref.values(b, sfb))
    c = [vb[i] @ va[i].t().contiguous() for i in range(va.shape[0])]
    s = [vb[i].abs() @ va[i].abs().t().contiguous() for i in range(va.shape[0])]
    return torch.stack(c).cpu().numpy(), torch.stack(s).cpu().numpy()


# every tile shape: N up to 32, 64, more with few and with many tiles; K of one
# stage and less, ragged stages, K % 64 = 32; M and N around the tiles' edges; batches
SHAPES = [(1, 1, 32, 1), (1, 1, 64, 2), (7, 3, 96, 2), (128, 16, 256, 1), (129, 32, 1056, 1), (300, 17, 4096, 2),
          (1000, 9, 2080, 1), (31, 33, 160, 3), (257, 64, 4128, 1), (128, 50, 96, 1), (130, 65, 224, 2),
          (256, 256, 128, 1), (255, 257, 992, 1), (513, 129, 160, 2), (100, 500, 7168, 1), (4096, 70, 64, 1),
          (1, 1000, 512, 1), (1000, 1, 512, 1), (4100, 2600, 288, 1), (2050, 5000, 96, 1), (120, 20, 16384, 2)]


@pytest.mark.parametrize("M,N,K,L", SHAPES)
def test_product(M, N, K, L):
    rng = np.random.default_rng([M, N, K, L])
    (a, sfa), (b, sfb) = operand(rng, L, M, K), operand(rng, L, N, K)
    want, size = reference(a, sfa, b, sfb)
    for dtype in DTYPES:
        got = {lay: run(a, sfa, b, sfb, dtype, lay) for lay in ("plain", "blocked")}
        ref.check_product(got["blocked"], want, size, K, dtype, f"{dtype}")
        assert torch.equal(got["plain"].view(torch.uint8), got["blocked"].view(torch.uint8)), dtype


# every tile, K of 64 and of 32, several batches, slices of K
TILES = [(7168, 2050, 544, 1, 256, 256, 1), (3285, 1349, 448, 3, 256, 256, 1), (1500, 1030, 224, 2, 128, 128, 1),
         (521, 1836, 256, 3, 128, 128, 1), (513, 1000, 96, 1, 64, 64, 1), (1025, 513, 192, 1, 64, 64, 1),
         (1074, 38, 22944, 2, 64, 64, 15), (3077, 101, 11520, 2, 64, 64, 2), (4100, 200, 96, 1, 128, 32, 1),
         (4100, 200, 320, 1, 128, 32, 1), (1062, 1, 12512, 2, 128, 32, 14), (2050, 100, 96, 1, 64, 32, 1),
         (2050, 100, 448, 1, 64, 32, 1), (1067, 1, 18912, 1, 64, 32, 15), (1074, 2, 5184, 2, 64, 32, 7),
         (513, 1000, 544, 1, 32, 32, 1), (1025, 513, 576, 1, 32, 32, 1), (2105, 1, 12064, 1, 32, 32, 8)]


@pytest.mark.parametrize("M,N,K,L,tile_m,tile_n,splits", TILES)
def test_every_tile(M, N, K, L, tile_m, tile_n, splits):
    plan = g.nvfp4_gemm_plan(M, N, K, L)
    assert (plan["tile_m"], plan["tile_n"], plan["k_splits"]) == (tile_m, tile_n, splits)
    rng = np.random.default_rng([M, N, K, L])
    (a, sfa), (b, sfb) = operand(rng, L, M, K), operand(rng, L, N, K)
    want, size = reference(a, sfa, b, sfb)
    for dtype in DTYPES:
        got = {lay: run(a, sfa, b, sfb, dtype, lay) for lay in ("plain", "blocked")}
        ref.check_product(got["blocked"], want, size, K, dtype, "blocked")
        assert torch.equal(got["plain"], got["blocked"])


@pytest.mark.parametrize("M,N,K", [(70, 5, 512), (70, 40, 512), (300, 200, 544), (3000, 3500, 96)])
def test_scales_and_edge_codes(M, N, K):
    """alpha and the device's global scales; zero, subnormal and largest block scales; sums past float16's range."""
    rng = np.random.default_rng([M, N, K])
    (a, sfa), (b, sfb) = operand(rng, 1, M, K, "edge"), operand(rng, 1, N, K, "edge")
    want, size = reference(a, sfa, b, sfb)
    for alpha, ga, gb in ((1.0, 0.03, 0.002), (-0.375, None, 1e-4), (2e-5, 0.5, None)):
        f = np.float64(np.float32(alpha)) * (np.float32(ga) if ga else 1.0) * (np.float32(gb) if gb else 1.0)
        for dtype in DTYPES:
            got = run(a, sfa, b, sfb, dtype, "blocked", alpha, ga, gb)
            ref.check_product(got, want * f, size * abs(f), K, dtype, f"{dtype} {alpha}")
    got = run(a, sfa, b, sfb, torch.float16, "plain").double().cpu().numpy()
    far = np.abs(want) > 70000
    assert far.any() and np.array_equal(got[far], np.sign(want[far]) * np.inf)


@pytest.mark.parametrize("N", [8, 48, 300])
def test_nan_scales_reach_their_rows_alone(N):
    rng = np.random.default_rng(N)
    M, K = 200, 1056
    (a, sfa), (b, sfb) = operand(rng, 1, M, K), operand(rng, 1, N, K)
    sfa[0, 77, 3], sfa[0, 199, 65], sfb[0, N - 1, 0] = 0x7F, 0xFF, 0x7F
    for layout in ("plain", "blocked"):
        bad = torch.isnan(run(a, sfa, b, sfb, torch.float32, layout)[0]).cpu()
        want = torch.zeros(N, M, dtype=torch.bool)
        want[:, 77] = want[:, 199] = want[N - 1] = True
        assert torch.equal(bad, want)


@pytest.mark.parametrize("M,N,K,L", [(128, 16, 16384, 1), (300, 5, 8192, 1), (100, 50, 7168, 1), (130, 300, 4096, 1)])
def test_split_k_repeats_its_bits(M, N, K, L):
    assert g.nvfp4_gemm_plan(M, N, K, L)["k_splits"] > 1
    rng = np.random.default_rng(M)
    (a, sfa), (b, sfb) = operand(rng, L, M, K), operand(rng, L, N, K)
    first = run(a, sfa, b, sfb, torch.float32, "blocked")
    for _ in range(3):
        assert torch.equal(run(a, sfa, b, sfb, torch.float32, "blocked"), first)


def test_small_n_agrees():
    """N = 4: the library's N-vector product, within both sides' tolerance."""
    M, N, K = 1000, 4, 4096
    rng = np.random.default_rng(4)
    (a, sfa), (b, sfb) = operand(rng, 1, M, K), operand(rng, 1, N, K)
    want, size = reference(a, sfa, b, sfb)
    got = run(a, sfa, b, sfb, torch.float16, "blocked")
    c = torch.zeros(N * M, dtype=torch.float16, device="cuda")
    g.nvfp4_gemm_small_n(dev(a), dev(b), dev(synth.to_blocked(sfa)), dev(synth.to_blocked(sfb)), c, M, N, K, 1, "blocked",
                         alpha=2.0 ** -8)
    ref.check_product(c.reshape(1, N, M), want * 2.0 ** -8, size * 2.0 ** -8, K, torch.float16)
    fine = np.abs(want) < 65000
    ref.check_product(got.float().cpu()[torch.from_numpy(fine)], want[fine], size[fine], K, torch.float16)


def test_workspace_is_shared_by_calls_on_a_stream():
    """One workspace for products of different shapes in a row."""
    shapes = [(128, 16, 16384), (300, 60, 8192), (77, 3, 4096), (130, 300, 4096)]
    ws = torch.zeros(max(g.nvfp4_gemm_workspace_bytes(M, N, K, 1) for M, N, K in shapes), dtype=torch.uint8, device="cuda")
    for M, N, K in shapes * 2:
        rng = np.random.default_rng([M, N, K])
        (a, sfa), (b, sfb) = operand(rng, 1, M, K), operand(rng, 1, N, K)
        c = torch.zeros(N * M, device="cuda")
        g.nvfp4_gemm(dev(a), dev(b), dev(sfa), dev(sfb), c, M, N, K, 1, "plain", workspace=ws)
        want, size = reference(a, sfa, b, sfb)
        ref.check_product(c, want, size, K, torch.float32, f"{M}x{N}x{K}")


@pytest.mark.parametrize("M,N,K", [(128, 16, 16384), (300, 200, 544), (2050, 2600, 96)])
def test_on_streams_and_in_a_graph(M, N, K):
    rng = np.random.default_rng(K)
    (a, sfa), (b, sfb) = operand(rng, 1, M, K), operand(rng, 1, N, K)
    ops = [dev(x) for x in (a, b, synth.to_blocked(sfa), synth.to_blocked(sfb))]
    need = g.nvfp4_gemm_workspace_bytes(M, N, K, 1)

    def call(c, ws):
        g.nvfp4_gemm(*ops, c, M, N, K, 1, "blocked", workspace=ws)

    make = lambda: (torch.zeros(N, M, dtype=torch.bfloat16, device="cuda"),  # noqa: E731
                    torch.zeros(need, dtype=torch.uint8, device="cuda"))
    want, ws = make()
    call(want, ws)
    sides = [torch.cuda.Stream() for _ in range(2)]
    outs = [make() for _ in sides]
    for s, (c, w) in zip(sides, outs):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(4):
                call(c, w)
    torch.cuda.synchronize()
    for c, _ in outs:
        assert torch.equal(c, want)
    c, ws = make()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(c, ws)
    for _ in range(3):
        c.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c, want)
        ops[0].copy_(ops[0].flip(1))                      # other weights, eagerly, between the replays
        call(want, ws)
        torch.cuda.synchronize()


def test_far_rows():
    """Operand A past 2^32 bytes: the last batch's product is its own."""
    M, N, K, L = 1 << 18, 2, 16384, 3                     # 6.4 GB of codes
    codes = torch.zeros(L, M, K // 2, dtype=torch.uint8, device="cuda")
    sfa = torch.zeros(L * M * (K // 16), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(1)
    (a, sa), (b, sfb) = operand(rng, 1, 64, K), operand(rng, L, N, K)
    codes[L - 1, M - 64:] = dev(a[0])
    sfa[-64 * (K // 16):] = dev(sa.reshape(-1))
    c = torch.full((L, N, M), 7.0, device="cuda")
    ws = torch.zeros(g.nvfp4_gemm_workspace_bytes(M, N, K, L), dtype=torch.uint8, device="cuda")
    g.nvfp4_gemm(codes, dev(b), sfa, dev(sfb), c, M, N, K, L, "plain", workspace=ws if ws.numel() else None)
    want, size = reference(a, sa, b[L - 1:], sfb[L - 1:])
    ref.check_product(c[L - 1:, :, M - 64:], want, size, K, torch.float32)
    assert not c[:L - 1].any() and not c[L - 1, :, :M - 64].any()


# alpha, ga, gb whose product, or part of it, is no normal float32: below its
# range, subnormal, above it on the way, above it beside sums of zero
FAR_SCALES = [(1.0, 2.0 ** -75 * 1.3, 2.0 ** -75 * 1.7), (1.0, 2.0 ** -70 * 1.1, 2.0 ** -70 * 1.3), (2.0 ** 60, 2.0 ** 100, 2.0 ** -120),
              (-2.0 ** -100, 2.0 ** -60, 2.0 ** 120), (1.0, 1e-40, 2.0 ** 20), (2.0 ** -149, 2.0 ** 127, 2.0 ** 20)]


def check_far(got, want, size, K, dtype, what):
    """check_product's bound on each result. Its bound on their norm is relative and does not
    hold here: many results lie below the type's normal numbers, where steps are absolute."""
    off = np.abs(got.double().cpu().numpy().reshape(want.shape) - want) - ref.product_tolerance(K, size, want, dtype)
    fine = np.abs(want) < torch.finfo(dtype).max * 0.99
    assert off[fine].max() <= 0, f"{what}: worst by {off[fine].max():.3g}"


@pytest.mark.parametrize("M,N,K", [(70, 5, 512), (70, 40, 512), (300, 200, 544), (3000, 3500, 96), (128, 16, 16384)])
def test_scales_far_from_one(M, N, K):
    """Scales whose product leaves float32's range where the scaled sums do not (product_tolerance counts four
    float32 roundings and half of the least step); sums of zero stay zero beside a product that overflows."""
    rng = np.random.default_rng([M, N, K, 2])
    (a, sfa), (b, sfb) = operand(rng, 1, M, K, "edge"), operand(rng, 1, N, K, "edge")
    sfa[0, M // 2] = 0
    want, size = reference(a, sfa, b, sfb)
    for alpha, ga, gb in FAR_SCALES:
        f = np.float64(np.float32(alpha)) * np.float64(np.float32(ga)) * np.float64(np.float32(gb))
        for dtype in DTYPES:
            got = run(a, sfa, b, sfb, dtype, "blocked", alpha, ga, gb)
            check_far(got, want * f, size * abs(f), K, dtype, f"{dtype} {alpha} {ga} {gb}")
    got = run(a, sfa, b, sfb, torch.float32, "plain", 1.0, 2.0 ** 100, 2.0 ** 100).double().cpu().numpy()
    assert (got[0, :, M // 2] == 0).all()
    sure = np.abs(want) > ref.product_tolerance(K, size, want, torch.float32)      # the sum's sign
    assert sure.any() and np.array_equal(got[sure], np.sign(want[sure]) * np.inf)
