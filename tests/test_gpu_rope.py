"""GPU: rotary positions against a 64-bit form: types, layouts, parts of the head,
strides, far and negative positions, in place, and the gradient against the formula's
and against differences."""
import numpy as np
import pytest

import attention_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_gemv_amd as g  # noqa: E402

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def inputs(seed, T, H, D, R, dtype, far=100000):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((T, H, D)) * 3).to(dtype)
    positions = torch.from_numpy(rng.integers(-far // 8, far, T))
    f = torch.tensor(g.nvfp4_rope_frequencies(R, 10000.0), dtype=torch.float64)
    return x, positions, f


def check(x, positions, f, R, layout, dtype, factor=1.0, transpose=False, out=None, **kw):
    T, H, D = x.shape
    dx = x.cuda()
    out = torch.full((T, H, D), float("nan"), dtype=dtype, device="cuda") if out is None else out
    g.nvfp4_rope(dx, out, positions.cuda(), f.cuda(), T, H, D, R, layout, factor=factor, transpose=transpose, **kw)
    xd = x.double().numpy()
    want = ref.rope(xd, positions.numpy(), f.numpy(), R, layout, np.float64(np.float32(factor)), transpose)
    ref.check_rope(out, xd, want, R, layout, factor, dtype)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("T,H,D,R", [(1, 1, 2, 2), (1, 40, 128, 128), (3, 5, 64, 32), (7, 2, 96, 96), (2, 3, 80, 20), (5, 1, 33, 32),
                                     (130, 9, 128, 64), (1100, 3, 64, 64), (4, 1, 2048, 2048), (2, 700, 256, 192), (9, 4, 24, 16)])
def test_matches_the_64_bit_form(T, H, D, R, dtype, layout):
    x, positions, f = inputs([T, H, D, R], T, H, D, R, DTYPES[dtype])
    check(x, positions, f, R, layout, DTYPES[dtype], factor=1.25 if T % 2 else 1.0)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_far_positions_are_as_exact_as_near_ones(layout):
    x, _, f = inputs(1, 64, 2, 128, 128, torch.float32)
    positions = torch.cat([torch.arange(16) + 2 ** 30, -torch.arange(16) - 2 ** 20, torch.arange(16) * 999983, torch.arange(16)])
    check(x, positions, f, 128, layout, torch.float32)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", sorted(DTYPES))
def test_strides_and_in_place(dtype, layout):
    dt = DTYPES[dtype]
    T, H, D, R = 19, 6, 64, 48
    x, positions, f = inputs(2, T, H + 3, D + 4, R, dt)
    packed = x.cuda()
    view = packed[:, 1:1 + H, :D]
    want = ref.rope(x[:, 1:1 + H, :D].double().numpy(), positions.numpy(), f.numpy(), R, layout)
    out = torch.full((H, T, D), float("nan"), dtype=dt, device="cuda")          # heads outside, tokens inside
    g.nvfp4_rope(view, out, positions.cuda(), f.cuda(), T, H, D, R, layout, token_stride=view.stride(0), head_stride=view.stride(1),
                 out_token_stride=D, out_head_stride=T * D)
    ref.check_rope(out.transpose(0, 1), x[:, 1:1 + H, :D].double().numpy(), want, R, layout, 1.0, dt)
    g.nvfp4_rope(view, view, positions.cuda(), f.cuda(), T, H, D, R, layout, token_stride=view.stride(0), head_stride=view.stride(1))
    assert torch.equal(view, out.transpose(0, 1))
    left = torch.ones(T, H + 3, D + 4, dtype=torch.bool)
    left[:, 1:1 + H, :D] = False
    assert torch.equal(packed.cpu()[left], x[left]), "values beside the heads changed"


def test_broadcast_input_and_values_that_are_not_finite():
    x, positions, f = inputs(3, 5, 1, 32, 16, torch.float32)
    x[2, 0, 3], x[4, 0, 20] = float("nan"), float("inf")
    dx = x[:, 0].cuda().contiguous()
    out = torch.empty(5, 7, 32, device="cuda")
    g.nvfp4_rope(dx, out, positions.cuda(), f.cuda(), 5, 7, 32, 16, token_stride=32, head_stride=0)
    assert torch.equal(out.nan_to_num(nan=7.0), out[:, :1].expand(5, 7, 32).nan_to_num(nan=7.0))
    nan = torch.isnan(out[:, 0]).cpu()
    assert nan.sum() == 2 and nan[2, 3] and nan[2, 11] and out[4, 0, 20] == float("inf")


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_gradient_by_the_formula_and_by_differences(layout):
    T, H, D, R, factor = 6, 3, 32, 24, 1.5
    x, positions, f = inputs(4, T, H, D, R, torch.float32, far=500)
    gen = torch.Generator().manual_seed(4)
    go = torch.randn(T, H, D, generator=gen)
    check(go, positions, f, R, layout, torch.float32, factor=factor, transpose=True)
    args = (positions.cuda(), f.cuda(), T, H, D, R, layout)
    gx = torch.empty(T, H, D, device="cuda")
    g.nvfp4_rope(go.cuda(), gx, *args, factor=factor, transpose=True)

    def loss(v):
        out = torch.empty_like(v)
        g.nvfp4_rope(v, out, *args, factor=factor)
        return (out.double() * go.cuda().double()).sum()

    # the map is linear: a difference of any width is the gradient; its sums of T H D
    # float32 results, each within 2^-21 of 6 at most, are off by 2^-21 * 6 * 3 * n in all
    for seed in range(4):
        way = torch.randn(T, H, D, generator=gen).cuda()
        xd = x.cuda()
        by_difference = (loss(xd + way) - loss(xd - way)) / 2
        formula = (gx.double() * ((xd + way).double() - (xd - way).double()) / 2).sum()
        assert abs(by_difference - formula) <= 2.0 ** -21 * 18 * T * H * D


def test_a_captured_call_replays_and_streams():
    T, H, D, R = 33, 4, 64, 64
    x, positions, f = inputs(5, T, H, D, R, torch.bfloat16)
    dx, dp, df, out = x.cuda(), positions.cuda(), f.cuda(), torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        g.nvfp4_rope(dx, out, dp, df, T, H, D, R)
    side.synchronize()
    want = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.nvfp4_rope(dx, out, dp, df, T, H, D, R)
    for k in range(3):
        dp.copy_(positions + k)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        eager = torch.empty_like(out)
        g.nvfp4_rope(dx, eager, dp, df, T, H, D, R)
        assert torch.equal(out, eager) and torch.equal(out, want) == (k == 0)


def test_binding_refuses_what_does_not_fit():
    x, positions, f = inputs(6, 4, 2, 64, 64, torch.float32)
    dx, dp, df = x.cuda(), positions.cuda(), f.cuda()
    out = torch.empty_like(dx)
    for bad, what in ((lambda: g.nvfp4_rope(dx, out, dp, df, 5, 2, 64, 64), "holds"),
                      (lambda: g.nvfp4_rope(dx, out, dp[:3], df, 4, 2, 64, 64), "positions holds"),
                      (lambda: g.nvfp4_rope(dx, out, dp.int(), df, 4, 2, 64, 64), "int32, not int64"),
                      (lambda: g.nvfp4_rope(dx, out, dp, df.float(), 4, 2, 64, 64), "float32, not float64"),
                      (lambda: g.nvfp4_rope(dx, out.half(), dp, df, 4, 2, 64, 64), "out is torch.float16"),
                      (lambda: g.nvfp4_rope(dx[:, :1], out, dp, df, 4, 1, 64, 64), "not contiguous"),
                      (lambda: g.nvfp4_rope(dx[:, :, ::2], out, dp, df, 4, 2, 32, 32, token_stride=128, head_stride=64), "rows of x"),
                      (lambda: g.nvfp4_rope(dx, out, dp, df, 4, 2, 64, 64, token_stride=1000, head_stride=64), "holds")):
        with pytest.raises(ValueError, match=what):
            bad()
    with pytest.raises(g.Nvfp4Error):
        g.nvfp4_rope(dx, out, dp, df, 4, 2, 64, 64, layout=7)
