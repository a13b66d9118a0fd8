"""CPU checks of the FP4 linear layers' C ABI: every refusal comes before any HIP
call, the binding checks types and sizes, plans and workspaces are consistent."""
import ctypes
import math
import os
import random
import re

import pytest

import block_scaled_fp4_gemv_amd as g
from conftest import no_gpu_only

P = 0x100000        # fake, aligned device addresses (never dereferenced: every call here is refused)
INF, NAN = float("inf"), float("nan")


def quantize(x=P, dtype=1, gs=P, codes=P, scales=P, rows=4, K=64, L=1, rs=64, bs=256, lay=1):
    return g.lib().nvfp4_quantize(x, dtype, gs, codes, scales, rows, K, L, rs, bs, lay, None)


def global_scale(x=P, dtype=1, scale=P, rows=4, K=64, L=1, rs=64, bs=256, ws=P, n=256):
    return g.lib().nvfp4_global_scale(x, dtype, scale, rows, K, L, rs, bs, ws, n, None)


def dequantize(codes=P, scales=P, gs=P, out=P, dtype=1, rows=4, K=64, L=1, lay=1):
    return g.lib().nvfp4_dequantize(codes, scales, gs, out, dtype, rows, K, L, lay, None)


def gemm(a=P, b=P, sfa=P, sfb=P, c=P, dtype=1, M=64, N=64, K=64, L=1, lay=1, alpha=1.0, ga=P, gb=P, ws=None, n=0):
    return g.lib().nvfp4_gemm(a, b, sfa, sfb, c, dtype, M, N, K, L, lay, alpha, ga, gb, ws, n, None)


def experts(a=P, b=P, sfa=P, sfb=P, c=P, dtype=1, M=64, K=64, E=4, rows=8, per=2, lay=1, off=P, order=P, alpha=1.0,
            ga=P, gb=P, ws=None, n=0):
    return g.lib().nvfp4_gemm_experts(a, b, sfa, sfb, c, dtype, M, K, E, rows, per, lay, off, order, alpha, ga, gb, ws,
                                      n, None)


def route(logits=P, dtype=1, bias=P, ids=P, weights=P, off=P, order=P, T=400, E=8, k=2, score=0, n_group=1, topk_group=1,
          group_top=1, renorm=1, scaling=1.0, ws=P, n=1 << 20, opts=True):
    o = g.Routing(score, n_group, topk_group, group_top, renorm, scaling)
    return g.lib().nvfp4_moe_route(logits, dtype, bias, ids, weights, off, order, T, E, k,
                                   ctypes.byref(o) if opts else None, ws, n, None)


def combine(y=P, dtype=1, ids=P, weights=P, out=P, T=4, k=2, M=64):
    return g.lib().nvfp4_moe_combine(y, dtype, ids, weights, out, T, k, M, None)


NULL, SHAPE, ALIGN, LAYOUT = (g.NVFP4_ERR_NULL_POINTER, g.NVFP4_ERR_INVALID_SHAPE, g.NVFP4_ERR_MISALIGNED,
                              g.NVFP4_ERR_INVALID_LAYOUT)
WORK, SCALE, STRIDE, TYPE, ROUTING = (g.NVFP4_ERR_WORKSPACE, g.NVFP4_ERR_INVALID_SCALE, g.NVFP4_ERR_INVALID_STRIDE,
                                      g.NVFP4_ERR_INVALID_TYPE, g.NVFP4_ERR_INVALID_ROUTING)


@pytest.mark.parametrize("call,bad,status", [
    (quantize, dict(x=None), NULL), (quantize, dict(codes=None), NULL), (quantize, dict(scales=None), NULL),
    (quantize, dict(dtype=3), TYPE), (quantize, dict(rows=0), SHAPE), (quantize, dict(K=48), SHAPE),
    (quantize, dict(L=0), SHAPE), (quantize, dict(rows=-1), SHAPE), (quantize, dict(rows=2 ** 31), SHAPE),
    (quantize, dict(lay=2), LAYOUT), (quantize, dict(rs=63), STRIDE), (quantize, dict(bs=-1), STRIDE),
    (quantize, dict(rs=2 ** 40), STRIDE), (quantize, dict(x=P + 1), ALIGN), (quantize, dict(dtype=2, x=P + 2), ALIGN),
    (quantize, dict(codes=P + 4), ALIGN), (quantize, dict(scales=P + 2), ALIGN), (quantize, dict(gs=P + 2), ALIGN),
    (quantize, dict(rows=2 ** 29, K=2 ** 20, rs=2 ** 20), SHAPE),
    (global_scale, dict(x=None), NULL), (global_scale, dict(scale=None), NULL), (global_scale, dict(ws=None), WORK),
    (global_scale, dict(n=255), WORK), (global_scale, dict(ws=P + 8), WORK), (global_scale, dict(dtype=-1), TYPE),
    (global_scale, dict(rows=0), SHAPE), (global_scale, dict(rows=2 ** 39, L=2 ** 39), SHAPE),
    (global_scale, dict(rs=10), STRIDE), (global_scale, dict(scale=P + 2), ALIGN),
    (dequantize, dict(codes=None), NULL), (dequantize, dict(out=None), NULL), (dequantize, dict(dtype=7), TYPE),
    (dequantize, dict(K=16), SHAPE), (dequantize, dict(lay=-1), LAYOUT), (dequantize, dict(codes=P + 1), ALIGN),
    (dequantize, dict(out=P + 1), ALIGN), (dequantize, dict(dtype=2, out=P + 2), ALIGN),
    (gemm, dict(a=None), NULL), (gemm, dict(b=None), NULL), (gemm, dict(sfa=None), NULL), (gemm, dict(sfb=None), NULL),
    (gemm, dict(c=None), NULL), (gemm, dict(dtype=9), TYPE), (gemm, dict(M=0), SHAPE), (gemm, dict(N=0), SHAPE),
    (gemm, dict(K=33), SHAPE), (gemm, dict(K=2 ** 23), SHAPE), (gemm, dict(L=0), SHAPE), (gemm, dict(N=2 ** 31), SHAPE),
    (gemm, dict(M=2 ** 30, N=2 ** 30), SHAPE), (gemm, dict(lay=5), LAYOUT), (gemm, dict(a=P + 8), ALIGN),
    (gemm, dict(b=P + 8), ALIGN), (gemm, dict(sfa=P + 4), ALIGN), (gemm, dict(sfb=P + 4), ALIGN),
    (gemm, dict(c=P + 1), ALIGN), (gemm, dict(dtype=2, c=P + 2), ALIGN), (gemm, dict(ga=P + 1), ALIGN),
    (gemm, dict(alpha=NAN), SCALE), (gemm, dict(alpha=INF), SCALE),
    (experts, dict(off=None), NULL), (experts, dict(order=None), NULL),
    (experts, dict(a=None), NULL), (experts, dict(dtype=3), TYPE), (experts, dict(E=0), SHAPE),
    (experts, dict(E=1025), SHAPE), (experts, dict(rows=0), SHAPE), (experts, dict(per=0), SHAPE),
    (experts, dict(per=2 ** 31), SHAPE), (experts, dict(K=0), SHAPE), (experts, dict(off=P + 2), ALIGN),
    (experts, dict(order=P + 1), ALIGN), (experts, dict(alpha=-INF), SCALE), (experts, dict(lay=3), LAYOUT),
    (route, dict(logits=None), NULL), (route, dict(ids=None), NULL), (route, dict(opts=False), NULL),
    (route, dict(dtype=3), TYPE), (route, dict(T=0), SHAPE), (route, dict(E=0), SHAPE), (route, dict(k=0), SHAPE),
    (route, dict(k=9), SHAPE), (route, dict(E=1025), SHAPE), (route, dict(E=128, k=65), SHAPE),
    (route, dict(T=2 ** 30), SHAPE), (route, dict(score=2), ROUTING), (route, dict(n_group=3), ROUTING),
    (route, dict(n_group=0), ROUTING), (route, dict(n_group=4, topk_group=5), ROUTING),
    (route, dict(topk_group=0), ROUTING), (route, dict(group_top=0), ROUTING), (route, dict(group_top=3), ROUTING),
    (route, dict(n_group=8, topk_group=4, group_top=2), ROUTING), (route, dict(E=128, n_group=128), ROUTING),
    (route, dict(renorm=2), ROUTING), (route, dict(scaling=NAN), SCALE), (route, dict(ids=P + 2), ALIGN),
    (route, dict(logits=P + 1), ALIGN), (route, dict(bias=P + 2), ALIGN), (route, dict(ws=None), WORK),
    (route, dict(n=8), WORK), (route, dict(ws=P + 16), WORK),
    (combine, dict(y=None), NULL), (combine, dict(ids=None), NULL), (combine, dict(out=None), NULL),
    (combine, dict(dtype=4), TYPE), (combine, dict(T=0), SHAPE), (combine, dict(k=0), SHAPE), (combine, dict(k=65), SHAPE),
    (combine, dict(M=0), SHAPE), (combine, dict(T=2 ** 30), SHAPE), (combine, dict(M=2 ** 31), SHAPE),
    (combine, dict(y=P + 1), ALIGN), (combine, dict(out=P + 1), ALIGN), (combine, dict(weights=P + 2), ALIGN),
], ids=lambda v: v.__name__ if callable(v) else "-".join(map(str, v)) if isinstance(v, dict) else str(v))
def test_refused(call, bad, status):
    assert call(**bad) == status


def test_products_that_split_k_want_a_workspace():
    M, N, K = 128, 16, 16384
    need = g.nvfp4_gemm_workspace_bytes(M, N, K, 1)
    assert need > 0 and need % 256 == 0 and g.nvfp4_gemm_plan(M, N, K, 1)["k_splits"] > 1
    assert gemm(M=M, N=N, K=K, ws=None, n=need) == WORK
    assert gemm(M=M, N=N, K=K, ws=P, n=need - 1) == WORK
    assert gemm(M=M, N=N, K=K, ws=P + 16, n=need) == WORK
    need = g.nvfp4_gemm_experts_workspace_bytes(M, K, 4, 16)
    assert need > 0
    assert experts(M=M, K=K, rows=8, per=2, ws=None, n=need) == WORK
    assert experts(M=M, K=K, rows=8, per=2, ws=P, n=need - 256) == WORK


def test_experts_rows_within_32_bit_offsets():
    """The rows are gathered by 32-bit offsets: rows * K / 2 is at most 2^32 bytes."""
    assert experts(M=1, K=64, E=1, rows=2 ** 27 + 1, per=1) == SHAPE
    assert experts(M=1, K=64, E=1, rows=2 ** 27, per=1, a=P + 4) == ALIGN


SHAPES = [(1, 1, 32, 1), (7168, 1, 16384, 1), (128, 16, 2048, 1), (7168, 16, 2048, 1), (1000, 33, 4096, 3),
          (4096, 64, 7168, 8), (4096, 333, 7168, 1), (7168, 4096, 16384, 1), (127, 1000, 64, 1), (513, 129, 160, 2),
          (8192, 4096, 16352, 2), (1, 4096, 16384, 1), (20000, 1, 32, 1), (64, 64, 1 << 22, 1), (1 << 20, 64, 64, 1)]


@pytest.mark.parametrize("M,N,K,L", SHAPES)
def test_plans_cover_the_shape(M, N, K, L):
    p = g.nvfp4_gemm_plan(M, N, K, L)
    tiles = g.cdiv(M, p["tile_m"]) * g.cdiv(N, p["tile_n"]) * L
    assert p["workgroups"] == tiles * p["k_splits"]
    assert p["k_per_split"] % 128 == 0 and 1 <= p["k_splits"] <= 16
    assert (p["k_splits"] - 1) * p["k_per_split"] < K <= p["k_splits"] * p["k_per_split"]
    need = g.nvfp4_gemm_workspace_bytes(M, N, K, L)
    assert (need > 0) == (p["k_splits"] > 1)
    if need:
        assert tiles <= 16384 and 65536 + p["k_splits"] * L * N * M * 4 <= need <= 65536 + (64 << 20) + 256


def test_workspace_bytes_of_bad_shapes_are_zero():
    assert g.nvfp4_gemm_workspace_bytes(0, 16, 2048, 1) == 0
    assert g.nvfp4_gemm_workspace_bytes(128, 16, 2047, 1) == 0
    assert g.nvfp4_gemm_experts_workspace_bytes(128, 64, 2000, 16) == 0
    assert g.nvfp4_moe_route_workspace_bytes(4, 8, 9) == 0
    with pytest.raises(g.Nvfp4Error):
        g.nvfp4_gemm_plan(128, 0, 64, 1)


class Fake:
    """A device tensor's face: dtype, size, contiguity."""
    is_cuda = True

    def __init__(self, n, dtype="torch.uint8", size=1):
        self.n, self.dtype, self.size = n, dtype, size

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return P

    def numel(self):
        return self.n

    def element_size(self):
        return self.size


def test_binding_checks_types_and_sizes():
    u8, f32, i32 = Fake(1 << 20), Fake(1 << 20, "torch.float32", 4), Fake(1 << 20, "torch.int32", 4)
    bf = Fake(1 << 20, "torch.bfloat16", 2)
    with pytest.raises(ValueError, match="c holds"):
        g.nvfp4_gemm(u8, u8, u8, u8, Fake(63 * 64, "torch.bfloat16", 2), 64, 64, 64, 1, "plain")
    with pytest.raises(ValueError, match="sfb holds"):
        g.nvfp4_gemm(u8, u8, u8, Fake(255), bf, 64, 64, 64, 1, "plain")
    with pytest.raises(ValueError, match="none of float16"):
        g.nvfp4_gemm(u8, u8, u8, u8, Fake(1 << 20, "torch.float64", 8), 64, 64, 64, 1, "plain")
    with pytest.raises(ValueError, match="scale_a is"):
        g.nvfp4_gemm(u8, u8, u8, u8, bf, 64, 64, 64, 1, "plain", scale_a=bf)
    with pytest.raises(ValueError, match="need dtype"):
        g.nvfp4_gemm(u8, u8, u8, u8, P, 64, 64, 64, 1, "plain")
    with pytest.raises(ValueError, match="offsets holds"):
        g.nvfp4_gemm_experts(u8, u8, u8, u8, bf, 64, 64, 4, 8, 2, "plain", Fake(4, "torch.int32", 4), i32)
    with pytest.raises(ValueError, match="order is"):
        g.nvfp4_gemm_experts(u8, u8, u8, u8, bf, 64, 64, 4, 8, 2, "plain", i32, f32)
    with pytest.raises(ValueError, match="ids is"):
        g.nvfp4_moe_combine(bf, f32, f32, bf, 4, 2, 64)
    with pytest.raises(ValueError, match="different types"):
        g.nvfp4_moe_combine(bf, i32, f32, f32, 4, 2, 64)
    with pytest.raises(ValueError, match="weights holds"):
        g.nvfp4_moe_route(f32, i32, Fake(7, "torch.float32", 4), i32, i32, 4, 8, 2, workspace=u8)
    with pytest.raises(ValueError, match="codes holds"):
        g.nvfp4_dequantize(Fake(10), u8, bf, 4, 64, 1, "plain")


class FakeView(Fake):
    """A view that is not contiguous, over `held` elements of memory from its first on."""

    def __init__(self, n, dtype, size, held):
        super().__init__(n, dtype, size)
        self.held = held

    def is_contiguous(self):
        return False

    def storage_offset(self):
        return 0

    def untyped_storage(self):
        return self

    def nbytes(self):
        return self.held * self.size


@pytest.mark.parametrize("call", [
    lambda x, **kw: g.nvfp4_global_scale(x, Fake(1, "torch.float32", 4), 4, 64, 1, Fake(256), **kw),
    lambda x, **kw: g.nvfp4_quantize(x, Fake(128), Fake(16), 4, 64, 1, "plain", **kw)], ids=["global_scale", "quantize"])
def test_a_view_wants_its_strides(call):
    """Rows 80 apart, taken as dense ones for want of strides, would be read wrongly without a word."""
    x = FakeView(4 * 64, "torch.bfloat16", 2, 3 * 80 + 64)
    with pytest.raises(ValueError, match="not contiguous"):
        call(x)
    with pytest.raises(ValueError, match="x holds 304 elements, the shape needs 307"):
        call(x, row_stride=81)


@pytest.mark.parametrize("call", [
    lambda x, **kw: g.nvfp4_global_scale(x, Fake(1, "torch.float32", 4), 4, 64, 1, Fake(256), dtype="torch.float32", **kw),
    lambda x, **kw: g.nvfp4_quantize(x, Fake(128), Fake(16), 4, 64, 1, "plain", dtype="torch.float32", **kw)],
    ids=["global_scale", "quantize"])
def test_a_given_type_counts_in_the_tensors_bytes(call):
    """float32 read from a tensor of 2-byte elements: half as many fit."""
    with pytest.raises(ValueError, match="x holds 255 elements, the shape needs 256"):
        call(Fake(511, "torch.bfloat16", 2))
    with pytest.raises(ValueError, match="x holds 303 elements, the shape needs 304"):
        call(FakeView(256, "torch.bfloat16", 2, 607), row_stride=80)


@pytest.mark.parametrize("call", [
    lambda **kw: g.nvfp4_global_scale(Fake(256, "torch.float32", 4), Fake(1, "torch.float32", 4), 4, 64, 1, **kw),
    lambda **kw: g.nvfp4_gemm(*[Fake(1 << 20)] * 4, Fake(2048, "torch.float32", 4), 128, 16, 16384, 1, "plain", **kw),
    lambda **kw: g.nvfp4_gemm_experts(*[Fake(1 << 22)] * 4, Fake(2048, "torch.float32", 4), 128, 16384, 4, 8, 2, "plain",
                                      Fake(5, "torch.int32", 4), Fake(16, "torch.int32", 4), **kw),
    lambda **kw: g.nvfp4_moe_route(Fake(3200, "torch.float32", 4), *[Fake(800, t, 4) for t in (
        "torch.int32", "torch.float32", "torch.int32", "torch.int32")], 400, 8, 2, **kw)],
    ids=["global_scale", "gemm", "gemm_experts", "moe_route"])
def test_workspace_bytes_are_the_tensors(call):
    """A size given beside the tensor is no larger than it: the library believes the size."""
    with pytest.raises(ValueError, match="workspace holds 128 bytes, the shape needs"):
        call(workspace=Fake(128), workspace_bytes=1 << 30)
    for ws in (Fake(128), P):
        with pytest.raises(ValueError, match="workspace_bytes is -1"):
            call(workspace=ws, workspace_bytes=-1)
    with pytest.raises(g.Nvfp4Error) as e:
        call(workspace=Fake(128), stream=0)
    assert e.value.status == WORK


def test_workspace_max_serves_every_shape():
    """A product's workspace does not rise with its rows; the documented size holds all of them."""
    text = open(os.path.join(os.path.dirname(g.PKG_DIR), "include", "nvfp4_gemv.h")).read()
    most = int(re.search(r"#define NVFP4_WORKSPACE_MAX_BYTES (\d+)", text).group(1))
    assert most == g.NVFP4_WORKSPACE_MAX_BYTES and most % 256 == 0
    assert g.nvfp4_gemm_workspace_bytes(2048, 64, 7168, 1) > g.nvfp4_gemm_workspace_bytes(2048, 256, 7168, 1)
    rng = random.Random(5)
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    near = 0
    for _ in range(4000):
        M, N, K = log(1, 1 << 20), log(1, 1 << 16), 32 * log(1, 1 << 17)
        got = max(g.nvfp4_gemm_workspace_bytes(M, N, K, log(1, 64)), g.nvfp4_gemm_experts_workspace_bytes(M, K, log(1, 1024), N),
                  g.nvfp4_moe_route_workspace_bytes(N, log(64, 1024), log(1, 64)))
        near = max(near, got)
        assert got <= most, (M, N, K)
    assert near > most // 2, "the sweep does not come near the size"
    assert g.nvfp4_moe_route_workspace_bytes(1 << 24, 1024, 64) <= most
    assert g.nvfp4_global_scale_workspace_bytes() <= most


G = 2 ** 24 - 1         # workgroups of 256 threads that a launch holds
# (call, arguments, largest value of one of them, that argument): the header's limits
LIMITS = [(quantize, dict(K=32, rs=32, bs=0, lay=1), 128 * (G // 8), "rows"), (quantize, dict(K=64, bs=0, lay=0), 64 * G, "rows"),
          (quantize, dict(rows=1, bs=0, lay=0), G, "L"), (dequantize, dict(rows=64, K=64), G, "L"),
          (route, dict(E=8, k=2), 16 * G, "T"), (route, dict(E=8, k=1), 16 * G, "T"), (route, dict(E=257, k=2), 4 * G, "T"),
          (route, dict(E=64, k=16), 4 * G, "T"), (combine, dict(k=2, M=512), 4 * G, "T"),
          (combine, dict(k=2, M=512, dtype=2), 2 * G, "T"), (combine, dict(T=256, k=1), 8 * G, "M")]


@pytest.mark.parametrize("call,args,most,name", LIMITS,
                         ids=lambda v: v.__name__ if callable(v) else str(v) if isinstance(v, (int, str)) else "")
def test_documented_limits_past_the_end(call, args, most, name):
    assert call(**args, **{name: most + 1}) == SHAPE


@no_gpu_only
@pytest.mark.parametrize("call,args,most,name", LIMITS,
                         ids=lambda v: v.__name__ if callable(v) else str(v) if isinstance(v, (int, str)) else "")
def test_documented_limits_are_reached(call, args, most, name):
    assert call(**args, **{name: most}) == g.NVFP4_ERR_HIP


def test_product_limits():
    """Workgroups of a product: the plan and the product refuse alike."""
    assert gemm(M=2 ** 30, N=2 ** 12, K=32) == SHAPE
    with pytest.raises(g.Nvfp4Error) as e:
        g.nvfp4_gemm_plan(2 ** 30, 2 ** 12, 32, 1)
    assert e.value.status == SHAPE
    assert experts(M=2 ** 30, K=32, E=4, rows=2 ** 12, per=1) == SHAPE
