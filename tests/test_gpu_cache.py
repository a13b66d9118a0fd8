"""GPU: keys and values written into the pages of an NVFP4 cache and read back: codes
and scales bit for bit those of the definition (and of nvfp4_quantize), everything else
left as it was."""
import numpy as np
import pytest

import attention_reference as ref
import fp4_reference as fp4

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import block_scaled_fp4_gemv_amd as g  # noqa: E402

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def on_device(c, code_page_stride=None, scale_page_stride=None):
    """A reference Cache on the device: (handle, its four tensors as [pages][heads][page_size][..] views)."""
    views = []
    for name, stride in (("kc", code_page_stride), ("ks", scale_page_stride), ("vc", code_page_stride), ("vs", scale_page_stride)):
        a = torch.from_numpy(getattr(c, name)).cuda()
        if stride is not None:
            room = torch.full((c.pages, stride), 0xA5, dtype=torch.uint8, device="cuda")
            view = room.as_strided(a.shape, (stride, a.stride(1), a.stride(2), 1))
            view.copy_(a)
            a = view
        views.append(a)
    gk, gv = (torch.tensor([v], dtype=torch.float32, device="cuda") for v in (c.gk, c.gv))
    handle = g.Nvfp4Cache(*views, c.pages, c.page_size, c.heads, c.D, k_scale=gk, v_scale=gv, code_page_stride=code_page_stride,
                          scale_page_stride=scale_page_stride)
    return handle, views


def rows_bits(c, x, gl):
    if not len(x):
        return np.zeros((*x.shape[:-1], c.D // 2), np.uint8), np.zeros((*x.shape[:-1], c.D // 16), np.uint8)
    codes, scales = fp4.quantize(x, gl)
    return fp4.pack(codes), scales


@pytest.mark.parametrize("dtype", sorted(DTYPES))
@pytest.mark.parametrize("T,heads,D,page_size,pages", [(1, 1, 32, 16, 1), (1, 8, 128, 16, 5), (33, 2, 96, 32, 4), (64, 3, 64, 16, 9),
                                                       (257, 1, 256, 64, 7), (500, 5, 160, 128, 6), (15, 4, 224, 4096, 1)])
def test_write_and_read_back(T, heads, D, page_size, pages, dtype):
    dt, rng = DTYPES[dtype], np.random.default_rng([T, heads, D])
    c = ref.Cache(rng, pages, page_size, heads, D, gk=0.013, gv=0.4)
    # one token in eight has no place: before, and behind the cache
    slots = rng.permutation(pages * page_size)[:T].astype(np.int64)
    slots[rng.random(T) < 0.125] = -1
    slots[rng.random(T) < 0.0625] = pages * page_size
    k, v = (torch.from_numpy(rng.standard_normal((T, heads, D)) * np.exp(rng.standard_normal(D))).to(dt) for _ in range(2))
    handle, views = on_device(c)
    ds = torch.from_numpy(slots).cuda()
    g.nvfp4_cache_write(handle, k.cuda(), v.cuda(), ds, T)
    kept = (slots >= 0) & (slots < pages * page_size)
    page, place = slots[kept] // page_size, slots[kept] % page_size
    for name, x, gl in (("k", k, c.gk), ("v", v, c.gv)):
        codes, scales = rows_bits(c, x.double().numpy()[kept], gl)
        getattr(c, name + "c")[page, :, place], getattr(c, name + "s")[page, :, place] = codes, scales
    for name, view in zip(("kc", "ks", "vc", "vs"), views):
        assert np.array_equal(view.cpu().numpy(), getattr(c, name)), name
    ko, vo = (torch.full((T, heads, D), float("nan"), dtype=dt, device="cuda") for _ in range(2))
    g.nvfp4_cache_read(handle, ko, vo, ds, T)
    for name, got in (("k", ko), ("v", vo)):
        want = np.zeros((T, heads, D))
        want[kept] = c.rows(name, slots[kept])
        off = np.abs(got.double().cpu().numpy() - want)
        assert (off <= (2.0 ** -24 + fp4.HALF_STEP[dt] * (1 + 2.0 ** -10)) * np.abs(want) + fp4.LEAST[dt]).all()


def test_same_bits_as_quantise_and_dequantise():
    T, heads, D, page_size = 48, 4, 128, 16
    gen = torch.Generator(device="cuda").manual_seed(5)
    k, v = (torch.randn(T, heads, D, device="cuda", generator=gen).bfloat16() for _ in range(2))
    k[3, 1, 40], k[9, 0, 0], v[11, 2, 100] = float("nan"), float("inf"), float("-inf")
    k[5] = 0
    c = ref.Cache(np.random.default_rng(0), 3, page_size, heads, D)
    handle, (kc, ks, vc, vs) = on_device(c)
    slots = torch.arange(T, device="cuda")
    g.nvfp4_cache_write(handle, k, v, slots, T)
    for x, codes, scales, gl in ((k, kc, ks, handle.tensors[4]), (v, vc, vs, handle.tensors[5])):
        q, s = torch.empty(T * heads, D // 2, dtype=torch.uint8, device="cuda"), torch.empty(T * heads, D // 16, dtype=torch.uint8, device="cuda")
        g.nvfp4_quantize(x, q, s, T * heads, D, 1, "plain", global_scale=gl)
        assert torch.equal(codes.transpose(1, 2).reshape(T * heads, D // 2), q)
        assert torch.equal(scales.transpose(1, 2).reshape(T * heads, D // 16), s)
        back = torch.empty(T, heads, D, dtype=torch.float32, device="cuda")
        g.nvfp4_dequantize(q, s, back, T * heads, D, 1, "plain", global_scale=gl)
        ko, vo = torch.empty_like(back), torch.empty_like(back)
        g.nvfp4_cache_read(handle, ko, vo, slots, T)
        got = ko if x is k else vo
        assert torch.equal(got.nan_to_num(nan=1e30), back.nan_to_num(nan=1e30))


def test_views_of_a_packed_projection_and_no_global_scale():
    T, heads, D = 21, 3, 64
    gen = torch.Generator(device="cuda").manual_seed(6)
    packed = torch.randn(T, 4 * heads, D, device="cuda", generator=gen).half()
    k, v = packed[:, 2 * heads:3 * heads], packed[:, 3 * heads:]
    views = [torch.zeros(2, heads, 16, D // n, dtype=torch.uint8, device="cuda") for n in (2, 16, 2, 16)]
    handle = g.Nvfp4Cache(*views, 2, 16, heads, D)
    slots = torch.arange(T, device="cuda") + 3
    g.nvfp4_cache_write(handle, k, v, slots, T, k_strides=(k.stride(0), k.stride(1)), v_strides=(v.stride(0), v.stride(1)))
    for x, codes, scales in ((k, views[0], views[1]), (v, views[2], views[3])):
        want = rows_bits(None, x.double().cpu().numpy(), 1.0)
        for view, w in zip((codes, scales), want):
            got = view.transpose(1, 2).reshape(32, heads, -1).cpu().numpy()
            assert np.array_equal(got[3:3 + T], w) and not got[:3].any() and not got[3 + T:].any()
    with pytest.raises(ValueError, match="not contiguous"):
        g.nvfp4_cache_write(handle, k, v, slots, T)


def test_page_strides_leave_the_gaps():
    rng = np.random.default_rng(7)
    c = ref.Cache(rng, 3, 16, 2, 64)
    code, scale = 16 * 2 * 32 + 48, 16 * 2 * 4 + 16
    handle, views = on_device(c, code, scale)
    T = 20
    slots = rng.permutation(48)[:T]
    x = torch.from_numpy(rng.standard_normal((T, 2, 64))).float()
    g.nvfp4_cache_write(handle, x.cuda(), x.cuda(), torch.from_numpy(slots).cuda(), T)
    for name, view in zip(("k", "k", "v", "v"), views):
        room = view.as_strided((3, view.stride(0)), (view.stride(0), 1))
        assert (room[:, view[0].numel():] == 0xA5).all()
    for name, gl in (("k", c.gk), ("v", c.gv)):
        codes, scales = rows_bits(c, x.double().numpy(), gl)
        vc, vs = (views[0], views[1]) if name == "k" else (views[2], views[3])
        assert np.array_equal(vc.cpu().numpy()[slots // 16, :, slots % 16], codes)
        assert np.array_equal(vs.cpu().numpy()[slots // 16, :, slots % 16], scales)


def test_pages_past_4_gib():
    """Three pages 3 GiB apart: byte offsets pass 32 bits."""
    stride, heads, D = 3 << 30, 1, 64
    room = torch.zeros(2 * stride + (1 << 12), dtype=torch.uint8, device="cuda")
    views = [room[i * 1024:i * 1024 + (16 * D // n)] for i, n in enumerate((2, 16, 2, 16))]
    handle = g.Nvfp4Cache(*views, 3, 16, heads, D, code_page_stride=stride, scale_page_stride=stride)
    gen = torch.Generator(device="cuda").manual_seed(8)
    x = torch.randn(3, heads, D, device="cuda", generator=gen)
    slots = torch.tensor([5, 16 + 6, 32 + 7], device="cuda")
    g.nvfp4_cache_write(handle, x, -x, slots, 3)
    codes, scales = rows_bits(None, x.double().cpu().numpy(), 1.0)
    for t, slot in enumerate(slots.tolist()):
        at = slot // 16 * stride + slot % 16 * 32
        assert np.array_equal(room[at:at + 32].cpu().numpy(), codes[t, 0])
        at = slot // 16 * stride + 1024 + slot % 16 * 4
        assert np.array_equal(room[at:at + 4].cpu().numpy(), scales[t, 0])
    ko, vo = torch.empty_like(x), torch.empty_like(x)
    g.nvfp4_cache_read(handle, ko, vo, slots, 3)
    assert torch.equal(ko, -vo) and np.array_equal(ko.double().cpu().numpy(), fp4.values(codes, scales))


def test_no_token_inside_writes_nothing_and_reads_zeros():
    c = ref.Cache(np.random.default_rng(9), 2, 16, 1, 32)
    handle, views = on_device(c)
    slots = torch.tensor([-1, 32, -2 ** 63, 2 ** 63 - 1, 2 ** 40], device="cuda")
    x = torch.ones(5, 1, 32, device="cuda")
    g.nvfp4_cache_write(handle, x, x, slots, 5)
    for name, view in zip(("kc", "ks", "vc", "vs"), views):
        assert np.array_equal(view.cpu().numpy(), getattr(c, name))
    ko, vo = torch.ones_like(x), torch.ones_like(x)
    g.nvfp4_cache_read(handle, ko, vo, slots, 5)
    assert not ko.any() and not vo.any()


def test_binding_refuses_what_does_not_fit():
    kc, ks, vc, vs = (torch.zeros(2, 3, 16, 64 // n, dtype=torch.uint8, device="cuda") for n in (2, 16, 2, 16))
    with pytest.raises(ValueError, match="k_codes holds"):
        g.Nvfp4Cache(kc, ks, vc, vs, 3, 16, 3, 64)
    with pytest.raises(ValueError, match="v_scales holds"):
        g.Nvfp4Cache(kc, ks, vc, vs[:1], 2, 16, 3, 64)
    with pytest.raises(ValueError, match="not uint8"):
        g.Nvfp4Cache(kc.view(torch.int8), ks, vc, vs, 2, 16, 3, 64)
    with pytest.raises(ValueError, match="float64"):
        g.Nvfp4Cache(kc, ks, vc, vs, 2, 16, 3, 64, k_scale=torch.ones(1, dtype=torch.float64, device="cuda"))
    with pytest.raises(ValueError, match="holds"):
        g.Nvfp4Cache(kc, ks, vc, vs, 2, 16, 3, 64, code_page_stride=1 << 20, scale_page_stride=192)
    handle = g.Nvfp4Cache(kc, ks, vc, vs, 2, 16, 3, 64)
    x, slots = torch.zeros(4, 3, 64, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    for bad, what in ((lambda: g.nvfp4_cache_write(handle, x, x.half(), slots, 4), "v is torch.float16"),
                      (lambda: g.nvfp4_cache_write(handle, x, x, slots.int(), 4), "int32"),
                      (lambda: g.nvfp4_cache_write(handle, x, x, slots, 5), "holds"),
                      (lambda: g.nvfp4_cache_write(handle, x[:, :2], x, slots, 4), "not contiguous"),
                      (lambda: g.nvfp4_cache_write(handle, x.double(), x, slots, 4), "none of"),
                      (lambda: g.nvfp4_cache_read(handle, x, x[:3], slots, 4), "holds")):
        with pytest.raises(ValueError, match=what):
            bad()
