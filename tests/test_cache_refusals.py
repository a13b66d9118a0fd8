"""CPU checks of the C ABI of rotary positions, the paged cache and attention: every
refusal comes before any HIP call, the binding checks types and sizes."""
import ctypes
import math

import pytest

import block_scaled_fp4_gemv_amd as g
from conftest import no_gpu_only

torch = pytest.importorskip("torch")

P = 0x100000        # fake, aligned device addresses (never dereferenced: every call here is refused)
INF, NAN = float("inf"), float("nan")
NULL, SHAPE, ALIGN, WORK = (g.NVFP4_ERR_NULL_POINTER, g.NVFP4_ERR_INVALID_SHAPE, g.NVFP4_ERR_MISALIGNED, g.NVFP4_ERR_WORKSPACE)
SCALE, STRIDE, TYPE, ROT, CACHE = (g.NVFP4_ERR_INVALID_SCALE, g.NVFP4_ERR_INVALID_STRIDE, g.NVFP4_ERR_INVALID_TYPE,
                                   g.NVFP4_ERR_INVALID_ROTATION, g.NVFP4_ERR_INVALID_CACHE)


def rope(x=P, dtype=1, out=2 * P, pos=P, f=P, T=4, H=8, D=128, R=128, xt=1024, xh=128, ot=1024, oh=128, layout=0, factor=1.0,
         transpose=0):
    return g.lib().nvfp4_rope(x, dtype, out, pos, f, T, H, D, R, xt, xh, ot, oh, layout, factor, transpose, None)


def cache_of(kc=P, ks=P, vc=P, vs=P, gk=P, gv=P, pages=10, ps=16, heads=2, D=128, cp=None, sp=None):
    cp = max(heads, 0) * ps * D // 2 if cp is None else cp
    sp = max(heads, 0) * ps * D // 16 if sp is None else sp
    return g.CacheStruct(kc, ks, vc, vs, gk, gv, pages, ps, heads, D, cp, sp)


def split(kw):
    names = ("kc", "ks", "vc", "vs", "gk", "gv", "pages", "ps", "heads", "D", "cp", "sp")
    return {k: v for k, v in kw.items() if k in names}, {k: v for k, v in kw.items() if k not in names}


def write(**kw):
    c, kw = split(kw)
    a = dict(k=P, v=P, dtype=1, slots=P, T=4, kt=256, kh=128, vt=256, vh=128, cache=True)
    a.update(kw)
    ref = ctypes.byref(cache_of(**c)) if a["cache"] else None
    return g.lib().nvfp4_cache_write(ref, a["k"], a["v"], a["dtype"], a["slots"], a["T"], a["kt"], a["kh"], a["vt"], a["vh"], None)


def read(**kw):
    c, kw = split(kw)
    a = dict(k=P, v=P, dtype=1, slots=P, T=4, cache=True)
    a.update(kw)
    ref = ctypes.byref(cache_of(**c)) if a["cache"] else None
    return g.lib().nvfp4_cache_read(ref, a["k"], a["v"], a["dtype"], a["slots"], a["T"], None)


def attend(**kw):
    c, kw = split(kw)
    a = dict(q=P, dtype=1, out=2 * P, lse=P, offsets=P, lengths=P, table=P, T=4, H=8, B=2, width=8, qt=1024, qh=128, max_q=2,
             max_length=100, window=0, scale=0.1, causal=1, ws=P, n=g.NVFP4_WORKSPACE_MAX_BYTES, cache=True, opts=True)
    a.update(kw)
    ref = ctypes.byref(cache_of(**c)) if a["cache"] else None
    o = g.Attention(a["qt"], a["qh"], a["max_q"], a["max_length"], a["window"], a["scale"], a["causal"])
    return g.lib().nvfp4_cache_attention(ref, a["q"], a["dtype"], a["out"], a["lse"], a["offsets"], a["lengths"], a["table"], a["T"],
                                         a["H"], a["B"], a["width"], ctypes.byref(o) if a["opts"] else None, a["ws"], a["n"], None)


BAD_CACHES = [(dict(kc=None), NULL), (dict(ks=None), NULL), (dict(vc=None), NULL), (dict(vs=None), NULL), (dict(cache=False), NULL),
              (dict(pages=0), CACHE), (dict(pages=2 ** 31), CACHE), (dict(ps=8), CACHE), (dict(ps=48), CACHE), (dict(ps=8192), CACHE),
              (dict(heads=0), CACHE), (dict(heads=4097), CACHE), (dict(D=16), CACHE), (dict(D=48), CACHE), (dict(D=288), CACHE),
              (dict(heads=4096, ps=4096, D=256), CACHE), (dict(cp=2032), STRIDE), (dict(sp=240), STRIDE), (dict(cp=2056), STRIDE),
              (dict(sp=264), STRIDE), (dict(cp=2 ** 40), STRIDE), (dict(sp=2 ** 32), STRIDE), (dict(kc=P + 8), ALIGN), (dict(ks=P + 8), ALIGN),
              (dict(vc=P + 4), ALIGN), (dict(vs=P + 4), ALIGN), (dict(gk=P + 2), ALIGN), (dict(gv=P + 1), ALIGN)]


@pytest.mark.parametrize("call,bad,status", [
    (rope, dict(x=None), NULL), (rope, dict(out=None), NULL), (rope, dict(pos=None), NULL), (rope, dict(f=None), NULL),
    (rope, dict(dtype=3), TYPE), (rope, dict(T=0), SHAPE), (rope, dict(H=0), SHAPE), (rope, dict(D=1), SHAPE),
    (rope, dict(R=0), SHAPE), (rope, dict(R=3), SHAPE), (rope, dict(R=130), SHAPE), (rope, dict(D=4096, R=2050), SHAPE),
    (rope, dict(H=2 ** 21), SHAPE), (rope, dict(T=2 ** 41), SHAPE), (rope, dict(T=2 ** 34), SHAPE),
    (rope, dict(layout=2), ROT), (rope, dict(transpose=2), ROT), (rope, dict(factor=NAN), SCALE), (rope, dict(factor=INF), SCALE),
    (rope, dict(xt=-1), STRIDE), (rope, dict(xh=2 ** 40), STRIDE), (rope, dict(ot=1000), STRIDE), (rope, dict(oh=100), STRIDE),
    (rope, dict(ot=0), STRIDE), (rope, dict(out=P, ot=2048), STRIDE), (rope, dict(out=P, T=1, oh=256), STRIDE),
    (rope, dict(x=P + 1), ALIGN), (rope, dict(dtype=2, out=P + 2), ALIGN), (rope, dict(pos=P + 4), ALIGN), (rope, dict(f=P + 4), ALIGN),
    (write, dict(k=None), NULL), (write, dict(v=None), NULL), (write, dict(slots=None), NULL), (write, dict(dtype=-1), TYPE),
    (write, dict(T=0), SHAPE), (write, dict(T=2 ** 28), SHAPE), (write, dict(kt=-1), STRIDE), (write, dict(vh=2 ** 40), STRIDE),
    (write, dict(k=P + 1), ALIGN), (write, dict(dtype=2, v=P + 2), ALIGN), (write, dict(slots=P + 4), ALIGN),
    (read, dict(k=None), NULL), (read, dict(v=None), NULL), (read, dict(slots=None), NULL), (read, dict(dtype=3), TYPE),
    (read, dict(T=-1), SHAPE), (read, dict(T=2 ** 40), SHAPE), (read, dict(k=P + 1), ALIGN), (read, dict(slots=P + 1), ALIGN),
    (attend, dict(q=None), NULL), (attend, dict(out=None), NULL), (attend, dict(offsets=None), NULL),
    (attend, dict(lengths=None), NULL), (attend, dict(table=None), NULL), (attend, dict(opts=False), NULL),
    (attend, dict(dtype=3), TYPE), (attend, dict(D=32), CACHE), (attend, dict(D=160), CACHE), (attend, dict(D=224), CACHE),
    (attend, dict(T=0), SHAPE), (attend, dict(B=0), SHAPE), (attend, dict(H=0), SHAPE), (attend, dict(H=9), SHAPE),
    (attend, dict(H=2 * 1025), SHAPE), (attend, dict(T=2 ** 31), SHAPE), (attend, dict(max_q=0), SHAPE),
    (attend, dict(max_q=5), SHAPE), (attend, dict(T=2 ** 20, max_q=2 ** 20, B=2 ** 11), SHAPE), (attend, dict(max_length=0), SHAPE),
    (attend, dict(max_length=129), SHAPE), (attend, dict(width=0), SHAPE), (attend, dict(width=2 ** 27), SHAPE),
    (attend, dict(max_length=2 ** 31, width=2 ** 30), SHAPE), (attend, dict(T=2 ** 30, max_q=2 ** 29, B=2), SHAPE),
    (attend, dict(window=-1), CACHE), (attend, dict(window=2 ** 31), CACHE), (attend, dict(causal=2), CACHE),
    (attend, dict(scale=NAN), SCALE), (attend, dict(scale=INF), SCALE), (attend, dict(qt=-1), STRIDE), (attend, dict(qh=2 ** 40), STRIDE),
    (attend, dict(q=P + 1), ALIGN), (attend, dict(out=P + 1), ALIGN), (attend, dict(dtype=2, q=P + 2), ALIGN),
    (attend, dict(lse=P + 2), ALIGN), (attend, dict(offsets=P + 2), ALIGN), (attend, dict(lengths=P + 1), ALIGN),
    (attend, dict(table=P + 2), ALIGN),
] + [(call, bad, status) for call in (write, read, attend) for bad, status in BAD_CACHES],
    ids=lambda v: v.__name__ if callable(v) else "-".join(map(str, v)) if isinstance(v, dict) else str(v))
def test_refused(call, bad, status):
    assert call(**bad) == status


def test_workspace_size_of_a_refused_call_is_zero():
    o = g.Attention(1024, 128, 1, 100, 0, 0.1, 1)
    f = g.lib().nvfp4_cache_attention_workspace_bytes
    assert f(None, 1, 4, 8, 2, ctypes.byref(o)) == 0 and f(ctypes.byref(cache_of()), 1, 4, 8, 2, None) == 0
    assert f(ctypes.byref(cache_of()), 7, 4, 8, 2, ctypes.byref(o)) == 0


def tensors(pages=10, ps=16, heads=2, D=128):
    return [torch.zeros(pages, heads, ps, D // n, dtype=torch.uint8) for n in (2, 16, 2, 16)]


def test_binding_wants_device_tensors_of_the_right_type_and_size():
    kc, ks, vc, vs = tensors()
    with pytest.raises(ValueError, match="device"):
        g.Nvfp4Cache(kc, ks, vc, vs, 10, 16, 2, 128)
    cache = g.Nvfp4Cache(P, P, P, P, 10, 16, 2, 128)
    x = torch.zeros(4, 2, 128)
    for call in (lambda: g.nvfp4_cache_write(cache, x, x, P, 4), lambda: g.nvfp4_cache_read(cache, x, x, P, 4),
                 lambda: g.nvfp4_rope(x, P, P, P, 4, 2, 128, 128),
                 lambda: g.nvfp4_cache_attention(cache, x, x, P, P, P, 4, 2, 1, 4, 100, table_width=10)):
        with pytest.raises(ValueError, match="device"):
            call()
    with pytest.raises(ValueError, match="dtype="):
        g.nvfp4_cache_write(cache, P, P, P, 4)
    with pytest.raises(ValueError, match="table_width="):
        g.nvfp4_cache_attention(cache, P, P, P, P, P, 4, 2, 1, 4, 100, dtype=torch.float16)
    with pytest.raises(g.Nvfp4Error) as e:
        g.nvfp4_cache_write(cache, P, P, P, 0, dtype=torch.float16, stream=0)
    assert e.value.status == SHAPE and "nvfp4_cache_write" in str(e.value)


@no_gpu_only
def test_a_good_call_reaches_the_launch():
    """Without a GPU the launch itself is what fails."""
    assert rope() == g.NVFP4_ERR_HIP and write() == g.NVFP4_ERR_HIP and read() == g.NVFP4_ERR_HIP and attend() == g.NVFP4_ERR_HIP
    assert attend(lse=None, gk=None, gv=None) == g.NVFP4_ERR_HIP


def test_status_strings_of_the_new_codes():
    for s in (ROT, CACHE):
        assert g.status_string(s) != "unknown status"
    assert math.isfinite(g.NVFP4_WORKSPACE_MAX_BYTES)
