"""Plain 64-bit forms of rotary positions, the paged NVFP4 cache and attention over
it, for the tests: numpy and torch on the CPU, written from the definitions, with no
code of the library."""
from __future__ import annotations

import numpy as np
import torch

import fp4_reference as fp4


def rope(x, positions, frequencies, R, layout, factor=1.0, transpose=False):
    """x float64 [T][H][D] -> float64; angles as exact products in extended precision."""
    y = x.copy()
    a = positions.astype(np.longdouble)[:, None] * frequencies.astype(np.longdouble)[None, :]
    # np's longdouble pi has 64 bits: taken off in turns, then two parts of 2 pi
    n = np.rint(a / (2 * np.longdouble(np.pi)))
    hi, lo = np.longdouble(6.283185307179586232), np.longdouble(2.4492935982947064e-16)
    r = (a - n * hi) - n * lo
    c, s = (factor * np.cos(r)).astype(np.float64)[:, None], (factor * np.sin(r)).astype(np.float64)[:, None]
    if transpose:
        s = -s
    i0 = np.arange(0, R, 2) if layout == "interleaved" else np.arange(R // 2)
    i1 = i0 + (1 if layout == "interleaved" else R // 2)
    x0, x1 = x[..., i0], x[..., i1]
    y[..., i0], y[..., i1] = x0 * c - x1 * s, x0 * s + x1 * c
    return y


def check_rope(got, x, ref, R, layout, factor, dtype):
    """cos and sin within 2^-22 of the true ones (angle 2^-24, their own sums and roundings
    2^-23), once more rounded with factor; two products and a sum in float32; the rounding to dtype."""
    i0 = np.arange(0, R, 2) if layout == "interleaved" else np.arange(R // 2)
    i1 = i0 + (1 if layout == "interleaved" else R // 2)
    size = np.zeros_like(ref)
    size[..., i0] = size[..., i1] = abs(factor) * (np.abs(x[..., i0]) + np.abs(x[..., i1]))
    tol = size * (2.0 ** -22 + 3 * 2.0 ** -24) + fp4.HALF_STEP[dtype] * (1 + 2.0 ** -10) * np.abs(ref) + fp4.LEAST[dtype]
    g = got.double().cpu().numpy()
    assert np.array_equal(g[..., R:], x[..., R:])
    assert (np.abs(g - ref) <= tol).all(), np.abs(g - ref).max()


class Cache:
    """numpy arrays of a cache: codes, scale bytes of keys and values, global scales."""

    def __init__(self, rng, pages, page_size, heads, D, gk=0.01, gv=0.02, fill=None):
        self.pages, self.page_size, self.heads, self.D = pages, page_size, heads, D
        self.gk, self.gv = np.float64(np.float32(gk)), np.float64(np.float32(gv))
        for name in ("k", "v"):
            if fill is None:
                x = rng.standard_normal((pages, heads, page_size, D)) * np.exp(rng.standard_normal(D) * 0.3)
                codes, scales = fp4.quantize(x, self.gk if name == "k" else self.gv)
                codes = fp4.pack(codes)
            else:
                codes = np.full((pages, heads, page_size, D // 2), fill[0], np.uint8)
                scales = np.full((pages, heads, page_size, D // 16), fill[1], np.uint8)
            setattr(self, name + "c", codes)
            setattr(self, name + "s", scales)

    def rows(self, name, slots):
        """Values float64 [n][heads][D] of slots."""
        page, place = slots // self.page_size, slots % self.page_size
        codes, scales = getattr(self, name + "c")[page, :, place], getattr(self, name + "s")[page, :, place]
        return fp4.values(codes, scales) * (self.gk if name == "k" else self.gv)


def attention(cache, q, offsets, lengths, table, max_q, max_length, scale, causal=True, window=0):
    """q float64 [T][H][D] -> dict of float64 arrays: out, lse [T][H], written [T] and, for the
    tolerance, size = sum p |v|, all = sum |v| and spread = the largest sum_d |scale q k| of a visible position."""
    T, H, D = q.shape
    G = H // cache.heads
    got = {"out": np.zeros((T, H, D)), "lse": np.full((T, H), -np.inf), "written": np.zeros(T, bool),
           "size": np.zeros((T, H, D)), "all": np.zeros((T, H, D)), "spread": np.zeros((T, H)), "count": np.zeros((T, H))}
    for b in range(len(lengths)):
        first = min(max(int(offsets[b]), 0), T)
        end = min(max(int(offsets[b + 1]), first), T)
        n, length = end - first, min(max(int(lengths[b]), 0), max_length)
        t = np.arange(length)
        page = table[b, t // cache.page_size].astype(np.int64)
        there = (page >= 0) & (page < cache.pages)
        slots = np.where(there, page, 0) * cache.page_size + t % cache.page_size
        k, v = cache.rows("k", slots), cache.rows("v", slots)
        for i in range(min(n, max_q)):
            p = length - n + i
            see = there & ((t <= p) if causal else (t >= 0))
            if window:
                see &= t > p - window
            row = first + i
            got["written"][row] = True
            if not see.any():
                continue
            kk, vv = np.repeat(k[see], G, 1), np.repeat(v[see], G, 1)               # [n][H][D]
            with np.errstate(invalid="ignore"):
                x = np.einsum("hd,nhd->nh", q[row], kk) * scale
                top = x.max(0)
                e = np.exp(x - top)
                got["lse"][row] = top + np.log(e.sum(0))
                w = e / e.sum(0)
                got["out"][row] = np.einsum("nh,nhd->hd", w, vv)
                got["size"][row] = np.einsum("nh,nhd->hd", w, np.abs(vv))
                got["all"][row] = np.abs(vv).sum(0)
                got["spread"][row] = np.einsum("hd,nhd->nh", np.abs(q[row]), np.abs(kk)).max(0) * abs(scale)
            bad = ~np.isfinite(q[row]).all(-1)
            got["out"][row][bad], got["lse"][row][bad] = np.nan, np.nan
            got["count"][row] = see.sum()
    return got


def check_attention(out, lse, want, dtype, what=""):
    """A logit: D products summed in float32, off by at most 256 steps of 2^-23 of the sum of
    sizes, q's rounding to float16 parts (2^-22) and four roundings of the factors: delta =
    (256 + 2 + 4) 2^-23 spread, and 2^-22 of the exponential. Weights change by twice that (numerator and norm); the
    sums over the positions add a step for each, in the norm and in the values, and so do
    the rescalings of the running maximum (at most one for each). Weights are
    rounded to float16, 2^-11 of each (float32: to two, 2^-22), and as they are held times 2^8,
    whose least step's half is 2^-25, by at most 2^-33 of the largest where they are smaller
    still: 2^-33 sum |v|. Then the rounding to dtype."""
    written = want["written"]
    o, ref = out.double().cpu().numpy(), want["out"]
    delta = (262 * 2.0 ** -23 * want["spread"] + 2.0 ** -22)[..., None]
    steps = (3 * want["count"][..., None] + 64) * 2.0 ** -23
    weight = 2.0 ** -22 if dtype == torch.float32 else 2.0 ** -11
    tol = want["size"] * (2 * delta + steps + weight) + 2.0 ** -33 * want["all"] + fp4.HALF_STEP[dtype] * (1 + 2.0 ** -7) * np.abs(ref) + fp4.LEAST[dtype]
    nan = np.isnan(ref)
    assert np.array_equal(np.isnan(o)[written], nan[written]), f"{what}: NaN at other places"
    fine = written[:, None, None] & ~nan
    off = np.abs(o - ref)[fine] - tol[fine]
    assert off.size == 0 or off.max() <= 0, f"{what}: {np.count_nonzero(off > 0)} of {off.size} off, worst by {off.max():.3g}"
    norm = np.linalg.norm(ref[fine])
    if norm > 0 and np.count_nonzero(fine) >= 64:
        # the errors of the weights and of the logits are independent: far below their bound together
        rel = np.linalg.norm((o - ref)[fine]) / norm
        assert rel <= fp4.HALF_STEP[dtype] + weight * 2 + 2.0 ** -15 * (dtype != torch.float32) + 4e-6, f"{what}: {rel:.3g} off"
    if lse is not None:
        g, r = lse.double().cpu().numpy()[written], want["lse"][written]
        assert np.array_equal(np.isnan(g), np.isnan(r)), what
        assert np.array_equal(np.isneginf(g), np.isneginf(r)), what
        fine = np.isfinite(r)
        tol = (delta + steps)[..., 0][written] + 4 * 2.0 ** -24 * np.abs(np.where(fine, r, 0))
        assert (np.abs(g[fine] - r[fine]) <= tol[fine]).all(), f"{what}: lse off"
