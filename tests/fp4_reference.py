"""Plain 64-bit forms of the FP4 linear layers and routed experts, for the
tests: numpy on the CPU, written from the definitions, with no code of the
library and none of its kernels' ways of deciding a rounding."""
from __future__ import annotations

import numpy as np
import torch

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)
E4M3 = np.array([(b % 8) * 2.0 ** -9 if b < 8 else (8 + b % 8) * 2.0 ** (b // 8 - 10) for b in range(127)], np.float64)

# half a step of a type, relative to the value, and the least step's half
HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
LEAST = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}


def cdiv(a, b):
    return -(-a // b)


def nearest_code(v, table):
    """Index of the table's nearest entry, ties to the even index; v >= 0, may be inf."""
    mids = (table[1:] + table[:-1]) / 2
    below, above = np.searchsorted(mids, v, "left"), np.searchsorted(mids, v, "right")
    # below < above: v is a midpoint, between entries `below` and `above`
    return np.where(below == above, below, below + below % 2)


def global_scale(x):
    """x float64 array of values -> the float32 global scale, as float64."""
    size = np.abs(x[np.isfinite(x)])
    top = size.max() if size.size else 0.0
    if top == 0.0:
        return 1.0
    # the product of two float32 is exact in float64: one rounding
    return float(max(np.float32(top * np.float64(np.float32(1.0 / 2688.0))), np.float32(2.0 ** -100)))


def quantize(x, g):
    """x float64 [..., K] -> (codes uint8 [..., K] with the sign in bit 3, scale codes [..., K/16])."""
    blocks = x.reshape(*x.shape[:-1], -1, 16)
    nan = np.isnan(blocks).any(-1)
    if not (np.isfinite(g) and g >= 2.0 ** -100):
        nan[...] = True
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        amax = np.where(nan, 0.0, np.abs(blocks).max(-1))
        scale = nearest_code(np.minimum(amax / (6 * g), 1e9), E4M3)
        unit = (E4M3[scale] * g)[..., None]
        ratio = np.where(unit > 0, np.abs(np.nan_to_num(blocks, nan=0.0, posinf=np.inf, neginf=-np.inf)) / unit, 0.0)
    code = nearest_code(ratio, E2M1).astype(np.uint8) | (np.signbit(blocks).astype(np.uint8) << 3)
    code = np.where((scale == 0)[..., None] | nan[..., None], 0, code)
    return code.astype(np.uint8).reshape(x.shape), np.where(nan, 0x7F, scale).astype(np.uint8)


def pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(packed):
    out = np.empty(packed.shape[:-1] + (2 * packed.shape[-1],), np.uint8)
    out[..., 0::2], out[..., 1::2] = packed & 15, packed >> 4
    return out


def e4m3(codes):
    """Values of E4M3 codes, NaN for 0x7F and 0xFF."""
    table = np.concatenate([E4M3, [np.nan], -E4M3, [np.nan]])
    return table[codes]


def values(packed, scales):
    """packed [..., K/2], plain scale codes [..., K/16] -> float64 [..., K]."""
    c = unpack(packed)
    v = np.where(c >= 8, -E2M1[c & 7], E2M1[c & 7])
    return v * np.repeat(e4m3(scales), 16, axis=-1)


def from_blocked(blocked, rows, K):
    """Blocked bytes of one batch -> plain codes [rows][K/16], by the position formula."""
    r, kb = np.arange(rows)[:, None], np.arange(K // 16)[None, :]
    return blocked[((r // 128) * cdiv(K, 64) + kb // 4) * 512 + (r % 32) * 16 + ((r % 128) // 32) * 4 + kb % 4]


def blocked_pad_mask(rows, K):
    """True where a byte of one batch's blocked scales is padding."""
    mask = np.ones(cdiv(rows, 128) * cdiv(K, 64) * 512, bool)
    r, kb = np.arange(rows)[:, None], np.arange(K // 16)[None, :]
    mask[((r // 128) * cdiv(K, 64) + kb // 4) * 512 + (r % 32) * 16 + ((r % 128) // 32) * 4 + kb % 4] = False
    return mask


def route(logits, bias, k, score, n_group=1, topk_group=1, group_top=1, renormalize=True, scaling=1.0):
    """logits float64 [T][E] -> (ids [T][k], weights float64 [T][k]); token by token."""
    T, E = logits.shape
    ids, weights = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        x = np.where(np.isnan(logits[t]), -np.inf, logits[t])
        masked = x == -np.inf
        with np.errstate(invalid="ignore", over="ignore"):
            if score == "softmax":
                top = x.max()
                e = np.where(masked, 0.0, np.where(x == top, 1.0, np.exp(x - top)))
                s = e / e.sum() if e.sum() > 0 else e
            else:
                s = np.where(masked, 0.0, 1 / (1 + np.exp(-x)))
            pick = s + (bias if bias is not None else 0.0)
        pick = np.where(masked | np.isnan(pick), -np.inf, pick)
        size = E // n_group
        if n_group > 1:
            value = []
            for g in range(n_group):
                best = sorted((v for v in pick[g * size:(g + 1) * size] if v > -np.inf), reverse=True)[:group_top]
                value.append(sum(best) if best else -np.inf)
            keep = sorted(range(n_group), key=lambda g: (-value[g], g))[:topk_group]
            pick = np.where(np.isin(np.arange(E) // size, keep), pick, -np.inf)
        best = [e for e in sorted(range(E), key=lambda e: (-pick[e], e)) if pick[e] > -np.inf][:k]
        ids[t, :len(best)] = best
        weights[t, :len(best)] = s[best]
        if renormalize:
            total = weights[t].sum()
            weights[t] = weights[t] / total if total > 0 else 0.0
    return ids, weights * np.float64(np.float32(scaling))


def lists(ids, E):
    """ids [T][k] -> (offsets [E+1], order of the slots in a list)."""
    flat = ids.reshape(-1)
    slots = np.nonzero((flat >= 0) & (flat < E))[0]
    order = slots[np.argsort(flat[slots], kind="stable")]
    counts = np.bincount(flat[slots], minlength=E)
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), order.astype(np.int32)


def product_tolerance(K, sum_abs, ref, dtype):
    """How far a float32-accumulated product of K exact terms may be from `ref`:
    K additions, each off by at most a step (2^-23) of a partial sum, which is at
    most the sum of the sizes; four float32 roundings of the scale and the scaled
    sum; the rounding to `dtype` (half a step, or half of the least one)."""
    return K * 2.0 ** -23 * sum_abs + (4 * 2.0 ** -24 + HALF_STEP[dtype] * (1 + 2.0 ** -10)) * np.abs(ref) + LEAST[dtype]


def check_product(got, ref, sum_abs, K, dtype, what=""):
    """got: torch tensor; ref, sum_abs: float64 arrays of the scaled product."""
    g = got.double().cpu().numpy().reshape(ref.shape)
    top = {torch.float16: 65504.0, torch.bfloat16: 3.38e38, torch.float32: 3.4e38}[dtype]
    fine = np.abs(ref) < top * 0.99
    assert np.isfinite(g[fine]).all(), f"{what}: not finite where the definition is"
    off = np.abs(g - ref)[fine] - product_tolerance(K, sum_abs, ref, dtype)[fine]
    assert off.size == 0 or off.max() <= 0, f"{what}: {np.count_nonzero(off > 0)} outputs off, worst by {off.max():.3g}"
    # the errors of K roundings of partial sums are independent: their 2-norm grows with the root of K
    norm = np.linalg.norm(ref[fine])
    if norm > 0:
        rel = np.linalg.norm((g - ref)[fine]) / norm
        scale = np.linalg.norm(sum_abs[fine]) / norm
        assert rel <= HALF_STEP[dtype] + 2.0 ** -22 + np.sqrt(K) * 2.0 ** -23 * max(1.0, scale / np.sqrt(K)), f"{what}: {rel:.3g} off"


def equals_at_the_last_pick(rng, T, E, k, sigmoid):
    """Logits (float32 tensor) whose order float32 scores cannot tell at the last of k picks:
    there, two or three experts of one logit stand among others of a larger one, all of the
    same float32 score."""
    x = torch.full((T, E), -8.0)
    for t in range(T):
        at = torch.from_numpy(rng.permutation(E))
        x[t, at[:k - 1]] = 60.0 if sigmoid else 30.0        # picked before; softmax: they take all of the sum
        close = at[k - 1:k + 3].sort().values
        low, high = (20.0, 24.0) if sigmoid else (2.0, 2.25) if k > 1 else (2.0, 2.0 + 2.0 ** -20)
        x[t, close] = low
        x[t, close[2 + t % 2]] = high
    return x
