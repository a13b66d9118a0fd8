"""Caches for the tests of attention: rows of sequences in pages in any order, NaN scales everywhere else."""
import numpy as np

import attention_reference as ref


def poisoned(rng, lengths, page_size, heads, D, spare=3, width=None):
    """A cache whose pages hold rows of the sequences, in any order, and NaN scales everywhere else; its table."""
    held = [-(-n // page_size) for n in lengths]
    width = width or max(1, max(held))
    pages = sum(held) + spare
    c = ref.Cache(rng, pages, page_size, heads, D)
    order = rng.permutation(pages)
    table = np.full((len(lengths), width), -1, np.int32)
    for name in ("ks", "vs"):
        scales, keep = getattr(c, name), np.zeros((pages, page_size), bool)
        at = 0
        for b, n in enumerate(lengths):
            table[b, :held[b]] = order[at:at + held[b]]
            for j in range(held[b]):
                keep[order[at + j], :min(page_size, n - j * page_size)] = True
            at += held[b]
        scales.transpose(0, 2, 1, 3)[~keep] = 0x7F
    return c, table
