"""Oracle of the int8 cache with one fp32 scale per (block, kv head).

TEST INFRASTRUCTURE ONLY (see the package docstring).  ``write`` follows the
format's definition token by token and block by block in numpy fp32, whose
divisions, products and rounding are IEEE's, so codes and scales can be
compared bit for bit; ``widen`` gives the values the codes stand for, on which
``oracle.attention`` (fp64) is the reference of the attention.
"""
from __future__ import annotations

import numpy as np

BLOCK = 16
FLOOR = np.float32(2.0 ** -60)
LARGEST = np.finfo(np.float32).max
f32 = np.float32


def _codes(x, inv):
    y = np.rint(x.astype(f32) * inv)
    y = np.where(np.isnan(y), 0, np.clip(y, -127, 127))
    return y.astype(np.int8)


def write(k, v, block_tables, context_lens, query_start_loc, k_cache, v_cache, k_scales, v_scales,
          num_blocks=None):
    """In place: the rows k, v (fp32 [T, Hkv, D]) of every sequence at its last
    positions.  Returns whether a non-finite element was seen."""
    odd = False
    for s in range(len(context_lens)):
        t, end = int(query_start_loc[s]), int(query_start_loc[s + 1])
        p = int(context_lens[s]) - (end - t)
        while t < end:
            o = p % BLOCK
            n = min(BLOCK - o, end - t)
            b = int(block_tables[s][p // BLOCK])
            for x, cache, scales in ((k, k_cache, k_scales), (v, v_cache, v_scales)):
                for h in range(cache.shape[2]):
                    rows = x[t:t + n, h].astype(f32)
                    fine = np.isfinite(rows)
                    odd |= not fine.all()
                    a = np.abs(rows[fine]).max() if fine.any() else f32(0)
                    new = max(f32(a) / f32(127), FLOOR)
                    if o > 0:
                        old = scales[b, h]
                        if not (old >= FLOOR and old <= LARGEST):
                            old = FLOOR
                        new = max(old, new)
                        if new > old:
                            ratio = f32(old / new)
                            part = cache[b, :o, h].astype(f32) * ratio
                            cache[b, :o, h] = np.rint(part).astype(np.int8)
                    scales[b, h] = new
                    with np.errstate(invalid="ignore"):
                        cache[b, o:o + n, h] = _codes(rows, f32(f32(1) / new))
            t, p = t + n, p + n
    return odd


def widen(codes, scales):
    """fp32 values [blocks, 16, Hkv, D] of codes and scales [blocks, Hkv]; a
    scale below 2^-60 counts as 2^-60."""
    s = np.where(scales < FLOOR, FLOOR, scales).astype(f32)
    return codes.astype(f32) * s[:, None, :, None]
