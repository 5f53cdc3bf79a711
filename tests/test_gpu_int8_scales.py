"""Stored scales of the int8 cache that no write makes, and scales at the ends
of their range: pkv_write_int8 bit for bit with the oracle, pkv_attention_int8
against the definition in fp64."""
import numpy as np
import pytest
import torch

from paged_kv_cache_43_gb300 import pkv
from tests.test_gpu_int8 import _lib, Cache, attend, batch, i32, rows, starts, tables, wide  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ write

@pytest.mark.parametrize("stored", [np.nan, np.inf, -np.inf, 0.0, -1.0, 2.0 ** -61, 2.0 ** -60])
@pytest.mark.parametrize("n", [1, 3])
@pytest.mark.parametrize("what", ["zero", "tiny", "nan", "ordinary"])
def test_write_replaces_a_stored_scale_that_is_not_one(stored, n, what):
    """A block continued under a scale that is NaN, infinite or below 2^-60: the
    scale in memory is a sound one afterwards, whatever the new rows hold."""
    cache = Cache(3, 2, 64, seed=n)
    for a, g in ((cache.ks, cache.gpu[2]), (cache.vs, cache.gpu[3])):
        a[:] = stored
        g.fill_(float(stored))
    gen = torch.Generator().manual_seed(5)
    k, v = rows(gen, 2 * n, 2, 64), rows(gen, 2 * n, 2, 64)
    if what != "ordinary":
        k[:], v[:] = {"zero": (0.0, -0.0), "tiny": (1e-30, -1e-25), "nan": (float("nan"),) * 2}[what]
    odd = cache.write(k, v, i32([[0], [2]]), i32([5 + n, 9 + n]), i32([0, n, 2 * n]), n)
    assert odd == (what == "nan")
    assert pkv.get_error() == (pkv.ERR_NONFINITE if odd else 0)
    cache.check()
    for scales in cache.gpu[2:]:
        held = scales[[0, 2]]
        assert torch.isfinite(held).all() and (held >= 2.0 ** -60).all()


# -------------------------------------------------------------- attention

def poison(cache, which, block, head, value):
    """The scale of (block, head) of K or V is `value` on the GPU; returns what undoes it."""
    t = cache.gpu[2 if which == "k" else 3]
    old = float(t[block, head])
    t[block, head] = value

    def undo():
        t[block, head] = old
    return undo


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("value", [np.nan, np.inf])
@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("hq,hkv,d,bound", [(8, 2, 128, None), (4, 2, 64, None), (6, 2, 128, 9000),
                                            (32, 2, 64, 9000), (260, 2, 64, None)])
def test_a_bad_scale_reaches_no_row_that_does_not_see_its_block(which, value, window, hq, hkv, d,
                                                                bound):
    """Chunks whose rows see different blocks: a scale that is NaN or infinite
    makes the rows that see a key of its block NaN, and leaves the others as they
    are."""
    q, ctx = [64, 100], [64, 333]
    b = batch(ctx, q, hq, hkv, d, seed=hq + d)
    cache, qs, bt, cl, qsl, scale = b
    # (row tiles side by side and, with the loose bound, parts of the keys)
    kw = dict(window=window, max_context_len=bound)
    group = hq // hkv
    pos = np.concatenate([np.arange(c - n, c) for n, c in zip(q, ctx)])
    seq = np.repeat([0, 1], q)
    for s, j in ((0, 3), (0, 1), (1, 20), (1, 17), (1, 14), (1, 16)):
        undo = poison(cache, which, int(bt[s, j]), 1, value)
        got, ref, tol = attend(*b, **kw)       # (the oracle's copy keeps the sound scale)
        undo()
        sees = (seq == s) & (pos >= 16 * j)
        if window:
            sees &= pos - window + 1 <= 16 * j + 15
        mine = np.zeros(got.shape[:2], bool)
        mine[sees, group:] = True
        assert mine.any() and not mine.all()
        assert np.isnan(got[mine]).all()
        bad = ~(np.abs(got - ref) <= tol)
        assert not bad[~mine].any(), (s, j, np.argwhere(bad.any(-1) & ~mine)[:4])
    assert pkv.get_error() == 0


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("ctx,chunk,hq,hkv,bound", [
    ([100, 60], 1, 8, 4, None),            # a CTA for the row
    ([1200, 600], 1, 8, 4, None),          # splits that merge in a cluster
    ([1200, 600], 1, 8, 4, 200000),        # teams
    ([1200, 600], 20, 8, 4, None),         # chunks, parts of the keys
    ([300, 200], 64, 40, 1, None),         # chunks
    ([300, 200], 5, 130, 1, None)])        # more q heads than a row tile has rows
def test_an_infinite_scale_makes_the_rows_that_see_it_nan(which, sign, ctx, chunk, hq, hkv, bound):
    """Also where every score against the block's codes has the same sign."""
    b = batch(ctx, [chunk] * 2, hq, hkv, 64, seed=7)
    cache, qs, bt, cl, qsl, scale = b
    blk = int(bt[0, 1])
    cache.kc[blk] = np.abs(cache.kc[blk])       # scores of this block: the query's sign
    cache.gpu[0][blk] = cache.gpu[0][blk].abs()
    qs[:] = sign * qs.abs()
    good, ref, tol = attend(*b, max_context_len=bound)
    assert (np.abs(good - ref) <= tol).all()
    undo = poison(cache, which, blk, 0, np.inf)
    got, _, _ = attend(*b, max_context_len=bound)
    undo()
    assert np.isnan(got[:chunk, :hq // hkv]).all()
    got[:chunk, :hq // hkv] = ref[:chunk, :hq // hkv]
    assert (np.abs(got - ref) <= tol).all()
    assert pkv.get_error() == 0


def definition(cache, qs, bt, cl, qsl, scale):
    """fp64 output of every row, and the tolerance: the output's rounding (2^-8 of
    it), and for each weight its rounding to fp16 and the error of its exponent
    (2^-11 and 2^-14, as where the other attention tests say why) relative to what
    it weighs: the largest magnitude that its block's V scale allows."""
    k, v = (x.astype(np.float64) for x in cache.values())
    q = qs.float().numpy().astype(np.float64)
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    group = q.shape[1] // k.shape[2]
    for s in range(len(cl)):
        L, t0, t1 = int(cl[s]), int(qsl[s]), int(qsl[s + 1])
        at = bt[s, :-(-L // 16)].numpy()
        top = 127 * np.repeat(np.maximum(cache.vs[at].astype(np.float64), 2.0 ** -60), 16, 0)[:L]
        for h in range(q.shape[1]):
            kh = k[at, :, h // group].reshape(-1, q.shape[2])[:L]
            vh = v[at, :, h // group].reshape(-1, q.shape[2])[:L]
            x = q[t0:t1, h] @ kh.T * scale
            x[np.arange(L)[None] > np.arange(L - (t1 - t0), L)[:, None]] = -np.inf
            w = np.exp(x - x.max(1, keepdims=True))
            w /= w.sum(1, keepdims=True)
            out[t0:t1, h] = w @ vh
            tol[t0:t1, h] = (2.0 ** -8 * np.abs(out[t0:t1, h])
                             + (2.0 ** -11 + 2.0 ** -14) * (w @ top[:, h // group])[:, None])
    return out, tol


@pytest.mark.parametrize("ctx,chunk,hq,hkv,d,bound", [
    ([100, 60], 1, 8, 4, 64, None),        # a CTA for the row
    ([1200, 600], 1, 8, 4, 128, None),     # splits that merge in a cluster
    ([1200, 600], 1, 8, 4, 64, 200000),    # teams
    ([1200, 600], 1, 8, 4, 128, 200000),
    ([1200, 600], 20, 8, 4, 128, None),    # chunks, parts of the keys
    ([300, 200], 150, 40, 1, 64, None),    # chunks
    ([300, 200], 150, 8, 2, 128, None),
    ([300, 200], 5, 130, 1, 64, None)])    # more q heads than a row tile has rows
@pytest.mark.parametrize("large", [20, 60, 118])
@pytest.mark.parametrize("sharp", [0.0, 1.0, 12.0])
def test_v_scales_at_both_ends_of_their_range(ctx, chunk, hq, hkv, d, bound, large, sharp):
    """Blocks of V of about 2^large beside blocks of zeros and ordinary ones, in
    any order: the weights of the small blocks count in full."""
    rng = np.random.default_rng(int(sharp) + large)
    b = batch(ctx, [min(chunk, c) for c in ctx], hq, hkv, d, seed=3)
    cache, qs, bt, cl, qsl, scale = b
    power = rng.choice([large, 0, -60, -200], cache.vs.shape, p=[0.2, 0.2, 0.2, 0.4])
    with np.errstate(under="ignore"):
        cache.vs[:] = np.maximum(cache.vs.astype(np.float64) * 2.0 ** power,
                                 2.0 ** -60).astype(np.float32)
    cache.vc[np.repeat((power == -200)[:, None], 16, 1)] = 0       # (blocks of zeros)
    cache.gpu[1].copy_(torch.from_numpy(cache.vc))
    cache.gpu[3].copy_(torch.from_numpy(cache.vs))
    qs = (qs.float() * sharp).to(torch.bfloat16)
    out = torch.full(qs.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    pkv.attention_int8(out, qs.cuda(), *cache.gpu[:2], wide(bt, bound).cuda(), cl.cuda(),
                       qsl.cuda(), scale, *cache.gpu[2:], max_query_len=chunk,
                       max_context_len=bound or max(ctx))
    assert pkv.get_error() == 0
    ref, tol = definition(cache, qs, bt, cl, qsl, scale)
    off = np.abs(out.float().cpu().numpy().astype(np.float64) - ref)
    assert (off <= tol).all(), float((off / tol).max())
