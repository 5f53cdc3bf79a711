"""Int8 KV cache with a scale per (block, kv head) on the GPU against the
oracle: pkv_write_int8 must give the oracle's codes and scales bit for bit;
pkv_attention_int8 must match the fp64 attention over code * scale.

Tolerance of the attention, per element: the output is rounded to bf16 (2^-8 of
the value); the kernels may round each softmax weight to fp16 (2^-11 of it)
before the product with V, which moves the result by at most 2^-11 max|V|; and
scores of up to 2^6 (log2 units) held to 2^-21 of their size move weights and
their sum by 2^-15 ln 2 each, together under 2^-14 max|V|."""
import numpy as np
import pytest
import torch

import oracle
from oracle import int8 as O8
from paged_kv_cache_43_gb300 import build, pkv
from paged_kv_cache_43_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    pkv.load()
    pkv.get_error(clear=True)
    yield
    assert pkv.get_error(clear=True) == 0


class Cache:
    """An int8 cache on the GPU and the oracle's copy of it.  Scales of blocks
    that were never written are NaN, their codes random."""

    def __init__(self, nb, hkv, d, seed=0):
        rng = np.random.default_rng(seed)
        shape = (nb, 16, hkv, d)
        self.kc = rng.integers(-127, 128, shape, dtype=np.int8)
        self.vc = rng.integers(-127, 128, shape, dtype=np.int8)
        self.ks = np.full((nb, hkv), np.nan, np.float32)
        self.vs = np.full((nb, hkv), np.nan, np.float32)
        self.gpu = [torch.from_numpy(a.copy()).cuda() for a in (self.kc, self.vc, self.ks, self.vs)]

    def write(self, k, v, bt, cl, qsl, max_query_len, **kw):
        """The same write on both sides (k, v: bf16 CPU tensors)."""
        odd = O8.write(k.float().numpy(), v.float().numpy(), bt.numpy(), cl.numpy(), qsl.numpy(),
                       self.kc, self.vc, self.ks, self.vs)
        pkv.write_int8(k.cuda(), v.cuda(), bt.cuda(), cl.cuda(), qsl.cuda(), *self.gpu,
                       max_query_len=max_query_len, **kw)
        return odd

    def check(self):
        for got, want in zip(self.gpu, (self.kc, self.vc, self.ks, self.vs)):
            got = got.cpu().numpy()
            assert got.tobytes() == want.tobytes(), np.argwhere(
                ~((got == want) | ((got != got) & (want != want))))[:5]

    def values(self):
        return O8.widen(self.kc, self.ks), O8.widen(self.vc, self.vs)


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def tables(ctx, nb, seed, pad=0):
    """A table of distinct random blocks for each sequence, -1 behind them."""
    n = [-(-c // 16) for c in ctx]
    assert sum(n) <= nb
    ids = np.random.default_rng(seed).permutation(nb)
    bt = np.full((len(ctx), max(max(n), 1) + pad), -1, np.int32)
    at = 0
    for s, m in enumerate(n):
        bt[s, :m] = ids[at:at + m]
        at += m
    return torch.from_numpy(bt)


def starts(q):
    return i32(np.concatenate([[0], np.cumsum(q)]).tolist())


def rows(gen, *shape, size=1.0):
    return (torch.randn(shape, generator=gen) * size).to(torch.bfloat16)


def fill(cache, ctx, bt, hkv, d, seed, step=None):
    """Writes whole contexts (in chunks of `step` tokens, or at once)."""
    gen = torch.Generator().manual_seed(seed)
    done = [0] * len(ctx)
    while any(a < c for a, c in zip(done, ctx)):
        q = [min(c - a, step or c) for a, c in zip(done, ctx)]
        done = [a + n for a, n in zip(done, q)]
        t = sum(q)
        cache.write(rows(gen, t, hkv, d), rows(gen, t, hkv, d, size=0.7), bt, i32(done), starts(q),
                    max(q))


def tolerance(ref, vmax):
    return 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -14) * vmax


def attend(cache, q, bt, cl, qsl, scale, window=0, out=None, **kw):
    """GPU output and the oracle's (fp64), with the tolerance."""
    kw.setdefault("max_query_len", int((qsl[1:] - qsl[:-1]).max()))
    kw["max_context_len"] = kw.get("max_context_len") or int(cl.max())
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda") if out is None else out
    pkv.attention_int8(out, q.cuda(), cache.gpu[0], cache.gpu[1],
                       wide(bt, kw["max_context_len"]).cuda(), cl.cuda(), qsl.cuda(), scale,
                       cache.gpu[2], cache.gpu[3], sliding_window=window, **kw)
    k, v = cache.values()
    ref, st = oracle.attention(q.float().numpy(), k, v, bt.numpy(), cl.numpy(), qsl.numpy(), scale,
                               window=window)
    assert not st.any()
    live = np.concatenate([bt.numpy()[s, :-(-int(c) // 16)] for s, c in enumerate(cl)])
    vmax = np.abs(v[live[live >= 0]]).max()
    return out.float().cpu().numpy().astype(np.float64), ref, tolerance(ref, vmax)


def check_attention(*args, **kw):
    got, ref, tol = attend(*args, **kw)
    assert np.isfinite(got).all()
    worst = (np.abs(got - ref) / tol).max()
    assert worst <= 1, worst


# ------------------------------------------------------------------ write

@pytest.mark.parametrize("hkv,d", [(8, 128), (1, 64), (5, 64), (3, 128)])
@pytest.mark.parametrize("step", [None, 1, 7, 16, 33])
def test_write_codes_and_scales_bit_exact(hkv, d, step):
    ctx = [1, 15, 16, 17, 33, 40]
    cache = Cache(20, hkv, d, seed=step or 0)
    fill(cache, ctx, tables(ctx, 20, hkv), hkv, d, seed=3, step=step)
    cache.check()
    assert pkv.get_error() == 0


def test_write_growing_scales_round_the_earlier_codes_again():
    """Every later token is twice as large: each step raises the scale."""
    cache = Cache(3, 2, 64)
    bt = i32([[2, 0]])
    gen = torch.Generator().manual_seed(1)
    for n in range(20):
        cache.write(rows(gen, 1, 2, 64, size=2.0 ** n), rows(gen, 1, 2, 64, size=2.0 ** -n), bt,
                    i32([n + 1]), i32([0, 1]), 1)
        cache.check()


def test_write_begins_a_reused_block_anew():
    cache = Cache(2, 2, 64)
    gen = torch.Generator().manual_seed(2)
    for size in (100.0, 0.01):   # the second owner's values are far smaller
        cache.write(rows(gen, 5, 2, 64, size=size), rows(gen, 5, 2, 64, size=size), i32([[1]]),
                    i32([5]), i32([0, 5]), 5)
    cache.check()
    assert float(cache.gpu[2][1].max()) < 0.001


def test_write_zeros_tiny_and_huge_values():
    cache = Cache(4, 1, 64)
    x = torch.zeros(3 * 16, 1, 64, dtype=torch.bfloat16)
    x[16:32] = 1e-30
    x[32:] = 3e38
    x[33] = -3e38
    cache.write(x, x.clone(), i32([[0, 1, 3]]), i32([48]), i32([0, 48]), 48)
    cache.check()
    assert pkv.get_error() == 0


def test_write_nonfinite_elements_are_flagged_and_do_not_reach_the_scale():
    cache = Cache(2, 2, 64)
    gen = torch.Generator().manual_seed(4)
    k = rows(gen, 20, 2, 64)
    k[3, 0, 5] = float("nan")
    k[4, 1, 6] = float("inf")
    k[17, 0, 7] = -float("inf")
    odd = cache.write(k, rows(gen, 20, 2, 64), i32([[1, 0]]), i32([20]), i32([0, 20]), 20)
    assert odd and pkv.get_error() == pkv.ERR_NONFINITE
    cache.check()
    assert cache.kc[1, 3, 0, 5] == 0 and cache.kc[1, 4, 1, 6] == 127 and cache.kc[0, 1, 0, 7] == -127


def test_write_continues_a_block_that_was_never_begun():
    cache = Cache(2, 2, 64)      # NaN scales
    cache.gpu[2][1] = 0.0
    cache.ks[1] = 0.0
    gen = torch.Generator().manual_seed(5)
    cache.write(rows(gen, 2, 2, 64), rows(gen, 2, 2, 64), i32([[0], [1]]), i32([5, 9]),
                i32([0, 1, 2]), 1)
    cache.check()


def test_write_skips_padding_bad_lengths_and_bad_blocks():
    """Sequences without rows write nothing; bad ones are skipped and flagged,
    the others written."""
    ctx = [0, 20, 5, 40, 3, 18]
    bt = tables(ctx, 12, 7)
    cache = Cache(12, 2, 64, seed=1)
    gen = torch.Generator().manual_seed(6)
    q = [0, 20, 5, 1, 3, 18]
    k, v = rows(gen, sum(q), 2, 64), rows(gen, sum(q), 2, 64)
    # (the oracle sees the good sequences only: rows of the bad ones left out)
    good = bt.clone()
    bt[2, 0] = 12                              # no such block
    cl = i32(ctx)
    cl[4] = 2                                  # more rows than keys
    keep = [1, 3, 5]
    take = torch.cat([torch.arange(sum(q[:s]), sum(q[:s + 1])) for s in keep])
    O8.write(k[take].float().numpy(), v[take].float().numpy(), good[keep].numpy(),
             np.array([ctx[s] for s in keep]), starts([q[s] for s in keep]).numpy(), cache.kc,
             cache.vc, cache.ks, cache.vs)
    pkv.write_int8(k.cuda(), v.cuda(), bt.cuda(), cl.cuda(), starts(q).cuda(), *cache.gpu,
                   max_query_len=20)
    assert pkv.get_error() == pkv.ERR_BLOCK_ID | pkv.ERR_QUERY_LEN
    cache.check()
    # a table too short for the length, one row a sequence
    pkv.write_int8(k[:1].cuda(), v[:1].cuda(), bt[1:2, :1].contiguous().cuda(), i32([17]).cuda(),
                   i32([0, 1]).cuda(), *cache.gpu, max_query_len=1)
    assert pkv.get_error() == pkv.ERR_CONTEXT_LEN
    # a sequence with more rows than max_query_len
    pkv.write_int8(k[:2].cuda(), v[:2].cuda(), bt[1:2].cuda(), i32([17]).cuda(),
                   i32([0, 2]).cuda(), *cache.gpu, max_query_len=1)
    assert pkv.get_error() == pkv.ERR_QUERY_LEN
    cache.check()


@pytest.mark.parametrize("seqs", [1, 2, 31, 32, 33, 70, 1100])
def test_write_many_sequences_of_a_few_rows(seqs):
    """The rows of every sequence are found, empty sequences between them."""
    rng = np.random.default_rng(seqs)
    q = rng.integers(0, 4, seqs)
    q[seqs // 2] = 3
    ctx = q + rng.integers(0, 20, seqs) * (q > 0)
    cache = Cache(int((-(-ctx // 16)).sum()) + 1, 1, 64)
    bt = tables(ctx.tolist(), cache.kc.shape[0], 5)
    gen = torch.Generator().manual_seed(8)
    t = int(q.sum())
    cache.write(rows(gen, t, 1, 64), rows(gen, t, 1, 64), bt, i32(ctx.tolist()),
                starts(q.tolist()), int(q.max()))
    cache.check()


# -------------------------------------------------------------- attention

# The bound on the contexts (max_context_len and the table's width) decides
# between the two decode kernels: the longest context (small batches: a CTA per
# split and head), or a bound of this many tokens (teams of warps over equal
# ranges of all the batch's blocks).
LOOSE = 20000
BOUNDS = [None, LOOSE]


def wide(bt, bound):
    """The table with room for `bound` tokens a sequence."""
    more = -(-(bound or 0) // 16) - bt.shape[1]
    return bt if more <= 0 else torch.nn.functional.pad(bt, (0, more), value=-1)

EDGE_CTX = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300, 511, 513, 700]


def batch(ctx, q, hq, hkv, d, seed, step=None, pad=0):
    nb = sum(-(-c // 16) for c in ctx) + 3
    cache = Cache(nb, hkv, d, seed=seed)
    bt = tables(ctx, nb, seed, pad=pad)
    fill(cache, ctx, bt, hkv, d, seed=seed + 1, step=step)
    gen = torch.Generator().manual_seed(seed + 2)
    return cache, rows(gen, sum(q), hq, d), bt, i32(ctx), starts(q), d ** -0.5


@pytest.mark.parametrize("bound", BOUNDS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(4, 4), (8, 2), (8, 1), (12, 4), (32, 2), (5, 1), (24, 2),
                                    (8, 8), (24, 24), (70, 2), (100, 1), (12, 12), (60, 20)])
def test_decode_edge_lengths_and_groups(hq, hkv, d, bound):
    b = batch(EDGE_CTX, [1] * len(EDGE_CTX), hq, hkv, d, seed=hq * 100 + hkv + d, step=100, pad=2)
    for split in (0, 64, 192):
        check_attention(*b, kv_split_tokens=split, max_context_len=bound)
    assert pkv.get_error() == 0


@pytest.mark.parametrize("hq,hkv,d", [(8, 8, 128), (12, 1, 64), (20, 2, 128)])
@pytest.mark.parametrize("ctx", [[129], [1000, 3], [1537, 700, 16], [4100], [16384, 1, 5000]])
def test_decode_few_sequences_merge_their_splits(ctx, hq, hkv, d):
    """A row's splits (up to 16) merge among themselves; shorter sequences of
    the batch have fewer, or none."""
    b = batch(ctx, [1] * len(ctx), hq, hkv, d, seed=hq + len(ctx), step=3000)
    for window in (0, 777):
        check_attention(*b, window=window)
    cache, qs, bt, cl, qsl, scale = b
    bad = bt.clone()
    bad[0, 1] = cache.kc.shape[0]              # the other sequences stay right
    good, ref, tol = attend(*b)
    out = torch.zeros(qs.shape, dtype=torch.bfloat16, device="cuda")
    pkv.attention_int8(out, qs.cuda(), *cache.gpu[:2], bad.cuda(), cl.cuda(), qsl.cuda(), scale,
                       *cache.gpu[2:], max_query_len=1, max_context_len=int(cl.max()))
    assert pkv.get_error() == pkv.ERR_BLOCK_ID
    assert len(ctx) == 1 or (np.abs(out.float().cpu().numpy() - ref) / tol)[1:].max() <= 1


@pytest.mark.parametrize("seqs", [1, 3, 255, 256, 257, 600])
def test_decode_many_short_sequences_and_empty_ones(seqs):
    """Ranges with many sequences in them; sequences without rows, single keys."""
    rng = np.random.default_rng(seqs)
    ctx = rng.integers(1, 70, seqs)
    ctx[seqs // 2] = 900
    full = batch(ctx.tolist(), [1] * seqs, 8, 8, 64, seed=seqs)
    for bound in BOUNDS:
        check_attention(*full, max_context_len=bound)
    cache, qs, bt, cl, qsl, scale = full
    live = rng.random(seqs) < 0.6
    live[seqs // 2] = True
    cl2 = torch.where(torch.from_numpy(live), cl, 0)
    qsl2 = starts(live.astype(int).tolist())
    for bound in BOUNDS:
        got, ref, tol = attend(cache, qs, bt, cl2.to(torch.int32), qsl2, scale,
                               max_context_len=bound,
                               out=torch.full(qs.shape, 7.0, dtype=torch.bfloat16, device="cuda"))
        n = int(live.sum())
        assert (np.abs(got - ref) / tol)[:n].max() <= 1 and (got[n:] == 7.0).all()
    assert pkv.get_error() == 0


@pytest.mark.parametrize("bound", BOUNDS)   # (a loose one cuts the keys into parts)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(4, 4), (8, 2), (32, 8), (3, 1), (10, 2), (16, 1), (128, 1),
                                    (130, 1)])
def test_prefill_edge_chunks(hq, hkv, d, bound):
    q = [1, 5, 16, 63, 64, 65, 97, 1, 40, 130]
    ctx = [1, 5, 40, 63, 130, 65, 97, 2, 200, 333]
    check_attention(*batch(ctx, q, hq, hkv, d, seed=7 * hq + d), max_context_len=bound)
    assert pkv.get_error() == 0


@pytest.mark.parametrize("group", [3, 5, 6, 7, 9, 10, 11, 13, 20, 33, 50, 65, 127])
def test_prefill_row_tiles_of_every_group_size(group):
    """Chunks that end just past the row tiles' and their pairs' ends."""
    tile = 128 // group
    q = sorted({n for m in (1, 2, 4, 6) for n in (m * tile, m * tile + 1, m * 128 // group)})
    check_attention(*batch([n + 150 for n in q], q, group, 1, 64, seed=group))


@pytest.mark.parametrize("window", [0, 700])
@pytest.mark.parametrize("q,ctx,hq,hkv,d", [
    ([40], [3000], 8, 2, 128), ([1, 1, 33, 200], [5, 2000, 1100, 2500], 12, 4, 64),
    ([300], [300], 4, 1, 64), ([128, 2], [4000, 2], 16, 2, 128), ([2, 2, 2], [1, 2, 5], 4, 2, 64)])
def test_prefill_with_few_rows_over_parts_of_the_keys(q, ctx, hq, hkv, d, window):
    """Few row tiles: the keys are cut into parts and merged; parts that rows of
    the tile see nothing of, and short sequences that have fewer tiles."""
    ctx = [max(a, b) for a, b in zip(q, ctx)]
    b = batch(ctx, q, hq, hkv, d, seed=sum(q) + d, step=600)
    nd = next((i for i, n in enumerate(q) if n > 1), len(q))
    for bound in (None, 9000):
        check_attention(*b, window=window, num_decode_seqs=nd, max_context_len=bound)
    assert pkv.get_error() == 0


@pytest.mark.parametrize("bound", [None, 9000])
@pytest.mark.parametrize("chunk", [1, 20])
def test_nan_queries_and_scales_reach_their_rows_only(chunk, bound):
    b = batch([1200, 90], [chunk] * 2, 8, 4, 64, seed=71)
    cache, qs, bt, cl, qsl, scale = b
    good = attend(*b, max_context_len=bound)[0]
    bad = qs.clone()
    bad[chunk - 1, 3, 5] = float("nan")          # the first sequence's last row, head 3
    out = torch.zeros(qs.shape, dtype=torch.bfloat16, device="cuda")
    args = (*cache.gpu[:2], wide(bt, bound).cuda(), cl.cuda(), qsl.cuda(), scale, *cache.gpu[2:])
    kw = dict(max_query_len=chunk, max_context_len=bound or 1200)
    pkv.attention_int8(out, bad.cuda(), *args, **kw)
    got = out.float().cpu().numpy()
    assert np.isnan(got[chunk - 1, 3]).all()
    got[chunk - 1, 3] = good[chunk - 1, 3]
    assert np.array_equal(got, good)
    cache.gpu[3][int(bt[1, 0]), 2] = float("nan")   # V scale of the other's first block, head 2
    pkv.attention_int8(out, qs.cuda(), *args, **kw)
    got = out.float().cpu().numpy()
    assert np.isnan(got[chunk:, 4:6]).all()
    got[chunk:, 4:6] = good[chunk:, 4:6]
    assert np.array_equal(got, good)
    assert pkv.get_error() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_prefill_full_tiles(d):
    q = [128, 129, 256, 300, 1]
    check_attention(*batch([128, 500, 256, 700, 50], q, 8, 8, d, seed=9 + d))
    check_attention(*batch([128, 500, 256, 700, 50], q, 12, 4, d, seed=10 + d))


@pytest.mark.parametrize("bound", BOUNDS)
@pytest.mark.parametrize("window", [1, 17, 100, 1000])
def test_sliding_window_never_reads_blocks_before_it(window, bound):
    q, ctx = [1, 1, 1, 40, 1, 64], [1, 300, 1000, 400, 1500, 1200]
    cache, qs, bt, cl, qsl, scale = batch(ctx, q, 16, 4, 128, seed=window)
    for nd in (-1, 3):
        check_attention(cache, qs, bt, cl, qsl, scale, window=window, num_decode_seqs=nd,
                        max_context_len=bound)
    # blocks wholly before every window: null entries give the same result
    for s in range(len(q)):
        first = max(0, ctx[s] - q[s] - window + 1) // 16
        bt[s, :first] = -1
    out = torch.empty_like(qs.cuda())
    pkv.attention_int8(out, qs.cuda(), *cache.gpu[:2], wide(bt, bound).cuda(), cl.cuda(),
                       qsl.cuda(), scale, *cache.gpu[2:], max_query_len=64,
                       max_context_len=bound or 1500,
                       num_decode_seqs=3,
                       sliding_window=window)
    assert pkv.get_error() == 0 and torch.isfinite(out.float()).all()


@pytest.mark.parametrize("bound", [None, 200000])
@pytest.mark.parametrize("nd", [-1, 0, 3, 6])
def test_mixed_batches_and_declared_decode_runs(nd, bound):
    q, ctx = [1, 1, 1, 1, 1, 1, 70, 1, 33], [5, 700, 64, 1, 333, 90, 300, 17, 33]
    check_attention(*batch(ctx, q, 16, 4, 128, seed=5), num_decode_seqs=nd, max_context_len=bound)


def test_rows_behind_the_last_sequence_and_empty_sequences_are_left_alone():
    ctx, q = [20, 0, 37, 9, 0], [1, 0, 1, 1, 0]
    cache, qs, bt, cl, qsl, scale = batch([20, 1, 37, 9, 1], [1] * 5, 8, 4, 64, seed=3)
    cl, qsl = i32(ctx), starts(q)
    qs = torch.cat([qs, qs])
    for kw in (dict(max_query_len=1, max_context_len=37),
               dict(max_query_len=1, max_context_len=200000),
               dict(max_query_len=4, num_decode_seqs=0, max_context_len=37)):
        out = torch.full(qs.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        pkv.attention_int8(out, qs.cuda(), *cache.gpu[:2], wide(bt, kw["max_context_len"]).cuda(),
                           cl.cuda(), qsl.cuda(), scale, *cache.gpu[2:], **kw)
        assert (out[3:] == 7.0).all() and (out[:3] != 7.0).any(-1).all()
    assert pkv.get_error() == 0


@pytest.mark.parametrize("chunk,bound", [(1, 200), (1, 200000), (20, 200)])
def test_bad_sequences_are_zero_and_flagged_the_others_right(chunk, bound):
    ctx, q = [100, 50, 200, 64, 90], [chunk] * 5
    b = batch(ctx, q, 8, 4, 64, seed=21)
    cache, qs, bt, cl, qsl, scale = b
    good, ref, tol = attend(*b)
    bt = wide(bt, bound)
    for bad_len, bits in ((0, pkv.ERR_CONTEXT_LEN), (16 * bt.shape[1] + 1, pkv.ERR_CONTEXT_LEN),
                          (-5, pkv.ERR_CONTEXT_LEN)) + (((chunk - 1, pkv.ERR_QUERY_LEN),)
                                                        if chunk > 1 else ()):
        cl2 = cl.clone()
        cl2[2] = bad_len
        for nd in ((-1,) if chunk > 1 else (-1, 0)):
            out = torch.full(qs.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
            # (max_query_len 2 sends single rows through the prefill path)
            mq = chunk if nd < 0 else 2
            pkv.attention_int8(out, qs.cuda(), *cache.gpu[:2], bt.cuda(), cl2.cuda(), qsl.cuda(),
                               scale, *cache.gpu[2:], max_query_len=mq, max_context_len=bound,
                               num_decode_seqs=nd)
            assert pkv.get_error() == bits
            got = out.float().cpu().numpy()
            mine = slice(2 * chunk, 3 * chunk)
            assert (got[mine] == 0).all()
            keep = np.r_[0:2 * chunk, 3 * chunk:5 * chunk]
            assert (np.abs(got - ref) / tol)[keep].max() <= 1
    # a bad block id: the other sequences are right
    bt2 = bt.clone()
    bt2[1, 1] = cache.kc.shape[0]
    bt2[3, 0] = -1
    out = torch.full(qs.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    pkv.attention_int8(out, qs.cuda(), *cache.gpu[:2], bt2.cuda(), cl.cuda(), qsl.cuda(), scale,
                       *cache.gpu[2:], max_query_len=chunk, max_context_len=bound)
    assert pkv.get_error() == pkv.ERR_BLOCK_ID
    got = out.float().cpu().numpy()
    keep = np.r_[0:chunk, 2 * chunk:3 * chunk, 4 * chunk:5 * chunk]
    assert (np.abs(got - ref) / tol)[keep].max() <= 1


@pytest.mark.parametrize("chunk,bound", [(1, None), (1, 200000), (30, None)])
def test_scales_of_very_different_size(chunk, bound):
    """Blocks whose V is 2^-30 of, or 2^20 times, the others', zero scales and
    large and tiny queries: every element to the tolerance of what it sums."""
    b = batch([400, 90, 700], [chunk] * 3, 8, 4, 128, seed=31)
    cache, qs, bt, cl, qsl, scale = b
    rng = np.random.default_rng(1)
    cache.vs *= (2.0 ** rng.integers(-30, 20, cache.vs.shape)).astype(np.float32)
    cache.ks *= (2.0 ** rng.integers(-3, 2, cache.ks.shape)).astype(np.float32)
    cache.vs[bt[0, 3]] = 0.0
    cache.ks[bt[0, 4]] = 0.0
    cache.gpu[2].copy_(torch.from_numpy(cache.ks))
    cache.gpu[3].copy_(torch.from_numpy(cache.vs))
    check_attention(*b, max_context_len=bound)
    check_attention(cache, (qs.float() * 2.0 ** 16).to(torch.bfloat16), bt, cl, qsl,
                    scale * 2.0 ** -16, max_context_len=bound)
    check_attention(cache, (qs.float() * 2.0 ** -40).to(torch.bfloat16), bt, cl, qsl,
                    scale * 2.0 ** 40, max_context_len=bound)
    # a negative and a zero softmax scale
    check_attention(cache, qs, bt, cl, qsl, -scale, max_context_len=bound)
    check_attention(cache, qs, bt, cl, qsl, 0.0, max_context_len=bound)


@pytest.mark.parametrize("chunk,bound", [(1, None), (1, 200000), (30, None), (30, 9000)])
@pytest.mark.parametrize("power", [100, -50])
def test_queries_and_keys_of_opposite_extreme_size(chunk, bound, power):
    """Keys of about 2^power, queries of 2^-power: ordinary scores."""
    ctx, q = [400, 90, 700], [chunk] * 3
    nb = 90
    cache, bt = Cache(nb, 4, 128, seed=1), tables(ctx, nb, 3)
    gen = torch.Generator().manual_seed(5)
    cache.write(rows(gen, sum(ctx), 4, 128, size=2.0 ** power), rows(gen, sum(ctx), 4, 128), bt,
                i32(ctx), starts(ctx), max(ctx))
    qs = rows(gen, sum(q), 8, 128, size=2.0 ** -power)
    check_attention(cache, qs, bt, i32(ctx), starts(q), 128 ** -0.5, max_context_len=bound)
    assert pkv.get_error() == 0


@pytest.mark.parametrize("hq,bound", [(8, 400), (8, 9000), (130, 400)])
def test_chunks_past_the_last_row_are_skipped_and_flagged(hq, bound):
    """A sequence whose rows end behind the batch's is left out whole."""
    cache, qs, bt, cl, qsl, scale = batch([300, 200], [40, 60], hq, 1, 64, seed=hq)
    got, ref, tol = attend(cache, qs, bt, cl, qsl, scale)
    out = torch.full((90, hq, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    pkv.attention_int8(out, qs[:90].cuda(), *cache.gpu[:2], wide(bt, bound).cuda(), cl.cuda(),
                       qsl.cuda(), scale, *cache.gpu[2:], max_query_len=60, max_context_len=bound)
    assert pkv.get_error() == pkv.ERR_QUERY_LEN
    got = out.float().cpu().numpy()
    assert (np.abs(got - ref[:90]) / tol[:90])[:40].max() <= 1 and (got[40:] == 7.0).all()


def test_write_flags_row_starts_that_decrease():
    """Whatever is written then lies in the sequences' own blocks."""
    ctx = [100, 120, 300]
    bt = tables(ctx, 40, 2)
    cache = Cache(40, 2, 64, seed=1)
    gen = torch.Generator().manual_seed(3)
    k, v = rows(gen, 200, 2, 64), rows(gen, 200, 2, 64)
    before = [t.clone() for t in cache.gpu]
    for qsl in ([0, 100, 50, 200], [0, 200, 190, 191], [0, 10, -20, 5], [50, 20, 10, 0]):
        pkv.write_int8(k.cuda(), v.cuda(), bt.cuda(), i32(ctx).cuda(), i32(qsl).cuda(), *cache.gpu,
                       max_query_len=200)
        assert pkv.get_error() & pkv.ERR_QUERY_LEN
    used = set(bt[bt >= 0].tolist())
    rest = [b for b in range(40) if b not in used]
    for a, b in zip(cache.gpu, before):
        assert torch.equal(a[rest].view(torch.uint8), b[rest].view(torch.uint8))


@pytest.mark.parametrize("chunk,bound", [(1, None), (1, 400000), (30, None)])
def test_a_sharp_softmax_on_a_block_of_tiny_values(chunk, bound):
    """All weight on keys of one block whose V is 2^-20 of the others': the
    tiny output keeps its relative precision."""
    b = batch([200], [chunk], 8, 4, 64, seed=41)
    cache, qs, bt, cl, qsl, scale = b
    k, _ = cache.values()
    blk = int(bt[0, 2])
    key = np.repeat(k[blk, 5], 2, 0)      # (each head's own key)
    qs = torch.from_numpy(np.tile(key * 30, (chunk, 1, 1))).to(torch.bfloat16)
    cache.vs[blk] *= np.float32(2.0 ** -20)
    cache.gpu[3].copy_(torch.from_numpy(cache.vs))
    got, ref, _ = attend(cache, qs, bt, cl, qsl, scale, max_context_len=bound)
    own = np.abs(O8.widen(cache.vc, cache.vs)[blk]).max()
    assert np.abs(ref).max() < 1.01 * own       # nothing but that block counts
    assert np.abs(got - ref).max() <= tolerance(np.abs(ref).max(), own)


def test_prefix_shared_blocks():
    ctx = [70, 80, 100]
    b = batch(ctx, [1, 1, 1], 8, 4, 128, seed=51)
    cache, qs, bt, cl, qsl, scale = b
    bt[1, :3] = bt[0, :3]
    bt[2, :3] = bt[0, :3]
    for bound in (None, 200000):
        check_attention(cache, qs, bt, cl, qsl, scale, max_context_len=bound)


def test_offsets_past_32_bits():
    """Blocks whose codes lie more than 2^32 bytes into the cache."""
    hkv, d, nb = 8, 128, 280000
    gpu = [torch.zeros((nb, 16, hkv, d), dtype=torch.int8, device="cuda") for _ in range(2)]
    gpu += [torch.full((nb, hkv), float("nan"), device="cuda") for _ in range(2)]
    gen = torch.Generator().manual_seed(3)
    n, qn = 50, 20
    k, v = rows(gen, n, hkv, d), rows(gen, n, hkv, d)
    far, near = i32([[nb - 1, nb - 4, 270001, 5]]), i32([[0, 3, 1, 2]])
    outs = []
    for bt, cache in ((far, gpu), (near, [t[:4].clone() for t in gpu])):
        pkv.write_int8(k.cuda(), v.cuda(), bt.cuda(), i32([n]).cuda(), i32([0, n]).cuda(), *cache,
                       max_query_len=n)
        for m, bound in ((1, n), (1, 400000), (qn, n)):
            q = rows(torch.Generator().manual_seed(m), m, 16, d).cuda()
            out = torch.empty_like(q)
            pkv.attention_int8(out, q, *cache[:2], wide(bt, bound).cuda(), i32([n]).cuda(),
                               i32([0, m]).cuda(), d ** -0.5, *cache[2:], max_query_len=m,
                               max_context_len=bound)
            outs.append(out)
    assert pkv.get_error() == 0
    assert all(torch.equal(a, b) for a, b in zip(outs[:3], outs[3:]))
    assert all(torch.isfinite(o.float()).all() and o.float().abs().max() > 0 for o in outs)


def test_workspace_refusals_and_extreme_bounds():
    b = batch([900, 40], [1, 1], 8, 4, 64, seed=81)
    cache, qs, bt, cl, qsl, scale = b
    out = torch.zeros_like(qs, device="cuda")
    args = (out, qs.cuda(), *cache.gpu[:2], bt.cuda(), cl.cuda(), qsl.cuda(), scale, *cache.gpu[2:])
    kw = dict(max_query_len=1, max_context_len=900, kv_split_tokens=64)
    meta = pkv.attn_meta(args[1], args[4], args[5], **kw)
    need = pkv.workspace_size_int8(cache.gpu[0], meta)
    assert need > 0
    ws = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
    with pytest.raises(pkv.PkvError, match="-5"):
        pkv.attention_int8(*args, workspace=ws[:need - 1], **kw)
    with pytest.raises(pkv.PkvError, match="-6"):
        pkv.attention_int8(*args, workspace=ws[16:], **kw)
    torch.cuda.synchronize()
    assert not out.any()
    pkv.attention_int8(*args, workspace=ws, **kw)
    assert out.any()
    # bounds at the end of 32 bits are the table's
    for window in (0, 2 ** 31 - 1):
        ref = attend(*b, window=window)
        out = torch.zeros_like(qs, device="cuda")
        for mq, nd in ((1, -1), (2 ** 31 - 1, 0), (2 ** 31 - 1, 1)):
            out.zero_()
            pkv.attention_int8(out, *args[1:], max_query_len=mq, max_context_len=2 ** 31 - 1,
                               num_decode_seqs=nd, sliding_window=window)
            assert (np.abs(out.float().cpu().numpy() - ref[1]) <= ref[2]).all()


def test_same_call_twice_gives_the_same_bits():
    b = batch([3000, 17, 900, 1200], [1, 1, 1, 1], 16, 4, 128, seed=61, step=500)
    for bound in (None, 100000):
        one = attend(*b, max_context_len=bound)[0]
        for _ in range(3):
            assert np.array_equal(one, attend(*b, max_context_len=bound)[0])


@pytest.mark.parametrize("bound", [900, 100000])
def test_other_stream_and_two_graphs(bound):
    """A write and an attention captured on their own streams into two graphs
    with a workspace each, replayed together with new inputs."""
    parts = []
    for seed in (1, 2):
        ctx = [900, 33, 520, 400]
        cache, qs, bt, cl, qsl, scale = batch(ctx, [1, 1, 1, 60], 16, 4, 128, seed=seed)
        gen = torch.Generator().manual_seed(seed + 50)
        k, v = rows(gen, 63, 4, 128), rows(gen, 63, 4, 128)
        bt = wide(bt, bound)
        dev = [t.cuda() for t in (qs, k, v, bt, cl, qsl)]
        out = torch.empty_like(dev[0])
        meta = pkv.attn_meta(dev[0], dev[3], dev[4], max_query_len=60, max_context_len=bound,
                             num_decode_seqs=3)
        ws = torch.empty(max(pkv.workspace_size_int8(cache.gpu[0], meta), 1), dtype=torch.uint8,
                         device="cuda")
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())

        def step(cache=cache, dev=dev, out=out, ws=ws, stream=stream, scale=scale):
            q, k, v, bt, cl, qsl = dev
            pkv.write_int8(k, v, bt, cl, qsl, *cache.gpu, max_query_len=60, stream=stream)
            pkv.attention_int8(out, q, *cache.gpu[:2], bt, cl, qsl, scale, *cache.gpu[2:],
                               max_query_len=60, max_context_len=bound, num_decode_seqs=3,
                               workspace=ws, stream=stream)

        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
        parts.append((graph, stream, cache, dev, out, (qs, k, v, bt, cl, qsl, scale), seed))
    for turn in range(3):
        for graph, stream, cache, dev, out, host, seed in parts:
            gen = torch.Generator().manual_seed(100 * turn + seed)
            dev[1].copy_(rows(gen, 63, 4, 128))
            dev[2].copy_(rows(gen, 63, 4, 128))
            dev[0].copy_(rows(gen, 63, 16, 128))
            out.fill_(float("nan"))
        torch.cuda.synchronize()
        for graph, stream, *_ in parts:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for graph, stream, cache, dev, out, host, seed in parts:
            q, k, v, bt, cl, qsl = (t.cpu() for t in dev)
            if turn == 0:   # the two eager and captured writes of the first rows
                O8.write(host[1].float().numpy(), host[2].float().numpy(), bt.numpy(), cl.numpy(),
                         qsl.numpy(), cache.kc, cache.vc, cache.ks, cache.vs)
            O8.write(k.float().numpy(), v.float().numpy(), bt.numpy(), cl.numpy(), qsl.numpy(),
                     cache.kc, cache.vc, cache.ks, cache.vs)
            cache.check()
            ref, st = oracle.attention(q.float().numpy(), *cache.values(), bt.numpy(), cl.numpy(),
                                       qsl.numpy(), host[6])
            tol = tolerance(ref, np.nanmax(np.abs(cache.values()[1])))
            assert (np.abs(out.float().cpu().numpy() - ref) <= tol).all()
    assert pkv.get_error() == 0
