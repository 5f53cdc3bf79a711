"""Int8 decode by the kernel that a batch takes, told from the workspace it asks
for: an all-decode batch of contexts up to 16384 keys takes clusters of its rows'
splits (no workspace) if the GPU holds them all at a time, or, where the blocks by
max_context_len are enough for every team, the team kernel (partials in a
workspace).  Windows, NaN, graph captures and waits that run out reach both."""
import numpy as np
import pytest
import torch

import oracle
from oracle import int8 as O8
from paged_kv_cache_43_gb300 import pkv
from tests.test_gpu_int8 import _lib, Cache, attend, batch, check_attention, i32, rows, starts, \
    tables, tolerance, wide  # noqa: F401

pytestmark = pytest.mark.gpu

TEAMS = 200000   # a bound at which 2 sequences of 4 kv heads are the team kernel's


def workspace(b, window=0, bound=None):
    cache, qs, bt, cl, qsl, _ = b
    meta = pkv.attn_meta(qs, wide(bt, bound), cl, max_query_len=1,
                         max_context_len=bound or int(cl.max()), sliding_window=window)
    return pkv.workspace_size_int8(cache.gpu[0], meta)


def ready(ctx, hq, hkv, d, seed):
    """A decode batch over a cache of random codes and scales."""
    nb = sum(-(-c // 16) for c in ctx) + 1
    cache = Cache(nb, hkv, d, seed=seed)
    rng = np.random.default_rng(seed)
    for i, s in enumerate((cache.ks, cache.vs)):
        s[:] = np.exp(0.3 * rng.standard_normal(s.shape)) * (0.02, 0.015)[i]
        cache.gpu[2 + i].copy_(torch.from_numpy(s))
    gen = torch.Generator().manual_seed(seed)
    return (cache, rows(gen, len(ctx), hq, d), tables(ctx, nb, seed), i32(ctx),
            starts([1] * len(ctx)), d ** -0.5)


# ---------------------------------------------------------------- windows

@pytest.mark.parametrize("seqs,hi,window,hq,hkv,d,bound", [
    (40, 9000, 4096, 16, 8, 64, 16384), (80, 6000, 4097, 8, 4, 128, 16384),
    (1300, 250, 100, 16, 8, 64, 4000), (5000, 60, 17, 8, 8, 64, 4000),
    (10000, 40, 1, 8, 8, 64, 4000)])
def test_window_on_the_team_kernel(seqs, hi, window, hq, hkv, d, bound):
    """Contexts below, at and above the window; blocks wholly before it are never
    looked at."""
    rng = np.random.default_rng(seqs)
    ctx = rng.integers(1, hi + 1, seqs)
    ctx[:6] = [1, min(window, hi), min(window + 1, hi), min(window + 15, hi), min(window + 16, hi), hi]
    b = ready(ctx.tolist(), hq, hkv, d, seed=seqs)
    assert workspace(b, window, bound) > 0
    check_attention(*b, window=window, max_context_len=bound)
    cache, qs, bt, cl, qsl, scale = b
    for s, c in enumerate(ctx):
        bt[s, :max(0, c - window) // 16] = -1
    out = torch.full(qs.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    pkv.attention_int8(out, qs.cuda(), *cache.gpu[:2], wide(bt, bound).cuda(), cl.cuda(),
                       qsl.cuda(), scale, *cache.gpu[2:], max_query_len=1, max_context_len=bound,
                       sliding_window=window)
    assert pkv.get_error() == 0
    again = torch.full(qs.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    pkv.attention_int8(again, qs.cuda(), *cache.gpu[:2], wide(b[2].clamp_min(0), bound).cuda(),
                       cl.cuda(), qsl.cuda(), scale, *cache.gpu[2:], max_query_len=1,
                       max_context_len=bound, sliding_window=window)
    assert torch.equal(out, again) and torch.isfinite(out).all()


def test_no_window_on_the_team_kernel_of_many_ragged_sequences():
    rng = np.random.default_rng(3)
    ctx = np.exp(rng.uniform(0, np.log(6000), 300)).astype(int)
    for hq, hkv, d in ((8, 8, 64), (32, 4, 128)):
        b = ready(ctx.tolist(), hq, hkv, d, seed=hq)
        assert workspace(b, bound=6000) > 0
        check_attention(*b, max_context_len=6000)


@pytest.mark.parametrize("seqs,lo,hi,hq,hkv,clusters", [
    (16, 8000, 16000, 10, 5, False), (7, 8000, 16000, 10, 5, True), (32, 1000, 3000, 32, 8, False),
    (8, 1000, 3000, 32, 8, True), (8, 1000, 3000, 130, 1, True)])
@pytest.mark.parametrize("d", [64, 128])
def test_clusters_only_where_the_gpu_holds_them_all(seqs, lo, hi, hq, hkv, clusters, d):
    """Middle batches with splits that would not all be resident as clusters merge
    through a workspace."""
    ctx = np.random.default_rng(seqs).integers(lo, hi + 1, seqs).tolist()
    b = ready(ctx, hq, hkv, d, seed=seqs)
    assert (workspace(b) == 0) == clusters
    check_attention(*b)
    check_attention(*b, window=700)


# -------------------------------------------------------------------- NaN

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bound", [None, TEAMS])
def test_nan_queries_and_scales_reach_their_rows_only(d, bound):
    b = batch([1200, 90], [1, 1], 8, 4, d, seed=71)
    assert (workspace(b, bound=bound) > 0) == (bound == TEAMS)
    cache, qs, bt, cl, qsl, scale = b
    good, ref, tol = attend(*b, max_context_len=bound)
    assert (np.abs(good - ref) <= tol).all()

    def call(q):
        out = torch.zeros(qs.shape, dtype=torch.bfloat16, device="cuda")
        pkv.attention_int8(out, q.cuda(), *cache.gpu[:2], wide(bt, bound).cuda(), cl.cuda(),
                           qsl.cuda(), scale, *cache.gpu[2:], max_query_len=1,
                           max_context_len=bound or 1200)
        assert pkv.get_error() == 0
        return out.float().cpu().numpy()

    bad = qs.clone()
    bad[0, 3, 5] = float("nan")
    got = call(bad)
    assert np.isnan(got[0, 3]).all()
    got[0, 3] = good[0, 3]
    assert np.array_equal(got, good)
    for scales in cache.gpu[2:]:
        for s, blk in ((0, 0), (0, 40), (0, 74), (1, 0), (1, 5)):   # (first, middle, last)
            at = int(bt[s, blk])
            was = float(scales[at, 2])
            scales[at, 2] = float("nan")
            got = call(qs)
            scales[at, 2] = was
            assert np.isnan(got[s, 4:6]).all(), (s, blk)
            got[s, 4:6] = good[s, 4:6]
            assert np.array_equal(got, good)
    # a window that begins behind the block: nothing of it is seen
    at = int(bt[0, 40])
    cache.gpu[2][at] = float("nan")
    cache.gpu[3][at] = float("nan")
    out = torch.zeros(qs.shape, dtype=torch.bfloat16, device="cuda")
    pkv.attention_int8(out, qs.cuda(), *cache.gpu[:2], wide(bt, bound).cuda(), cl.cuda(), qsl.cuda(),
                       scale, *cache.gpu[2:], max_query_len=1, max_context_len=bound or 1200,
                       sliding_window=500)
    assert torch.isfinite(out).all()


# ---------------------------------------------------------- graph captures

@pytest.mark.parametrize("ctx,bound", [([900, 33, 520, 400], None), ([4100, 33, 2000, 400], None),
                                       ([900, 33, 520, 400], 100000)])
def test_decode_steps_in_two_graphs(ctx, bound):
    """A write and an all-decode attention (a cluster launch of 2 to 8 splits, of
    9 to 16, the team kernel and its merge) captured on their own streams into two
    graphs, replayed together with new rows and contexts that grow by a token."""
    parts = []
    for seed in (1, 2):
        b = batch(ctx, [1] * 4, 16, 4, 128, seed=seed, pad=1, step=3000)
        cache, qs, bt, cl, qsl, scale = b
        need = workspace(b, bound=bound or max(ctx) + 4)
        assert (need > 0) == (bound is not None)
        spare = iter(sorted(set(range(cache.kc.shape[0])) - set(bt.flatten().tolist())))
        for s in range(4):                        # (room for the tokens to come)
            at = (int(cl[s]) + 2) // 16
            if bt[s, at] < 0:
                bt[s, at] = next(spare)
        bt = wide(bt, bound)
        gen = torch.Generator().manual_seed(seed + 50)
        dev = [t.cuda() for t in (qs, rows(gen, 4, 4, 128), rows(gen, 4, 4, 128), bt, cl, qsl)]
        out = torch.empty_like(dev[0])
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())

        def step(cache=cache, dev=dev, out=out, ws=ws, stream=stream, scale=scale):
            q, k, v, bt, cl, qsl = dev
            pkv.write_int8(k, v, bt, cl, qsl, *cache.gpu, max_query_len=1, stream=stream)
            pkv.attention_int8(out, q, *cache.gpu[:2], bt, cl, qsl, scale, *cache.gpu[2:],
                               max_query_len=1, max_context_len=bound or max(ctx) + 4,
                               workspace=ws, stream=stream)

        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            step()
        parts.append((graph, stream, cache, dev, out, scale, seed))
    for turn in range(4):
        for graph, stream, cache, dev, out, scale, seed in parts:
            gen = torch.Generator().manual_seed(100 * turn + seed)
            dev[0].copy_(rows(gen, 4, 16, 128))
            dev[1].copy_(rows(gen, 4, 4, 128, size=1.0 + turn))
            dev[2].copy_(rows(gen, 4, 4, 128, size=1.0 + turn))
            dev[4] += turn > 0
            out.fill_(float("nan"))
        torch.cuda.synchronize()
        for graph, stream, *_ in parts:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for graph, stream, cache, dev, out, scale, seed in parts:
            q, k, v, bt, cl, qsl = (t.cpu() for t in dev)
            O8.write(k.float().numpy(), v.float().numpy(), bt.numpy(), cl.numpy(), qsl.numpy(),
                     cache.kc, cache.vc, cache.ks, cache.vs)
            cache.check()
            ref, st = oracle.attention(q.float().numpy(), *cache.values(), bt.numpy(), cl.numpy(),
                                       qsl.numpy(), scale)
            assert not st.any()
            tol = tolerance(ref, np.nanmax(np.abs(cache.values()[1])))
            assert (np.abs(out.float().cpu().numpy() - ref) <= tol).all()
    assert pkv.get_error() == 0


# ------------------------------------------------------- waits that run out

@pytest.mark.parametrize("ctx", [[900, 33, 520, 400], [4100, 33, 2000, 400], [16000]])
@pytest.mark.parametrize("hq,hkv,d", [(16, 4, 128), (8, 8, 64)])
def test_waits_of_a_cluster_run_out_then_the_device_recovers(ctx, hq, hkv, d):
    """Clusters of 2 to 8 splits and of 9 to 16: CTAs whose wait gave up still
    meet the others at the cluster's barriers, and the launch ends."""
    b = ready(ctx, hq, hkv, d, seed=len(ctx))
    assert workspace(b) == 0
    cache, qs, bt, cl, qsl, scale = b
    pkv.debug_wait_test(True)
    try:
        for _ in range(2):
            out = torch.zeros_like(qs, device="cuda")
            pkv.attention_int8(out, qs.cuda(), *cache.gpu[:2], bt.cuda(), cl.cuda(), qsl.cuda(),
                               scale, *cache.gpu[2:], max_query_len=1, max_context_len=max(ctx))
            torch.cuda.synchronize()
            assert pkv.get_error(clear=True) & pkv.ERR_TIMEOUT
    finally:
        pkv.debug_wait_test(False)
    for _ in range(2):
        check_attention(*b)
        assert pkv.get_error(clear=True) == 0
