"""The int8 cache, page copies, forks and resizes together, as a serving loop
uses them: DecodeLoop over a small pool with prefix hits, chunked prefill,
preemption, forked requests and caches that change their size.  Every step's
codes and scales are compared bit for bit with the oracle's (which makes the
same block copies and writes), every output with its fp64 attention."""
import numpy as np
import pytest
import torch

import oracle
from oracle import int8 as O8
from paged_kv_cache_43_gb300 import build, pkv
from paged_kv_cache_43_gb300 import workloads as W
from paged_kv_cache_43_gb300.decode_loop import DecodeLoop
from tests.test_gpu_int8 import tolerance

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


def host(t):
    return t.cpu().numpy().copy()


def run(loop, events, limit=400):
    """Steps until done; events {step: callable}.  Returns outputs by
    (request, position), preemptions and copied blocks."""
    caches = [host(t) for t in loop.buffers()]
    rows, preempted, copied, steps = {}, 0, 0, 0
    while not loop.done():
        if steps in events:
            before = loop.k_cache.shape[0]
            events[steps](loop)
            torch.cuda.synchronize()
            if loop.k_cache.shape[0] != before:
                # (a resize makes its copies itself: start from what it left)
                caches = [host(t) for t in loop.buffers()]
        st = loop.step()
        assert st is not None
        steps += 1
        assert steps < limit
        preempted += len(st.preempted)
        copied += len(st.copies)
        torch.cuda.synchronize()
        assert pkv.get_error() == 0
        for a, b in st.copies:
            for c in caches:
                c[b] = c[a]
        bt, cl, qsl = host(st.block_tables), host(st.context_lens), host(st.query_start_loc)
        O8.write(host(st.k_new.float()), host(st.v_new.float()), bt, cl, qsl, *caches)
        for got, want in zip(loop.buffers(), caches):
            assert host(got).tobytes() == want.tobytes()
        k, v = O8.widen(caches[0], caches[2]), O8.widen(caches[1], caches[3])
        ref, status = oracle.attention(host(st.q.float()), k, v, bt, cl, qsl, loop.scale,
                                       window=loop.window)
        assert not status.any()
        out = host(st.out.float()).astype(np.float64)
        assert (np.abs(out - ref) <= tolerance(ref, np.nanmax(np.abs(v)))).all()
        for i, rid in enumerate(st.req_ids):
            for j, p in enumerate(st.positions[i]):
                rows[(rid, p)] = out[qsl[i] + j]
    return rows, preempted, copied


def loop_of(num_blocks, window=0, caching=True, d=128, seed=3, requests=8):
    rng = np.random.default_rng(seed)
    loop = DecodeLoop(num_blocks=num_blocks, num_q_heads=8, num_kv_heads=2, head_size=d,
                      caching=caching, window=window, max_batch_tokens=160, seed=seed,
                      dtype=torch.int8)
    system = [int(x) for x in rng.integers(0, 512, 40)]
    for i in range(requests):
        tail = [int(x) for x in rng.integers(0, 512, int(rng.integers(3, 30)))]
        loop.add_request(system + tail, max_new_tokens=int(rng.integers(12, 25)))
    return loop


def test_forks_and_resizes_match_the_oracle_every_step():
    ids = []

    def fork(lp):
        for r in list(lp.running)[:3]:
            ids.append((r.rid, len(r.tokens), lp.fork_request(r.rid)))

    events = {3: fork, 7: fork, 9: lambda lp: lp.resize(40) or lp.resize(80),
              12: lambda lp: lp.resize(150), 14: lambda lp: lp.resize(60)}
    rows, _, copied = run(loop_of(96), events)
    assert len(ids) == 6 and copied >= 3
    for parent, n, child in ids:            # a child goes on by itself
        assert any((child, p) in rows for p in range(n, n + 5))


def test_a_small_pool_preempts_forked_requests():
    def fork(lp):
        for r in list(lp.running)[:2]:
            lp.fork_request(r.rid)

    _, preempted, _ = run(loop_of(16), {4: fork, 8: fork})
    assert preempted > 0


@pytest.mark.parametrize("window", [16, 33])
def test_sliding_window(window):
    def fork(lp):
        lp.fork_request(lp.running[0].rid)

    run(loop_of(64, window=window, caching=False, d=64), {3: fork})


def test_int8_outputs_are_near_the_bf16_loop():
    """The same requests over a bf16 cache: quantisation alone between them.
    An int8 element is off by at most half a step, amax / 254 (a whole one where
    a later token made the block round again), so K and V of size ~1 move an
    output by a few hundredths at most."""
    rows, _, _ = run(loop_of(96), {})
    loop = loop_of(96)
    ref = DecodeLoop(num_blocks=96, num_q_heads=8, num_kv_heads=2, head_size=128, seed=3,
                     max_batch_tokens=160)
    for r in loop.waiting:
        ref.add_request(r.tokens, r.max_new)
    worst = 0.0
    while not ref.done():
        st = ref.step()
        qsl = host(st.query_start_loc)
        out = host(st.out.float())
        for i, rid in enumerate(st.req_ids):
            for j, p in enumerate(st.positions[i]):
                worst = max(worst, float(np.abs(out[qsl[i] + j] - rows[(rid, p)]).max()))
    assert worst < 0.1


def test_bf16_loop_forks_and_resizes():
    """The page copies under the bf16 cache: every step against the oracle."""
    rng = np.random.default_rng(9)
    loop = DecodeLoop(num_blocks=60, num_q_heads=4, num_kv_heads=2, head_size=64, seed=9,
                      max_batch_tokens=160)
    for _ in range(4):
        loop.add_request([int(x) for x in rng.integers(0, 512, 37)], 14)
    A = W.as_oracle_array
    steps, copied = 0, 0
    while not loop.done():
        if steps == 3:
            for r in list(loop.running):
                loop.fork_request(r.rid)
        if steps == 6:
            assert loop.resize(40) and loop.resize(50)
        kc, vc = A(loop.k_cache).copy(), A(loop.v_cache).copy()
        st = loop.step()
        steps += 1
        for a, b in st.copies:
            kc[b], vc[b] = kc[a], vc[a]
        copied += len(st.copies)
        assert oracle.write(A(st.k_new), A(st.v_new), A(st.slot_mapping), kc, vc) == 0
        assert A(loop.k_cache).tobytes() == kc.tobytes()
        exp, status = oracle.attention(A(st.q), kc, vc, A(st.block_tables), A(st.context_lens),
                                       A(st.query_start_loc), loop.scale)
        assert not status.any()
        assert np.abs(st.out.float().cpu().numpy() - exp).max() <= 2e-2
    assert copied >= 4
