"""pkv_pool_take_back: drafted positions that were not accepted go back to the pool.  Against the
oracle on random traces of drafted steps, with a shadow of what every slot holds.  Host only."""
import ctypes
import random

import pytest

from oracle import pool as O
from paged_kv_cache_43_gb300 import build, pkv
from paged_kv_cache_43_gb300 import pool as N
from tests.test_pool_native import _same_state


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()


def test_the_next_slots_follow_the_kept_ones():
    p = N.BlockPool(12, caching=False)
    p.add_request(0, range(14))
    assert list(p.allocate_slots(0, 14)) == [16 + i for i in range(14)]
    assert list(p.allocate_slots(0, 40))[:3] == [30, 31, 32]      # drafts over blocks 1 .. 4
    assert p.num_free() == 7
    p.take_back([0], [16 + 5])
    assert p.num_computed(0) == 21 and p.block_table(0) == [1, 2] and p.num_free() == 9
    assert p.free_queue()[:2] == [3, 4]
    assert list(p.allocate_slots(0, 2)) == [2 * 16 + 5, 2 * 16 + 6]
    p.take_back([0], [21])                                        # none of them accepted
    p.take_back([0], [21])                                        # (and again: nothing to do)
    assert list(p.allocate_slots(0, 12))[-2:] == [2 * 16 + 15, 3 * 16]
    p.take_back([0], [32])                                        # a block's end: the next block goes
    assert p.block_table(0) == [1, 2]


def test_refusals_change_nothing():
    p = N.BlockPool(12)
    p.add_request(0, range(20))
    p.allocate_slots(0, 20)
    p.allocate_slots(0, 9)
    state = lambda: (p.num_computed(0), p.block_table(0), p.free_queue())
    before = state()
    for ids, n in (([0], [19]), ([0], [30]), ([0], [-1]), ([7], [20])):
        with pytest.raises(pkv.PkvError):
            p.take_back(ids, n)
        assert state() == before
    with pytest.raises(pkv.PkvError):
        p.take_back([0], [20, 20])
    lib = N._lib()
    one, req = ctypes.c_int32(20), ctypes.c_int64(0)
    assert lib.pkv_pool_take_back(None, ctypes.byref(req), ctypes.byref(one), 1) == -1
    assert lib.pkv_pool_take_back(p._p, None, ctypes.byref(one), 1) == -1
    assert lib.pkv_pool_take_back(p._p, ctypes.byref(req), ctypes.byref(one), -1) == -3
    assert lib.pkv_pool_take_back(p._p, None, None, 0) == 0
    p.take_back([], [])
    assert state() == before
    # tokens of drafts that were appended too early are in the prefix cache
    p.append_tokens(0, range(20))
    p.allocate_slots(0, 9)
    with pytest.raises(pkv.PkvError):
        p.take_back([0], [31])
    p.take_back([0], [32])
    assert p.num_computed(0) == 32


def test_it_stops_at_the_first_that_it_cannot_serve():
    p = N.BlockPool(30)
    for i in range(3):
        p.add_request(i, range(5))
        p.allocate_slots(i, 5)
        p.allocate_slots(i, 6)
    with pytest.raises(pkv.PkvError):
        p.take_back([0, 9, 2], [7, 7, 7])
    assert [p.num_computed(i) for i in range(3)] == [7, 11, 11]


def test_a_fork_keeps_what_the_parent_takes_back():
    p = N.BlockPool(20, caching=False)
    p.add_request(0, range(10))
    p.allocate_slots(0, 10)
    p.allocate_slots(0, 25)                # blocks 1, 2, 3
    p.fork_request(0, 1)
    p.take_back([0], [12])
    assert p.block_table(1) == [1, 2, 3] and p.block_state(2)[0] == 1
    assert list(p.allocate_slots(0, 1)) == [4 * 16 + 12]          # block 1 is the fork's, too: a copy
    assert p.take_copies().tolist() == [[1, 4]]
    p.take_back([1], [20])                 # (the fork's last allocation is its parent's)
    assert p.block_table(1) == [1, 2]


@pytest.mark.parametrize("seed,nb,caching,window", [(1, 60, True, 0), (2, 30, True, 0), (3, 40, False, 0),
                                                    (4, 60, True, 24), (5, 25, True, 40), (6, 18, True, 0)])
def test_random_drafted_steps_against_the_oracle(seed, nb, caching, window):
    """Requests that come (some with a common prefix), draft, keep a part and go; every slot
    of a kept position holds that position's token, whatever the others did in between."""
    rng = random.Random(seed)
    o, n = O.Pool(nb, caching=caching), N.BlockPool(nb, caching=caching)
    holds, live, next_id, kept_back, hits = {}, [], 0, 0, 0
    base = [rng.randrange(5) for _ in range(60)]

    def write(rid, slots, first, tokens):
        for i, s in enumerate(slots):
            holds[s] = tuple(tokens[:first + i + 1])

    def copies():
        pairs = o.take_copies()
        assert [tuple(x) for x in n.take_copies()] == pairs
        for a, b in pairs:
            for i in range(16):
                holds[b * 16 + i] = holds.get(a * 16 + i)

    for _ in range(600):
        if rng.random() < 0.1 or not live:
            rid, next_id = next_id, next_id + 1
            toks = base[:rng.randrange(61)] + [rng.randrange(5) for _ in range(rng.randrange(1, 20))]
            for p in (o, n):
                p.add_request(rid, toks)
            first = n.admit(rid)
            assert first == o.admit(rid)
            hits += first > 0
            so, sn = o.allocate_slots(rid, len(toks) - first, window), n.allocate_slots(rid, len(toks) - first, window)
            assert (so is None) == (sn is None)
            if so is None:
                o.free_request(rid)
                n.free_request(rid)
                continue
            assert list(sn) == so
            copies()
            write(rid, so, first, toks)
            live.append(rid)
            for p in (o, n):
                p.append_token(rid, 7)               # the first sampled token: the next step's root
        elif rng.random() < 0.08:
            rid = live.pop(rng.randrange(len(live)))
            o.free_request(rid)
            n.free_request(rid)
        elif rng.random() < 0.05:
            rid, next_id = next_id, next_id + 1
            src = rng.choice(live)
            o.fork_request(src, rid)
            n.fork_request(src, rid)
            live.append(rid)
        else:                                        # a drafted step: the root and some drafts
            rid = rng.choice(live)
            k = rng.randrange(1, 40)
            first = o.num_computed(rid)
            known = list(o.reqs[rid].tokens)
            assert len(known) == first + 1
            so, sn = o.allocate_slots(rid, k, window), n.allocate_slots(rid, k, window)
            assert (so is None) == (sn is None)
            if so is None:
                victim = live.pop(rng.randrange(len(live)))
                o.free_request(victim)
                n.free_request(victim)
                continue
            assert list(sn) == so
            copies()
            for i, s in enumerate(so):
                holds[s] = ("draft", i)
            take = rng.randrange(1, k + 1)
            accepted = [known[-1]] + [rng.randrange(5) for _ in range(take - 1)]
            write(rid, so[:take], first, known[:-1] + accepted)      # (the accepted rows, moved)
            o.take_back(rid, first + take)
            n.take_back([rid], [first + take])
            kept_back += k - take
            for t in accepted[1:] + [7]:
                for p in (o, n):
                    p.append_token(rid, t)
        _same_state(o, n, live, nb)
        for rid in live:
            r = o.reqs[rid]
            for pos in range(r.num_computed):
                b = r.blocks[pos // 16]
                if b != o.null_block:
                    assert holds[b * 16 + pos % 16] == tuple(r.tokens[:pos + 1]), (rid, pos)
    assert kept_back > 500 and (not caching or hits > 0)
