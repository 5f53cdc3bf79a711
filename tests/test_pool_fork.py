"""Forking, copy on write, resizing (compaction) and freeing in the C++ pool:
against the oracle on random traces, and against a shadow of the blocks'
contents that follows the noted copies.  Host only, no GPU."""
import random

import numpy as np
import pytest

from oracle import pool as O
from paged_kv_cache_43_gb300 import build, pkv
from paged_kv_cache_43_gb300 import pool as N
from tests.test_pool_native import _same_state


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()


class Shadow:
    """What the caches would hold: a (tokens so far) value in every slot."""

    def __init__(self, nb):
        self.slot = {}
        self.nb = nb

    def copy(self, pairs):
        for a, b in pairs:
            for o in range(16):
                self.slot[b * 16 + o] = self.slot.get(a * 16 + o)

    def write(self, req, slots, first):
        for i, s in enumerate(slots):
            self.slot[s] = tuple(req.tokens[:first + i + 1])

    def check(self, req, null):
        for p in range(req.num_computed):
            b = req.blocks[p // 16]
            if b != null:
                assert self.slot[b * 16 + p % 16] == tuple(req.tokens[:p + 1]), p


@pytest.mark.parametrize("seed,nb,caching,window", [
    (1, 60, True, 0), (2, 25, True, 0), (3, 25, False, 0), (4, 60, True, 20), (5, 18, True, 33),
    (6, 200, True, 0), (7, 12, True, 0)])
def test_random_traces_against_the_oracle(seed, nb, caching, window):
    rng = random.Random(seed)
    o, n = O.Pool(nb, caching=caching), N.BlockPool(nb, caching=caching)
    shadow = Shadow(nb)
    base = [rng.randrange(9) for _ in range(40)]
    live, next_id, forks, moves, cows = [], 0, 0, 0, 0

    def grow(rid):
        todo = len(o.reqs[rid].tokens) - o.num_computed(rid)
        if todo <= 0:
            t = rng.randrange(9)
            o.append_token(rid, t)
            n.append_token(rid, t)
            todo = 1
        first = o.num_computed(rid)
        so, sn = o.allocate_slots(rid, todo, window), n.allocate_slots(rid, todo, window)
        assert (so is None) == (sn is None)
        if so is None:
            return False
        assert list(sn) == so
        co = o.take_copies()
        assert [tuple(x) for x in n.take_copies()] == co
        shadow.copy(co)
        shadow.write(o.reqs[rid], so, first)
        return len(co)

    for step in range(500):
        op = rng.random()
        if op < 0.15 or not live:
            rid, next_id = next_id, next_id + 1
            toks = base[:rng.randrange(41)] + [rng.randrange(9) for _ in range(rng.randrange(1, 30))]
            o.add_request(rid, toks)
            n.add_request(rid, toks)
            assert n.admit(rid) == o.admit(rid)
            live.append(rid)
            if grow(rid) is False:
                live.remove(rid)
                o.free_request(rid)
                n.free_request(rid)
        elif op < 0.3:
            rid, next_id = next_id, next_id + 1
            parent = rng.choice(live)
            o.fork_request(parent, rid)
            n.fork_request(parent, rid)
            live.append(rid)
            forks += 1
        elif op < 0.75:
            rid = rng.choice(live)
            got = grow(rid)
            if got is False:
                live.remove(rid)
                o.free_request(rid)
                n.free_request(rid)
            else:
                cows += got
        elif op < 0.85:
            size = max(2, nb + rng.randrange(-nb // 2, nb // 2 + 1))
            done = o.resize(size)
            assert n.resize(size) == done
            if done:
                nb = size
            pairs = o.take_copies()
            assert [tuple(x) for x in n.take_copies()] == pairs
            shadow.copy(pairs)
            moves += len(pairs)
        else:
            rid = live.pop(rng.randrange(len(live)))
            o.free_request(rid)
            n.free_request(rid)
        _same_state(o, n, live, nb)
        for rid in live:
            shadow.check(o.reqs[rid], o.null_block)
    assert forks > 20 and cows > 5 and moves > 0


def test_copies_wait_until_they_are_taken_and_keep_their_order():
    """Copies noted over many steps, taken in parts: the contents still follow."""
    o, n = O.Pool(4000), N.BlockPool(4000)
    n.add_request(0, list(range(20)))
    n.allocate_slots(0, 20)
    for i in range(1, 700):
        n.fork_request(0, i)
        n.append_token(i, i)
        assert n.allocate_slots(i, 1) is not None
    first = n.block_table(0)[1]
    got = n.take_copies()
    assert got.shape == (699, 2) and (got[:, 0] == first).all()
    assert len(set(got[:, 1].tolist())) == 699
    assert n.take_copies().shape == (0, 2)
    assert n.resize(1000) and n.take_copies().shape == (0, 2)   # ids are low already


def test_the_last_holder_keeps_the_block():
    n = N.BlockPool(10)
    n.add_request(0, [1, 2, 3])
    n.allocate_slots(0, 3)
    block = n.block_table(0)[0]
    n.fork_request(0, 1)
    n.append_token(1, 4)
    n.append_token(0, 5)
    assert n.allocate_slots(1, 1)[0] // 16 != block
    assert n.allocate_slots(0, 1)[0] // 16 == block
    assert n.take_copies().tolist() == [[block, n.block_table(1)[0]]]
    # freed parents leave the child's blocks alone
    n.fork_request(1, 2)
    n.free_request(1)
    n.append_token(2, 6)
    assert n.allocate_slots(2, 1) is not None and n.take_copies().size == 0


def test_a_fork_on_a_block_border_needs_no_copy():
    n = N.BlockPool(10)
    n.add_request(0, list(range(32)))
    n.allocate_slots(0, 32)
    n.fork_request(0, 1)
    n.append_token(1, 7)
    assert n.allocate_slots(1, 1) is not None
    assert n.take_copies().size == 0 and n.block_table(1)[:2] == n.block_table(0)


def test_no_space_for_the_copy_changes_nothing():
    n = N.BlockPool(3, caching=False)       # the null block and two others
    n.add_request(0, list(range(20)))
    n.allocate_slots(0, 20)
    n.fork_request(0, 1)
    n.append_token(1, 7)
    assert n.allocate_slots(1, 1) is None
    assert n.take_copies().size == 0 and n.block_table(1) == n.block_table(0)
    assert n.num_computed(1) == 20 and not n.resize(2)


def test_refusals():
    n = N.BlockPool(4)
    n.add_request(0, [1])
    for bad in ((5, 6), (0, 0)):            # unknown parent, known child
        with pytest.raises(pkv.PkvError):
            n.fork_request(*bad)
    for bad in (0, -3):
        with pytest.raises(pkv.PkvError):
            n.resize(bad)
    lib = n._lib
    assert lib.pkv_pool_fork_request(None, 0, 1) < 0 and lib.pkv_pool_resize(None, 3) < 0
    assert lib.pkv_pool_take_copies(n._p, None, 1, None) < 0


def test_growing_hands_out_the_new_blocks_first():
    n = N.BlockPool(2)
    assert n.resize(5)
    n.add_request(0, list(range(48)))
    n.allocate_slots(0, 48)
    assert n.block_table(0) == [2, 3, 4] and n.free_queue() == [1]
    assert np.array_equal(n.block_tables([0], 4), [[2, 3, 4, -1]])
