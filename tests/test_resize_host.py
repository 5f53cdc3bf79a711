"""DecodeLoop.resize on CPU, the kernel calls replaced by stand-ins: a resize
whose new caches cannot be had changes nothing, and the page copies of one that
shrinks carry every request's rows along."""
import numpy as np
import pytest
import torch

from paged_kv_cache_43_gb300 import build
from paged_kv_cache_43_gb300 import decode_loop as DL


@pytest.fixture(autouse=True)
def _host_kernels(monkeypatch):
    """Writes and copies done on the host; attention left out."""
    build.build()
    made = []

    def write(k, v, slots, kc, vc, stream=None):
        for x, cache in ((k, kc), (v, vc)):
            cache.view(-1, *cache.shape[2:])[slots] = x

    def copy_blocks(buffers, pairs, stream=None):
        made.extend((int(a), int(b)) for a, b in pairs)
        for t in buffers:
            for a, b in pairs:
                t[b] = t[a].clone()

    monkeypatch.setattr(DL.pkv, "write", write)
    monkeypatch.setattr(DL.pkv, "copy_blocks", copy_blocks)
    monkeypatch.setattr(DL.pkv, "attention", lambda out, *a, **kw: out.zero_())
    return made


def loop_of(num_blocks, lengths, seed=1):
    rng = np.random.default_rng(seed)
    loop = DL.DecodeLoop(num_blocks=num_blocks, num_q_heads=2, num_kv_heads=1, head_size=64,
                         max_batch_tokens=400, device="cpu", seed=seed)
    for prompt, new in lengths:
        loop.add_request([int(x) for x in rng.integers(0, 512, prompt)], new)
    return loop


def check_rows(loop):
    """Every computed position of every running request holds its own K and V."""
    for r in loop.running:
        n = loop.pool.num_computed(r.rid)
        bt = loop.pool.block_table(r.rid)
        p = np.arange(n)
        at = torch.from_numpy(np.asarray(bt)[p // 16].astype(np.int64))
        assert int(at.max()) < loop.k_cache.shape[0]
        _, k, v = loop.rows(r.tokens[:n], p)
        off = torch.from_numpy(p % 16)
        assert torch.equal(loop.k_cache[at, off], k) and torch.equal(loop.v_cache[at, off], v)


@pytest.mark.parametrize("size", [12, 60])
def test_a_resize_without_memory_changes_nothing(size, monkeypatch):
    loop = loop_of(30, [(40, 20), (35, 20)])
    for _ in range(3):
        loop.step()
    free, state = loop.pool.num_free(), [t.clone() for t in loop.buffers()]
    monkeypatch.setattr(loop, "_new_caches", lambda n: (_ for _ in ()).throw(MemoryError("no room")))
    with pytest.raises(MemoryError):
        loop.resize(size)
    monkeypatch.undo()
    assert loop.pool.num_free() == free and loop.k_cache.shape[0] == 30
    assert len(loop.pool.take_copies()) == 0
    for a, b in zip(loop.buffers(), state):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_a_resize_without_memory_then_steps(monkeypatch, _host_kernels):
    """The loop goes on in the blocks it has."""
    loop = loop_of(30, [(40, 30), (35, 30)])
    for _ in range(3):
        loop.step()
    with monkeypatch.context() as m:
        m.setattr(loop, "_new_caches", lambda n: (_ for _ in ()).throw(MemoryError("no room")))
        with pytest.raises(MemoryError):
            loop.resize(200)
    while not loop.done():
        st = loop.step()
        assert int(st.slot_mapping.max()) < 30 * 16
        check_rows(loop)


def test_shrinking_moves_blocks_in_use(_host_kernels):
    """Short requests leave low blocks, long ones hold high ones: the caches are
    made as small as the blocks in use allow."""
    loop = loop_of(64, [(60, 3), (100, 3), (40, 40), (70, 40), (33, 40)])
    moved = 0
    for step in range(30):
        loop.step()
        check_rows(loop)
        if step in (5, 15):
            used = {b for r in loop.running for b in loop.pool.block_table(r.rid)}
            del _host_kernels[:]
            assert not loop.resize(len(used))          # (the null block needs one, too)
            assert not _host_kernels
            n = len(used) + 1
            high = [b for b in used if b >= n]
            assert loop.resize(n) and loop.k_cache.shape[0] == n
            assert sorted(a for a, _ in _host_kernels) == sorted(high)
            moved += len(high)
            check_rows(loop)
            assert loop.resize(64)
            check_rows(loop)
    assert moved >= 3
