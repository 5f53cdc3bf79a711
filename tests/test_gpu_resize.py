"""A shrinking DecodeLoop on the GPU: the page copies of the compaction, in int8
caches (K, V and both scales) and bf16 ones.  The expected caches are made on the
host from the caches before the resize and the noted pairs, and followed from
there by the oracle's writes, bit for bit."""
import numpy as np
import pytest
import torch

import oracle
from oracle import int8 as O8
from paged_kv_cache_43_gb300 import decode_loop as DL
from paged_kv_cache_43_gb300 import pkv
from paged_kv_cache_43_gb300 import workloads as W
from tests.test_gpu_int8 import _lib, tolerance  # noqa: F401

pytestmark = pytest.mark.gpu


def host(t):
    return W.as_oracle_array(t.cpu()).copy()


@pytest.mark.parametrize("dtype,d", [(torch.int8, 128), (torch.int8, 64), (torch.bfloat16, 64)])
def test_shrinking_moves_blocks_in_use(dtype, d, monkeypatch):
    int8 = dtype == torch.int8
    pairs = []
    real = pkv.copy_blocks

    def copy_blocks(buffers, p, stream=None):
        pairs.extend((int(a), int(b)) for a, b in p)
        real(buffers, p, stream)

    monkeypatch.setattr(DL.pkv, "copy_blocks", copy_blocks)
    rng = np.random.default_rng(d)
    loop = DL.DecodeLoop(num_blocks=64, num_q_heads=8, num_kv_heads=2, head_size=d, dtype=dtype,
                         max_batch_tokens=400, seed=d)
    for prompt, new in ((60, 3), (100, 3), (40, 30), (70, 30), (33, 30)):
        loop.add_request([int(x) for x in rng.integers(0, 512, prompt)], new)
    caches = [host(t) for t in loop.buffers()]
    moved = steps = 0
    while not loop.done():
        if steps in (6, 10):                      # (shared blocks move; copies on write follow)
            loop.fork_request(loop.running[0].rid)
        if steps in (6, 9, 18):
            used = {b for r in loop.running for b in loop.pool.block_table(r.rid)}
            n = len(used) + 1                     # (and the null block)
            high = sorted(b for b in used if b >= n)
            del pairs[:]
            assert loop.resize(n)
            torch.cuda.synchronize()
            assert sorted(a for a, _ in pairs) == high
            moved += len(high)
            for a, b in pairs:
                for c in caches:
                    c[b] = c[a]
            caches = [c[:n] for c in caches]
            for got, want in zip(loop.buffers(), caches):
                assert host(got).tobytes() == want.tobytes()
            assert loop.resize(64)                # room again: nothing moves
            assert len(pairs) == len(high)
            more = [host(t) for t in loop.buffers()]
            for old, new in zip(caches, more):
                assert new[:n].tobytes() == old.tobytes()
            caches = [np.concatenate([old, new[n:]]) for old, new in zip(caches, more)]
        st = loop.step()
        steps += 1
        assert pkv.get_error() == 0
        for a, b in st.copies:
            for c in caches:
                c[b] = c[a]
        A = W.as_oracle_array
        if int8:
            O8.write(st.k_new.float().cpu().numpy(), st.v_new.float().cpu().numpy(),
                     host(st.block_tables), host(st.context_lens), host(st.query_start_loc), *caches)
            k, v = O8.widen(caches[0], caches[2]), O8.widen(caches[1], caches[3])
            q = st.q.float().cpu().numpy()
        else:
            assert oracle.write(A(st.k_new.cpu()), A(st.v_new.cpu()), host(st.slot_mapping), *caches) == 0
            k, v, q = *caches, A(st.q.cpu())
        for got, want in zip(loop.buffers(), caches):
            assert host(got).tobytes() == want.tobytes()
        ref, status = oracle.attention(q, k, v, host(st.block_tables), host(st.context_lens),
                                       host(st.query_start_loc), loop.scale)
        assert not status.any()
        out = st.out.float().cpu().numpy().astype(np.float64)
        if int8:
            assert (np.abs(out - ref) <= tolerance(ref, np.nanmax(np.abs(v)))).all()
        else:
            assert np.abs(out - ref).max() <= 2e-2
    assert moved >= 6
