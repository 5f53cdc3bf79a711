"""Drafted steps whose slots come from the framework's own block pool, many after one another, in a pool so
small that what one sequence drops another gets: against decoding the same tokens one by one."""
import numpy as np
import pytest
import torch

from drafts import ancestors, mask_words
from paged_kv_cache_43_gb300 import build, pkv
from paged_kv_cache_43_gb300.pool import BlockPool
from test_gpu_drafted_step import BS, D, HKV, LAYERS, Model, State, decode, i32, write

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


class Pooled(State):
    """Caches of the pool's size; NaN where nothing was written."""

    def __init__(self, fp8, seqs, blocks, stride):
        super().__init__(fp8, seqs, 16)
        dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
        nan = torch.full((blocks, BS, HKV, D), float("nan"), device="cuda")
        self.caches = [[nan.to(dt) for _ in range(2)] for _ in range(LAYERS)]
        self.pool, self.stride = BlockPool(blocks), stride


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("most", [6, 40])
def test_steps_on_the_pool_equal_decoding(fp8, most):
    rng = np.random.default_rng(most)
    m, S, stride = Model(), 5, 24
    blocks = 40 if most == 6 else 52
    spec, plain = Pooled(fp8, S, blocks, stride), State(fp8, S, 512, seed=1)
    pool = spec.pool
    head = [int(x) for x in rng.integers(0, 300, 32)]        # a prompt's start that some share
    tokens = [(head if s % 2 else []) + [int(x) for x in rng.integers(0, 300, 20 + 17 * s)] for s in range(S)]
    dropped = 0
    for s, t in enumerate(tokens):                           # the prompts but for their last token
        pool.add_request(s, t)
        first = pool.admit(s)
        assert first == (32 if s == 3 else 0)
        pos = np.arange(first, len(t) - 1)
        slots = pool.allocate_slots(s, len(pos))
        for layer in range(LAYERS):
            write(m, spec, layer, t[first:-1], pos, slots)
            write(m, plain, layer, t[:-1], np.arange(len(t) - 1), plain.slots(s, np.arange(len(t) - 1)))
    for step in range(10):
        before = [pool.num_computed(s) for s in range(S)]
        assert before == [len(t) - 1 for t in tokens]
        n = [int(rng.integers(1, most + 1)) for _ in range(S)]
        slots, done = pool.allocate_slots_batch(range(S), n)
        assert done == S and len(pool.take_copies()) == 0
        bits = [[b | 1 for b in ancestors(rng, k)] for k in n]            # (node 0: the last token)
        ids = [[t[-1]] + [int(x) for x in rng.integers(0, 300, k - 1)] for t, k in zip(tokens, n)]
        pos = np.array([p + bin(b).count("1") - 1 for p, rows in zip(before, bits) for b in rows])
        starts = np.concatenate([[0], np.cumsum(n)])
        L = [p + k for p, k in zip(before, n)]
        bt = torch.from_numpy(pool.block_tables(range(S), stride)).cuda()
        mask = mask_words([b for rows in bits for b in rows], -(-max(n) // 64)).cuda()
        outs = []
        for layer in range(LAYERS):
            q = write(m, spec, layer, [x for row in ids for x in row], pos, slots)
            out = torch.empty_like(q)
            args = (out, q, *spec.caches[layer], bt, i32(L), i32(starts.tolist()), mask, D ** -0.5)
            kw = dict(max_query_len=max(n), max_context_len=stride * BS)
            if fp8:
                pkv.attention_tree_fp8(*args, spec.descale, spec.descale, **kw)
            else:
                pkv.attention_tree(*args, **kw)
            outs.append(out)
        path = []
        for k, rows in zip(n, bits):
            end = int(rng.integers(0, k))
            path.append([j for j in range(k) if rows[end] >> j & 1])
        width = max(len(p) for p in path)
        new = torch.zeros(S, dtype=torch.int32, device="cuda")
        pkv.accept_drafts([c for layer in spec.caches for c in layer], bt, i32(L), i32(starts.tolist()),
                          i32([p + [-1] * (width - len(p)) for p in path]), i32([len(p) for p in path]),
                          new_context_lens=new)
        kept = [p + len(x) for p, x in zip(before, path)]
        pool.take_back(range(S), kept)
        dropped += sum(L) - sum(kept)
        assert new.tolist() == kept
        for j in range(width):          # the same tokens one by one
            live = [s for s in range(S) if j < len(path[s])]
            if j > 0:
                for s in live:
                    tokens[s].append(ids[s][path[s][j]])
            got = decode(m, plain, tokens)
            for s in live:
                at = int(starts[s]) + path[s][j]
                for layer in range(LAYERS):
                    a, b = outs[layer][at].float(), got[layer, s].float()
                    # two roundings to bf16 apart, and weights in 8 bits (tree) or 8 to 11:
                    # 2^-7 of the value and of the spread of V (4 and less, in N(0, 1))
                    assert bool(((a - b).abs() <= 2.0 ** -7 * (b.abs() + 4)).all())
        for s in range(S):              # the next root
            tokens[s].append(int(rng.integers(0, 300)))
            pool.append_tokens(s, tokens[s][-len(path[s]):])
        if step == 6:                   # one that goes, and a new one with its tokens: their blocks are hits
            pool.free_request(2)
            pool.add_request(2, tokens[2])
            first = pool.admit(2)
            assert first == (len(tokens[2]) - 1) // BS * BS
            at = np.arange(first, len(tokens[2]) - 1)
            slots = pool.allocate_slots(2, len(at))
            for layer in range(LAYERS):
                write(m, spec, layer, tokens[2][first:-1], at, slots)
    assert dropped > 30
