"""A step with drafted tokens as it is used -- rotation and write of a tree's tokens, attention
of the tree, the accepted path's rows kept -- against decoding the same tokens one by one."""
import numpy as np
import pytest
import torch

from drafts import ancestors, mask_words
from paged_kv_cache_43_gb300 import build, pkv

pytestmark = pytest.mark.gpu
HQ, HKV, D, LAYERS, BS = 8, 2, 128, 2, 16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    pkv.load()
    pkv.get_error(clear=True)
    yield
    assert pkv.get_error(clear=True) == 0


class Model:
    """q, k, v rows of a token id in each layer, before norms and rotation."""

    def __init__(self, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.t = [torch.randn(300, HQ + 2 * HKV, D, generator=g).to(torch.bfloat16).cuda()
                  for _ in range(LAYERS)]
        self.qw, self.kw = ((1 + 0.2 * torch.randn(D, generator=g)).to(torch.bfloat16).cuda()
                            for _ in range(2))
        f = 10000.0 ** -(torch.arange(D // 2, dtype=torch.float64) / (D // 2))
        a = torch.arange(4096, dtype=torch.float64)[:, None] * f
        self.cs = torch.cat([a.cos(), a.sin()], 1).float().cuda()

    def rows(self, layer, ids):
        x = self.t[layer][torch.as_tensor(ids, device="cuda")]
        return x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:]


class State:
    def __init__(self, fp8, seqs, room, seed=0):
        self.fp8 = fp8
        dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
        per = -(-room // BS)
        nb = seqs * per + 4
        order = np.random.default_rng(seed).permutation(nb)[:seqs * per].reshape(seqs, per)
        self.table = order.astype(np.int32)
        self.bt = torch.from_numpy(self.table).cuda()
        nan = torch.full((nb, BS, HKV, D), float("nan"), device="cuda")
        self.caches = [[nan.to(dt) for _ in range(2)] for _ in range(LAYERS)]
        self.scale = torch.full((HKV,), 0.02, device="cuda")
        self.descale = torch.full((seqs, HKV), 0.02, device="cuda")

    def slots(self, s, positions):
        p = np.asarray(positions)
        return self.table[s, p // BS].astype(np.int64) * BS + p % BS


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def write(m, st, layer, ids, pos, slots):
    q, k, v = m.rows(layer, ids)
    out = torch.zeros((len(ids), HQ, D), dtype=torch.bfloat16, device="cuda")
    args = (out, q, k, v, torch.as_tensor(pos, device="cuda"), m.cs,
            torch.as_tensor(slots, device="cuda"), *st.caches[layer])
    kw = dict(q_weight=m.qw, k_weight=m.kw)
    if st.fp8:
        pkv.rope_write_fp8(*args, st.scale, st.scale, **kw)
    else:
        pkv.rope_write(*args, **kw)
    return out


def decode(m, st, tokens):
    """Each sequence's last token, one by one: the outputs [layers, seqs, HQ, D]."""
    S = len(tokens)
    pos = np.array([len(t) - 1 for t in tokens])
    slots = np.concatenate([st.slots(s, [p]) for s, p in enumerate(pos)])
    outs = []
    for layer in range(LAYERS):
        q = write(m, st, layer, [t[-1] for t in tokens], pos, slots)
        out = torch.empty_like(q)
        args = (out, q, *st.caches[layer], st.bt, i32([len(t) for t in tokens]),
                i32(list(range(S + 1))), D ** -0.5)
        kw = dict(max_query_len=1, max_context_len=st.bt.shape[1] * BS)
        if st.fp8:
            pkv.attention_fp8(*args, st.descale, st.descale, **kw)
        else:
            pkv.attention(*args, **kw)
        outs.append(out)
    return torch.stack(outs)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("most", [6, 40])
def test_speculative_steps_equal_decoding(fp8, most):
    rng = np.random.default_rng(most)
    m, S = Model(), 5
    spec, plain = State(fp8, S, 512), State(fp8, S, 512, seed=1)
    tokens = [[int(x) for x in rng.integers(0, 300, 20 + 31 * s)] for s in range(S)]
    for st in (spec, plain):       # the prompts
        for s, t in enumerate(tokens):
            pos = np.arange(len(t))
            for layer in range(LAYERS):
                write(m, st, layer, t, pos, st.slots(s, pos))
    for step in range(6):
        n = [int(rng.integers(1, most + 1)) for _ in range(S)]
        L = [len(t) + k for t, k in zip(tokens, n)]
        # trees of ids: node 0 the root, a node's position by its depth
        bits = [ancestors(rng, k) for k in n]
        bits = [[b | 1 for b in rows] for rows in bits]       # (one root)
        depth = [[bin(b).count("1") - 1 for b in rows] for rows in bits]
        ids = [[int(x) for x in rng.integers(0, 300, k)] for k in n]
        flat = [x for row in ids for x in row]
        pos = np.array([len(t) + d for t, row in zip(tokens, depth) for d in row])
        slots = np.concatenate([spec.slots(s, np.arange(len(t), len(t) + k))
                                for s, (t, k) in enumerate(zip(tokens, n))])
        starts = np.concatenate([[0], np.cumsum(n)])
        mask = mask_words([b for row in bits for b in row], -(-max(n) // 64)).cuda()
        outs = []
        for layer in range(LAYERS):
            q = write(m, spec, layer, flat, pos, slots)
            out = torch.empty_like(q)
            args = (out, q, *spec.caches[layer], spec.bt, i32(L), i32(starts.tolist()), mask, D ** -0.5)
            kw = dict(max_query_len=max(n), max_context_len=spec.bt.shape[1] * BS)
            if fp8:
                pkv.attention_tree_fp8(*args, spec.descale, spec.descale, **kw)
            else:
                pkv.attention_tree(*args, **kw)
            outs.append(out)
        # a path from the root down to some node is right
        path = []
        for k, rows in zip(n, bits):
            end = int(rng.integers(0, k))
            path.append([j for j in range(k) if rows[end] >> j & 1])
        width = max(len(p) for p in path)
        accepted = i32([p + [-1] * (width - len(p)) for p in path])
        new = torch.zeros(S, dtype=torch.int32, device="cuda")
        pkv.accept_drafts([c for layer in spec.caches for c in layer], spec.bt, i32(L),
                          i32(starts.tolist()), accepted, i32([len(p) for p in path]),
                          new_context_lens=new)
        # the same tokens one by one
        for j in range(width):
            live = [s for s in range(S) if j < len(path[s])]
            for s in live:
                tokens[s].append(ids[s][path[s][j]])
            got = decode(m, plain, tokens)     # (the others once more: the same rows)
            for s in live:
                at = int(starts[s]) + path[s][j]
                for layer in range(LAYERS):
                    a, b = outs[layer][at].float(), got[layer, s].float()
                    # two roundings to bf16 apart, and weights in 8 bits (tree) or 8 to 11:
                    # 2^-7 of the value and of the spread of V (4 and less, in N(0, 1))
                    assert bool(((a - b).abs() <= 2.0 ** -7 * (b.abs() + 4)).all())
        assert new.tolist() == [len(t) for t in tokens]
        for layer in range(LAYERS):            # the kept rows are the decoded ones, bit for bit
            for x, y in zip(spec.caches[layer], plain.caches[layer]):
                for s, t in enumerate(tokens):
                    p = np.arange(len(t))
                    u, v = (c.view(torch.uint8).flatten(0, 1)[torch.from_numpy(st.slots(s, p)).cuda()]
                            for c, st in ((x, spec), (y, plain)))
                    assert torch.equal(u, v)


def test_a_step_in_a_graph():
    """Write, attention and accepted rows captured together, replayed on other lengths, tokens,
    masks and paths."""
    rng = np.random.default_rng(0)
    m, S, k = Model(), 3, 7
    st, eager = State(False, S, 256), State(False, S, 256)
    for x in (st, eager):
        for layer in range(LAYERS):
            for c in x.caches[layer]:
                c.copy_(torch.randn(c.shape, generator=torch.Generator().manual_seed(layer)))
    x = dict(q=torch.zeros(S * k, HQ + 2 * HKV, D, dtype=torch.bfloat16, device="cuda"),
             pos=torch.zeros(S * k, dtype=torch.int64, device="cuda"),
             slots=torch.zeros(S * k, dtype=torch.int64, device="cuda"),
             mask=torch.zeros(S * k, 1, dtype=torch.int64, device="cuda"),
             L=i32([k] * S), starts=i32([k * s for s in range(S + 1)]), path=i32([[0] * 4] * S),
             taken=i32([1] * S), new=i32([0] * S))
    out = torch.zeros(S * k, HQ, D, dtype=torch.bfloat16, device="cuda")
    rot = torch.zeros_like(out)
    meta = pkv.attn_meta(out, st.bt, x["L"], max_query_len=k, max_context_len=256)
    ws = torch.empty(max(pkv.workspace_size_tree(st.caches[0][0], meta), 256), dtype=torch.uint8,
                     device="cuda")

    def step(s):
        q, kk, v = x["q"][:, :HQ], x["q"][:, HQ:HQ + HKV], x["q"][:, HQ + HKV:]
        for layer in range(LAYERS):
            pkv.rope_write(rot, q, kk, v, x["pos"], m.cs, x["slots"], *s.caches[layer])
            pkv.attention_tree(out, rot, *s.caches[layer], s.bt, x["L"], x["starts"], x["mask"],
                               D ** -0.5, max_query_len=k, max_context_len=256, workspace=ws)
        pkv.accept_drafts([c for l in s.caches for c in l], s.bt, x["L"], x["starts"], x["path"],
                          x["taken"], new_context_lens=x["new"])

    def inputs():
        before = rng.integers(0, 200, S)
        x["q"].normal_()
        x["pos"].copy_(torch.from_numpy(rng.integers(0, 4096, S * k)))
        x["slots"].copy_(torch.from_numpy(np.concatenate(
            [st.slots(s, np.arange(b, b + k)) for s, b in enumerate(before)])))
        x["mask"].copy_(mask_words([b for _ in range(S) for b in ancestors(rng, k)], 1))
        x["L"].copy_(torch.from_numpy(before + k).int())
        x["path"].copy_(torch.from_numpy(np.stack([np.sort(rng.permutation(k)[:4])
                                                   for _ in range(S)])).int())
        x["taken"].copy_(torch.from_numpy(rng.integers(0, 5, S)).int())

    inputs()
    step(st)
    for a, b in zip(st.caches, eager.caches):
        for u, v in zip(a, b):
            v.copy_(u)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(st)
    for _ in range(3):
        inputs()
        g.replay()
        got, lens = out.clone(), x["new"].clone()
        step(eager)
        assert torch.equal(got, out) and torch.equal(lens, x["new"])
        for a, b in zip(st.caches, eager.caches):
            for u, v in zip(a, b):
                assert torch.equal(u.view(torch.int16), v.view(torch.int16))
