"""Timed cases of a decoding step with drafted tokens over the paged cache.

Three operators, in the order in which a step of speculative decoding calls them:

* ``rope``: the pass between the QKV projection and attention.  Each query and key head's row x
  is normalised, y = x / sqrt(mean(x^2) + eps) * w (where the model has such norms), the first
  rot_dim elements of y are rotated by the token's position, q goes to its own tensor, k and v to
  their rows of the cache (bf16, fp32, or e4m3 codes of value / scale), or k to rows of its own.
* ``tree``: softmax attention of a tree of drafted tokens.  The last n keys of a sequence are its
  n drafted tokens; token i sees every key before them, and drafted key j where bit j of its mask
  row is set.
* ``accept``: the rows of the accepted path's tokens, in every layer's caches, move to the places
  right behind the keys that were there before the drafts.

``run`` computes them with elementary torch operations in fp32, or through the package's calls
where ``own`` is true.
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = 16
BYTES = {"bf16": 2, "f32": 4, "e4m3": 1}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # a quiet server: one sequence's next token, 32 query and 8 kv heads with norms
        dict(name="rope 1", op="rope", tokens=1, hq=32, hkv=8, d=128, rot=128, norm=True,
             interleaved=False, cache="bf16", packed=True, pad=0.0, max_position=8192),
        # 64 sequences with a tree of 16 drafts each, LLaMA-7B heads, no norms
        dict(name="rope 64 x 16", op="rope", tokens=1024, hq=32, hkv=32, d=128, rot=128,
             norm=False, interleaved=False, cache="bf16", packed=True, pad=0.0, max_position=8192),
        # a padded batch into an e4m3 cache, 5 kv heads of 64, half of the head rotated, in pairs
        dict(name="rope e4m3 pairs", op="rope", tokens=2999, hq=15, hkv=5, d=64, rot=32, norm=True,
             interleaved=True, cache="e4m3", packed=True, pad=0.2, max_position=4096),
        # prompts of 16384 tokens in one step
        dict(name="rope 16384", op="rope", tokens=16384, hq=32, hkv=8, d=128, rot=128, norm=True,
             interleaved=False, cache="bf16", packed=True, pad=0.0, max_position=32768),
        # one user, 16 drafts over a short context: latency alone counts
        dict(name="tree 1 x 16", op="tree", seqs=1, nodes_lo=16, nodes_hi=16, lo=1000, hi=1000,
             log=False, hq=32, hkv=8, d=128, cache="bf16", blank=0.0, shape=1),
        # few users with the largest usual trees
        dict(name="tree 8 x 64", op="tree", seqs=8, nodes_lo=64, nodes_hi=64, lo=2048, hi=8192,
             log=False, hq=32, hkv=8, d=128, cache="bf16", blank=0.0, shape=2),
        # the default decode batch, small trees, a kv head for every query head
        dict(name="tree 64 x 16 heads", op="tree", seqs=64, nodes_lo=8, nodes_hi=16, lo=128,
             hi=4096, log=False, hq=32, hkv=32, d=128, cache="bf16", blank=0.0, shape=3),
        # long documents, 8 query heads on a kv head
        dict(name="tree 16 long", op="tree", seqs=16, nodes_lo=26, nodes_hi=26, lo=16384, hi=32768,
             log=False, hq=64, hkv=8, d=128, cache="bf16", blank=0.0, shape=4),
        # an e4m3 cache under many sequences of very different lengths
        dict(name="tree e4m3 128", op="tree", seqs=128, nodes_lo=1, nodes_hi=24, lo=64, hi=8192,
             log=True, hq=32, hkv=8, d=128, cache="e4m3", blank=0.0, shape=5),
        # a ragged batch, 3 query heads on a kv head of 64, drafts that see no draft at all
        dict(name="tree ragged", op="tree", seqs=23, nodes_lo=0, nodes_hi=77, lo=1, hi=3000,
             log=True, hq=12, hkv=4, d=64, cache="bf16", blank=0.1, shape=6),
        # one user's accepted path, 16 layers
        dict(name="accept 1", op="accept", seqs=1, nodes_lo=16, nodes_hi=16, most=4, lo=1000,
             hi=1000, layers=16, hkv=8, d=128, cache="bf16", shape=4),
        # a busy server's, 16 layers
        dict(name="accept 256", op="accept", seqs=256, nodes_lo=8, nodes_hi=32, most=8, lo=64,
             hi=512, layers=16, hkv=8, d=128, cache="bf16", shape=8),
    ]


def _log_int(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "tree", "tree", "tree", "accept"])
    d = rng.choice([64, 128, 128])
    shape = rng.randrange(1 << 20)
    if op == "rope":
        hkv = rng.choice([1, 2, 3, 5, 8, 32])
        hq = hkv * rng.choice([1, 2, 3, 4, 7, 8] if hkv < 32 else [1, 2])
        cache = rng.choice(["bf16", "bf16", "e4m3", "f32", "rows"])
        most = 16384 * 48 * 128 // ((hq + 2 * hkv) * d * (2 if cache == "f32" else 1))
        return dict(op=op, tokens=_log_int(rng, 1, min(most, 16384)), hq=hq, hkv=hkv, d=d,
                    rot=rng.choice([d, d, d // 2, d // 4, 6]), norm=rng.random() < 0.7,
                    interleaved=rng.random() < 0.4, cache=cache, packed=rng.random() < 0.7,
                    pad=0.0 if cache == "rows" else rng.choice([0.0, 0.0, 0.3]),
                    max_position=_log_int(rng, 64, 100000))
    if op == "accept":
        lo, hi = sorted(rng.randrange(1, 65) for _ in range(2))
        return dict(op=op, seqs=_log_int(rng, 1, 256), nodes_lo=lo, nodes_hi=hi,
                    most=rng.randrange(1, min(lo, 8) + 1), lo=rng.randrange(0, 64),
                    hi=_log_int(rng, 64, 400), layers=rng.randrange(1, 9),
                    hkv=rng.choice([1, 2, 5, 8]), d=d, cache=rng.choice(["bf16", "e4m3", "f32"]),
                    shape=shape)
    cache = rng.choice(["bf16", "bf16", "bf16", "e4m3", "e4m3", "f32"])
    group = rng.choice([1, 2, 3, 4, 5, 8, 16])
    hkv = rng.choice([1, 2, 3, 4, 8]) if group > 4 else rng.choice([2, 4, 5, 8, 16])
    nodes_hi = _log_int(rng, 1, 150)
    nodes_lo = rng.randrange(0, nodes_hi + 1)
    hi = _log_int(rng, 8, 3000 if cache == "f32" else 20000)
    # sequences x keys x kv heads, and with the query rows too, stay under the listed batches
    most = min((1 << 21) // (hi * hkv), (1 << 28) // (hi * hkv * group * max(nodes_hi, 4)))
    if cache == "f32":
        most = min(most, 8)
    return dict(op=op, seqs=_log_int(rng, 1, max(1, min(128, most))), nodes_lo=nodes_lo,
                nodes_hi=nodes_hi, lo=_log_int(rng, 1, hi), hi=hi, log=rng.random() < 0.5,
                hq=group * hkv, hkv=hkv, d=d, cache=cache, blank=rng.choice([0.0, 0.0, 0.2]),
                shape=shape)


def _drafts(case):
    """(drafted tokens, keys with them) of each sequence."""
    rng = random.Random(case["shape"])
    n = [rng.randint(case["nodes_lo"], case["nodes_hi"]) for _ in range(case["seqs"])]
    if not sum(n):
        n[0] = 1
    before = [_log_int(rng, max(case["lo"], 1), max(case["hi"], 1)) if case.get("log")
              else rng.randint(case["lo"], case["hi"]) for _ in n]
    # (now and then a tree at the very start of its sequence)
    if case["op"] == "tree" and case["blank"]:
        before[-1] = 0
    return n, [b + k for b, k in zip(before, n)]


def _paths(case):
    """The accepted nodes of each sequence: rising, from the first node on."""
    rng = random.Random(case["shape"] + 1)
    n, _ = _drafts(case)
    out = []
    for k in n:
        take = rng.randint(0, min(case["most"], k))
        out.append([0] + sorted(rng.sample(range(1, k), take - 1)) if take else [])
    return out


def work(case):
    d, hkv = case["d"], case["hkv"]
    if case["op"] == "rope":
        tokens = case["tokens"] - int(case["tokens"] * case["pad"])
        e = BYTES.get(case["cache"], 2)
        x = 4 if e == 4 else 2
        q, kv = case["hq"] * d, (1 if case["cache"] == "rows" else 2) * hkv * d
        rows = 8 * case["rot"] // 2 * min(tokens, case["max_position"])
        norms = 2 * d * x if case["norm"] else 0
        return {"bytes": tokens * (2 * q * x + kv * (x + e) + 8) + 8 * case["tokens"] + rows + norms,
                "flops": 0}
    if case["op"] == "accept":
        moved = sum(j != p for path in _paths(case) for j, p in enumerate(path))
        # the tables' touched entries, lengths and paths, and the rows
        small = case["seqs"] * (16 + 4 * case["most"]) + 8 * moved
        return {"bytes": 2 * 2 * case["layers"] * moved * hkv * d * BYTES[case["cache"]] + small,
                "flops": 0}
    n, keys = _drafts(case)
    keys = [k if m else 0 for m, k in zip(n, keys)]
    e = BYTES[case["cache"]]
    moved = 2 * hkv * d * e * sum(keys) + sum(n) * case["hq"] * d * 2 * (4 if e == 4 else 2)
    moved += 4 * sum(-(-k // BLOCK) for k in keys) + 8 * sum(n) * -(-max(n) // 64)
    # (a draft sees about a tenth of its tree: the keys before the tree are counted, and itself)
    flops = 4 * d * case["hq"] * sum(m * (k - m + 1) for m, k in zip(n, keys))
    return {"bytes": moved, "flops": flops}


# ------------------------------------------------------------------ inputs

def _cache_of(kind, x):
    """x as a cache holds it (e4m3: codes of x / 0.02)."""
    if kind == "e4m3":
        return (x / 0.02).clamp(-448, 448).to(torch.float8_e4m3fn)
    return x.float() if kind == "f32" else x.to(torch.bfloat16)


def _batch(case, host, dev):
    """Tables, lengths and row starts of the drafted batch, in a pool a tenth larger than it needs."""
    n, keys = _drafts(case)
    nblk = [-(-k // BLOCK) for k in keys]
    nb = sum(nblk) + sum(nblk) // 10 + 1
    order = host.permutation(nb).astype(np.int32)
    tables = np.full((len(n), max(max(nblk), 1)), -1, np.int32)
    at = 0
    for s, b in enumerate(nblk):
        tables[s, :b] = order[at:at + b]
        at += b
    starts = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    return dict(case=case, tokens=int(sum(n)), blocks=nb, max_query_len=max(n),
                max_context_len=max(keys), tables=torch.from_numpy(tables).to(dev),
                lens=torch.tensor(keys, dtype=torch.int32, device=dev),
                starts=torch.from_numpy(starts).to(dev))


def _masks(case, host):
    """Bits of each drafted token's mask row: itself and its ancestors in a random tree, whose
    first token is the root; a share of `blank` sees no draft, itself neither."""
    n, _ = _drafts(case)
    words = -(-max(n) // 64)
    rows = []
    for k in n:
        seen = []
        for i in range(k):
            parent = int(host.integers(max(0, i - 12), i)) if i else -1
            seen.append((seen[parent] if i else 0) | 1 << i)
        rows += [0 if host.random() < case["blank"] else b for b in seen]
    out = np.zeros((len(rows), words), np.uint64)
    for t, b in enumerate(rows):
        for w in range(words):
            out[t, w] = b >> 64 * w & (1 << 64) - 1
    return torch.from_numpy(out.view(np.int64))


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    host = np.random.default_rng(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    hkv, d, kind = case["hkv"], case["d"], case["cache"]
    # keys have channels of different size, as projections leave them
    channel = (0.5 * normal(hkv, d)).exp()
    if case["op"] == "accept":
        st = _batch(case, host, dev)
        shape = (st["blocks"], BLOCK, hkv, d)
        st["buffers"] = [_cache_of(kind, normal(*shape) * channel)
                         for _ in range(2 * case["layers"])]
        paths = _paths(case)
        path = np.full((len(paths), case["most"]), -1, np.int32)
        for s, p in enumerate(paths):
            path[s, :len(p)] = p
        st["path"] = torch.from_numpy(path).to(dev)
        st["taken"] = torch.tensor([len(p) for p in paths], dtype=torch.int32, device=dev)
        st["new_lens"] = torch.zeros_like(st["lens"])
        return st
    if case["op"] == "tree":
        st = _batch(case, host, dev)
        x = torch.float32 if kind == "f32" else torch.bfloat16
        shape = (st["blocks"], BLOCK, hkv, d)
        st["k_cache"] = _cache_of(kind, normal(*shape) * channel)
        st["v_cache"] = _cache_of(kind, normal(*shape))
        st["mask"] = _masks(case, host).to(dev)
        st["q"] = normal(st["tokens"], case["hq"], d).to(x)
        st["out"] = torch.zeros_like(st["q"])
        st["scale"] = 1.0 / math.sqrt(d)
        if kind == "e4m3":   # a scale for each sequence and kv head
            st["k_descale"] = 0.02 * (0.1 * normal(case["seqs"], hkv)).exp()
            st["v_descale"] = 0.02 * (0.1 * normal(case["seqs"], hkv)).exp()
        return st
    tokens, hq, rot = case["tokens"], case["hq"], case["rot"]
    x = torch.float32 if kind == "f32" else torch.bfloat16
    st = dict(case=case)
    if case["packed"]:   # slices of one projection's output
        qkv = (normal(tokens, hq + 2 * hkv, d) * 1.5).to(x).view(tokens, -1)
        st["q"], st["k"], st["v"] = (t.view(tokens, -1, d) for t in
                                     qkv.split([hq * d, hkv * d, hkv * d], 1))
    else:
        st["q"] = (normal(tokens, hq, d) * 1.5).to(x)
        st["k"], st["v"] = ((normal(tokens, hkv, d) * 1.5).to(x) for _ in range(2))
    st["q_weight"] = (1 + 0.2 * normal(d)).to(x) if case["norm"] else None
    st["k_weight"] = (1 + 0.2 * normal(d)).to(x) if case["norm"] else None
    st["eps"] = 1e-6
    # cosines and sines of position x frequency, angles in 64 bits
    freq = 10000.0 ** -(torch.arange(rot // 2, device=dev, dtype=torch.float64) / (rot // 2))
    angle = torch.arange(case["max_position"], device=dev, dtype=torch.float64)[:, None] * freq
    st["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    st["positions"] = torch.from_numpy(host.integers(0, case["max_position"], tokens)).to(dev)
    st["q_out"] = torch.zeros((tokens, hq, d), dtype=x, device=dev)
    if kind == "rows":
        st["k_out"] = torch.zeros((tokens, hkv, d), dtype=x, device=dev)
        return st
    nb = -(-tokens // BLOCK) + tokens // (10 * BLOCK) + 1
    slots = host.permutation(nb * BLOCK)[:tokens].astype(np.int64)
    slots[host.permutation(tokens)[:int(tokens * case["pad"])]] = -1
    st["slots"] = torch.from_numpy(slots).to(dev)
    for name in ("k_cache", "v_cache"):
        st[name] = _cache_of(kind, normal(nb, BLOCK, hkv, d))
    if kind == "e4m3":   # a scale for each kv head: its largest magnitudes near 448
        st["k_scale"] = 0.02 * (0.1 * normal(hkv)).exp()
        st["v_scale"] = 0.02 * (0.1 * normal(hkv)).exp()
    return st


# --------------------------------------------------------------- plain forms

def _rotated(x, weight, eps, c, s, interleaved):
    """x [tokens, heads, d] in fp32: normalised, its first 2 x c.shape[1] elements rotated."""
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * weight.float()
    half = c.shape[1]
    turn, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = turn[..., 0::2], turn[..., 1::2]
    else:
        a, b = turn[..., :half], turn[..., half:]
    c, s = c[:, None], s[:, None]
    a, b = a * c - b * s, b * c + a * s
    turn = torch.stack([a, b], -1).flatten(2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([turn, rest], -1)


def _plain_rope(st):
    case = st["case"]
    c, s = st["cos_sin"][st["positions"]].chunk(2, 1)
    how = (st["eps"], c, s, case["interleaved"])
    q = _rotated(st["q"].float(), st["q_weight"], *how).to(st["q_out"].dtype)
    k = _rotated(st["k"].float(), st["k_weight"], *how)
    if case["cache"] == "rows":
        return dict(q=q, k=k.to(q.dtype))
    live = st["slots"] >= 0
    at = st["slots"][live]
    v = st["v"].float()
    if case["cache"] == "e4m3":
        k = (k / st["k_scale"][:, None]).clamp(-448, 448)
        v = (v / st["v_scale"][:, None]).clamp(-448, 448)
    st["q_out"][live] = q[live]
    # (indexed assignment of one-byte floats goes by their bytes)
    e = torch.uint8 if case["cache"] == "e4m3" else st["k_cache"].dtype
    st["k_cache"].view(e).flatten(0, 1)[at] = k[live].to(st["k_cache"].dtype).view(e)
    st["v_cache"].view(e).flatten(0, 1)[at] = v[live].to(st["v_cache"].dtype).view(e)
    return dict(q=st["q_out"], k_cache=st["k_cache"], v_cache=st["v_cache"])


def _plain_tree(st):
    """Blocks gathered and widened, sequences padded to the longest, one masked softmax."""
    case = st["case"]
    hkv = case["hkv"]
    dev = st["q"].device
    blocks = st["tables"].long().clamp_min(0)

    def gathered(name):
        byte = case["cache"] == "e4m3"
        x = st[name + "_cache"]
        x = (x.view(torch.uint8)[blocks].view(x.dtype) if byte else x[blocks]).float()
        x = x.flatten(1, 2)                                  # [seqs, keys, kv heads, d]
        return x * st[name + "_descale"][:, None, :, None] if byte else x

    k, v = gathered("k"), gathered("v")
    starts, lens = st["starts"].long(), st["lens"].long()
    n = starts[1:] - starts[:-1]
    j = torch.arange(st["max_query_len"], device=dev)
    rows = (starts[:-1, None] + j).clamp_max(st["tokens"] - 1)
    q = st["q"].float()[rows].unflatten(2, (hkv, -1))        # [seqs, rows, kv heads, group, d]
    bits = st["mask"][rows][..., None] >> torch.arange(64, device=dev) & 1
    bits = bits.flatten(2).bool()                            # [seqs, rows, drafts]
    key = torch.arange(k.shape[1], device=dev)
    draft = key - (lens - n)[:, None]                        # [seqs, keys]
    at = draft.clamp(0, bits.shape[2] - 1)[:, None].expand(-1, rows.shape[1], -1)
    seen = bits.gather(2, at) & ((draft >= 0) & (draft < n[:, None]))[:, None]
    hidden = ~(seen | (draft < 0)[:, None])
    s = torch.einsum("srhgd,skhd->shgrk", q, k) * st["scale"]
    s.masked_fill_(hidden[:, None, None], -math.inf)
    s -= s.amax(-1, keepdim=True).clamp_min(-1e30)
    s.exp_()
    total = s.sum(-1, keepdim=True)
    v = v.masked_fill((key >= lens[:, None])[:, :, None, None], 0.0)
    o = torch.einsum("shgrk,skhd->shgrd", s, v) / torch.where(total > 0, total, 1.0)
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)               # [seqs, rows, query heads, d]
    t = torch.arange(st["tokens"], device=dev)
    seq = torch.searchsorted(starts[1:], t, right=True)
    return o[seq, t - starts[seq]].to(st["q"].dtype)


def _plain_accept(st):
    starts, lens = st["starts"].long(), st["lens"].long()
    before = lens - (starts[1:] - starts[:-1])
    j = torch.arange(st["path"].shape[1], device=lens.device)
    seq, at = torch.nonzero(j < st["taken"][:, None], as_tuple=True)
    tables = st["tables"].long()

    def slot(p):
        return tables[seq, p // BLOCK] * BLOCK + p % BLOCK

    src = slot(before[seq] + st["path"].long()[seq, at])
    dst = slot(before[seq] + at)
    e = torch.uint8 if st["case"]["cache"] == "e4m3" else st["buffers"][0].dtype
    rows = [b.view(e).flatten(0, 1) for b in st["buffers"]]
    moved = [r.index_copy_(0, dst, r.index_select(0, src)) for r in rows]
    new = (before + st["taken"]).int()
    return dict(buffers=st["buffers"] if moved else [], lens=new)


def run(state):
    st, case = state, state["case"]
    if not own:
        return {"rope": _plain_rope, "tree": _plain_tree, "accept": _plain_accept}[case["op"]](st)
    from paged_kv_cache_43_gb300 import pkv
    if case["op"] == "rope":
        kw = dict(q_weight=st["q_weight"], k_weight=st["k_weight"], eps=st["eps"],
                  interleaved=case["interleaved"])
        if case["cache"] == "rows":
            pkv.rope(st["q_out"], st["k_out"], st["q"], st["k"], st["positions"], st["cos_sin"],
                     **kw)
            return dict(q=st["q_out"], k=st["k_out"])
        if case["cache"] == "e4m3":
            pkv.rope_write_fp8(st["q_out"], st["q"], st["k"], st["v"], st["positions"],
                               st["cos_sin"], st["slots"], st["k_cache"], st["v_cache"],
                               st["k_scale"], st["v_scale"], **kw)
        else:
            pkv.rope_write(st["q_out"], st["q"], st["k"], st["v"], st["positions"], st["cos_sin"],
                           st["slots"], st["k_cache"], st["v_cache"], **kw)
        return dict(q=st["q_out"], k_cache=st["k_cache"], v_cache=st["v_cache"])
    if case["op"] == "tree":
        kw = dict(max_query_len=st["max_query_len"], max_context_len=st["max_context_len"])
        if case["cache"] == "e4m3":
            pkv.attention_tree_fp8(st["out"], st["q"], st["k_cache"], st["v_cache"], st["tables"],
                                   st["lens"], st["starts"], st["mask"], st["scale"],
                                   st["k_descale"], st["v_descale"], **kw)
        else:
            pkv.attention_tree(st["out"], st["q"], st["k_cache"], st["v_cache"], st["tables"],
                               st["lens"], st["starts"], st["mask"], st["scale"], **kw)
        return st["out"]
    pkv.accept_drafts(st["buffers"], st["tables"], st["lens"], st["starts"], st["path"],
                      st["taken"], new_context_lens=st["new_lens"])
    return dict(buffers=st["buffers"], lens=st["new_lens"])


# --------------------------------------------------------------- definitions

def _exact_rope(st):
    case = st["case"]
    half = case["rot"] // 2
    table = st["cos_sin"].double()[st["positions"]]
    turn = torch.complex(table[:, :half], table[:, half:])[:, None]

    def one(x, w):
        x = x.double()
        if w is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / case["d"] + st["eps"]).sqrt() * w.double()
        y = x.clone()
        first = slice(0, 2 * half, 2) if case["interleaved"] else slice(0, half)
        second = slice(1, 2 * half, 2) if case["interleaved"] else slice(half, 2 * half)
        z = torch.complex(x[..., first], x[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    q, k = one(st["q"], st["q_weight"]), one(st["k"], st["k_weight"])
    if case["cache"] == "rows":
        return dict(q=q, k=k)
    v = st["v"].double()
    if case["cache"] == "e4m3":
        k = (k / st["k_scale"].double()[:, None]).clamp(-448, 448)
        v = (v / st["v_scale"].double()[:, None]).clamp(-448, 448)
    out = dict(q=st["q_out"].double(), k_cache=st["k_cache"].double(),
               v_cache=st["v_cache"].double())
    live = st["slots"] >= 0
    out["q"][live] = q[live]
    for name, x in (("k_cache", k), ("v_cache", v)):
        out[name].view(-1, *x.shape[1:])[st["slots"][live]] = x[live]
    return out


def _exact_tree(st):
    """Sequence by sequence and kv head by kv head, from the definition."""
    case = st["case"]
    group = case["hq"] // case["hkv"]
    lens, starts = st["lens"].tolist(), st["starts"].tolist()
    masks = [sum((w & (1 << 64) - 1) << 64 * i for i, w in enumerate(row))
             for row in st["mask"].tolist()]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=st["q"].device)
    for s in range(case["seqs"]):
        t0, t1 = starts[s], starts[s + 1]
        n, length = t1 - t0, lens[s]
        if not n:
            continue
        seen = np.ones((n, length), bool)
        for i in range(n):
            seen[i, length - n:] = [masks[t0 + i] >> j & 1 for j in range(n)]
        hidden = torch.from_numpy(~seen).to(out.device)
        empty = hidden.all(1)[None, :, None]
        at = st["tables"][s, :-(-length // BLOCK)].long()
        for h in range(case["hkv"]):
            k, v = (st[c + "_cache"][:, :, h][at] if case["cache"] != "e4m3" else
                    st[c + "_cache"].view(torch.uint8)[:, :, h][at].view(torch.float8_e4m3fn)
                    for c in "kv")
            k, v = (x.double().flatten(0, 1)[:length] for x in (k, v))
            if case["cache"] == "e4m3":
                k = k * st["k_descale"][s, h].double()
                v = v * st["v_descale"][s, h].double()
            heads = slice(h * group, (h + 1) * group)
            x = st["q"][t0:t1, heads].double().transpose(0, 1) @ k.T / math.sqrt(case["d"])
            w = torch.softmax(x.masked_fill(hidden, -math.inf), -1).masked_fill(empty, 0.0)
            out[t0:t1, heads] = (w @ v).transpose(0, 1)
    return out


def _exact_accept(st):
    lens, starts = st["lens"].tolist(), st["starts"].tolist()
    tables, taken, path = st["tables"].tolist(), st["taken"].tolist(), st["path"].tolist()
    src, dst = [], []
    for s, count in enumerate(taken):
        first = lens[s] - (starts[s + 1] - starts[s])
        for j in range(count):
            for p, to in ((first + path[s][j], src), (first + j, dst)):
                to.append(tables[s][p // BLOCK] * BLOCK + p % BLOCK)
    out = []
    for b in st["buffers"]:
        x = b.double()
        rows = x.view(-1, *x.shape[2:])
        rows[dst] = rows[src].clone()
        out.append(x)
    return dict(buffers=out, lens=None)


def exact(case, seed):
    return {"rope": _exact_rope, "tree": _exact_tree, "accept": _exact_accept}[case["op"]](
        prepare(case, seed))
