"""Timed cases of the block-scaled int8 KV cache and of the page copies.

Three operators of a paged cache [num_blocks, 16, kv heads, head size]:

* ``write``: this step's K and V rows into an int8 cache whose scale is one
  fp32 number for each block of 16 tokens and kv head.  With a the largest
  magnitude of the rows a call puts into a block, the block's scale becomes
  s = max(a / 127, 2^-60), or max(s_old, a / 127) where the block already holds
  earlier tokens; if it grows, their codes become rint(code * (s_old / s)); the
  new codes are rint(x * (1 / s)).
* ``attention``: softmax attention of the step's query rows over code * scale,
  causal inside a chunk, with shared kv heads and an optional sliding window.
* ``copy``: whole pages of many buffers from one block to another.

``run`` computes them with elementary torch operations in fp32, or through the
package's calls where ``own`` is true.
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = 16
FLOOR = 2.0 ** -60


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one sequence of a quiet server writes the token it has just made
        dict(name="write decode 1", op="write", decode=1, lo=100, hi=100, log=False, chunks=0,
             chunk=0, hkv=8, d=128, lens=1),
        # a decode step of 256 sequences, one token each, at every offset of their last blocks
        dict(name="write decode 256", op="write", decode=256, lo=64, hi=8192, log=True, chunks=0,
             chunk=0, hkv=8, d=128, lens=2),
        # prompts in chunks that begin and end inside blocks, beside a few decodes; 5 kv heads of 64
        dict(name="write chunks", op="write", decode=33, lo=17, hi=900, log=False, chunks=7,
             chunk=2047, hkv=5, d=64, lens=3),
        # the same quiet server's attention: latency alone counts
        dict(name="decode 1", op="attention", decode=1, lo=100, hi=100, log=False, chunks=0,
             chunk=0, hq=32, hkv=8, d=128, window=0, lens=4),
        # the default decode batch: 64 sequences, a kv head for every query head
        dict(name="decode 64 x 32 heads", op="attention", decode=64, lo=128, hi=4096, log=False,
             chunks=0, chunk=0, hq=32, hkv=32, d=128, window=0, lens=5),
        # a busy server: many sequences of very different lengths, 4 query heads on a kv head
        dict(name="decode 256 grouped", op="attention", decode=256, lo=64, hi=8192, log=True,
             chunks=0, chunk=0, hq=32, hkv=8, d=128, window=0, lens=6),
        # long documents: few sequences, 16K to 32K keys, 8 query heads on a kv head
        dict(name="decode 16 long", op="attention", decode=16, lo=16384, hi=32768, log=False,
             chunks=0, chunk=0, hq=64, hkv=8, d=128, window=0, lens=7),
        # a step of chunked prefill: 48 decodes and 4 chunks of 512 tokens in one call
        dict(name="mixed 48 + 4 x 512", op="attention", decode=48, lo=256, hi=4096, log=False,
             chunks=4, chunk=512, hq=32, hkv=8, d=128, window=0, lens=8),
        # prompts alone: 4 chunks of 2048 tokens over 2K to 8K keys
        dict(name="prefill 4 x 2048", op="attention", decode=0, lo=2048, hi=8192, log=False,
             chunks=4, chunk=2048, hq=32, hkv=8, d=128, window=0, lens=9),
        # a sliding window, 3 query heads on a kv head of 64, ragged lengths
        dict(name="window ragged", op="attention", decode=37, lo=1, hi=5000, log=True, chunks=3,
             chunk=333, hq=12, hkv=4, d=64, window=1000, lens=10),
        # a fork's last blocks: 16 pages of one layer's bf16 cache
        dict(name="copy fork", op="copy", pairs=16, layers=1, blocks=256, hkv=8, d=128,
             int8=False),
        # a pool made smaller: 512 pages of 16 layers' int8 caches, with their scales
        dict(name="copy compact", op="copy", pairs=512, layers=16, blocks=1200, hkv=8, d=128,
             int8=True),
    ]


def _log_int(rng, lo, hi):
    return int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))


def draw(rng):
    op = rng.choice(["write", "attention", "attention", "attention", "copy"])
    d = rng.choice([64, 128, 128])
    if op == "copy":
        layers = _log_int(rng, 1, 16)
        pairs = _log_int(rng, 1, 500)
        return dict(op=op, pairs=pairs, layers=layers, blocks=2 * pairs + rng.randrange(1, 200),
                    hkv=rng.randrange(1, 9), d=d, int8=rng.random() < 0.5)
    lens = rng.randrange(1 << 20)
    if op == "write":
        chunks = rng.choice([0, 0, rng.randrange(1, 8)])
        hi = _log_int(rng, 2, 8192)
        return dict(op=op, decode=_log_int(rng, 1, 256) if not chunks else rng.randrange(0, 40),
                    lo=_log_int(rng, 1, hi), hi=hi, log=rng.random() < 0.5, chunks=chunks,
                    chunk=_log_int(rng, 2, 2000) if chunks else 0, hkv=rng.randrange(1, 9), d=d,
                    lens=lens)
    group = rng.choice([1, 2, 3, 4, 5, 8, 16])
    hkv = rng.choice([1, 2, 3, 4, 8]) if group > 4 else rng.choice([2, 4, 5, 8, 16])
    kind = rng.choice(["decode", "decode", "mixed", "prefill"])
    window = rng.choice([0, 0, 0, _log_int(rng, 1, 4000)])
    if kind == "decode":
        # sequences x longest context x kv heads stays under the listed batches
        hi = _log_int(rng, 16, 20000)
        most = max(1, min(256, (1 << 21) // (hi * hkv)))
        return dict(op=op, decode=_log_int(rng, 1, most), lo=_log_int(rng, 1, hi), hi=hi,
                    log=rng.random() < 0.5, chunks=0, chunk=0, hq=group * hkv, hkv=hkv, d=d,
                    window=window, lens=lens)
    chunks = rng.randrange(1, 5)
    chunk = _log_int(rng, 2, 700 if group * hkv > 32 else 1000)
    hi = _log_int(rng, chunk, 4000)
    return dict(op=op, decode=0 if kind == "prefill" else rng.randrange(1, 40),
                lo=_log_int(rng, 1, hi), hi=hi, log=rng.random() < 0.5, chunks=chunks,
                chunk=chunk, hq=group * hkv, hkv=hkv, d=d, window=window, lens=lens)


def _lengths(case):
    """(new tokens, keys) of each sequence: the decodes, then the chunks."""
    rng = random.Random(case["lens"])
    lo, hi = case["lo"], case["hi"]

    def length():
        if case["log"]:
            return max(lo, min(hi, _log_int(rng, lo, hi)))
        return rng.randint(lo, hi)

    q = [1] * case["decode"] + [case["chunk"]] * case["chunks"]
    return q, [max(length(), n) for n in q]


def _visible_keys(n, length, window):
    """Keys of the cache that some query row of the sequence sees."""
    return length if window <= 0 else min(length, window + n - 1)


def _visible_pairs(n, length, window):
    """(query row, key) pairs that the mask leaves."""
    first, last = length - n + 1, length        # keys that the first and the last row see
    if window <= 0 or window >= last:
        return (first + last) * n // 2
    if window <= first:
        return window * n
    short = window - first                      # rows that see less than the window
    return (first + window - 1) * short // 2 + window * (n - short)


def work(case):
    d, hkv = case["d"], case["hkv"]
    if case["op"] == "copy":
        page = BLOCK * hkv * d * (1 if case["int8"] else 2) + (4 * hkv if case["int8"] else 0)
        return {"bytes": 2 * 2 * case["layers"] * case["pairs"] * page, "flops": 0}
    q, ctx = _lengths(case)
    tokens = sum(q)
    if case["op"] == "write":
        blocks = sum((c - 1) // BLOCK - (c - n) // BLOCK + 1 for n, c in zip(q, ctx))
        # rows in, codes out, the touched blocks' scales in and out, the block ids
        return {"bytes": 2 * tokens * hkv * d * 3 + 2 * blocks * hkv * 8 + 4 * blocks, "flops": 0}
    window, hq = case["window"], case["hq"]
    keys = [_visible_keys(n, c, window) for n, c in zip(q, ctx)]
    blocks = sum(-(-k // BLOCK) for k in keys)
    # codes and scales of the keys in sight, the query rows, the output rows, the block ids
    moved = 2 * hkv * d * sum(keys) + 2 * hkv * 4 * blocks + 2 * tokens * hq * d * 2 + 4 * blocks
    pairs = sum(_visible_pairs(n, c, window) for n, c in zip(q, ctx))
    return {"bytes": moved, "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------ inputs

def _quantise(x):
    """Codes and scales of whole blocks [blocks, 16, heads, d]."""
    top = x.abs().amax((1, 3))
    scale = (top / torch.full_like(top, 127.0)).clamp_min(FLOOR)
    return torch.round(x / scale[:, None, :, None]).clamp(-127, 127).to(torch.int8), scale


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    host = np.random.default_rng(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    hkv, d = case["hkv"], case["d"]
    if case["op"] == "copy":
        nb, n = case["blocks"], case["pairs"]
        ids = host.permutation(nb)[:2 * n].astype(np.int32)
        pairs = np.ascontiguousarray(ids.reshape(2, n).T)      # (from, to), no block twice
        buffers = []
        for _ in range(2 * case["layers"]):
            if case["int8"]:
                buffers.append(torch.randint(-127, 128, (nb, BLOCK, hkv, d), generator=gen,
                                             device=dev, dtype=torch.int8))
            else:
                buffers.append(normal(nb, BLOCK, hkv, d).to(torch.bfloat16))
        if case["int8"]:
            buffers += [normal(nb, hkv).exp() * 0.02 for _ in range(2 * case["layers"])]
        return dict(case=case, buffers=buffers, pairs=pairs)
    q, ctx = _lengths(case)
    tokens, seqs = sum(q), len(q)
    nblk = [-(-c // BLOCK) for c in ctx]
    total = sum(nblk)
    nb = total + total // 10 + 1
    order = host.permutation(nb)[:total].astype(np.int32)
    tables = np.full((seqs, max(nblk)), -1, np.int32)
    at = 0
    for s, n in enumerate(nblk):
        tables[s, :n] = order[at:at + n]
        at += n
    starts = np.concatenate([[0], np.cumsum(q)]).astype(np.int32)
    state = dict(case=case, seqs=seqs, tokens=tokens, max_query_len=max(q),
                 max_context_len=max(ctx), decodes=case["decode"],
                 tables=torch.from_numpy(tables).to(dev),
                 lens=torch.tensor(ctx, dtype=torch.int32, device=dev),
                 starts=torch.from_numpy(starts).to(dev))
    # keys have channels of different size, as projections leave them
    channel = (0.5 * normal(hkv, d)).exp()
    if case["op"] == "write":
        # a cache that holds the earlier tokens, and this step's rows
        history = normal(nb, BLOCK, hkv, d)
        state["k_cache"], state["k_scales"] = _quantise(history * channel * 0.8)
        state["v_cache"], state["v_scales"] = _quantise(history.flip(0) * 0.8)
        state["k"] = (normal(tokens, hkv, d) * channel).to(torch.bfloat16)
        state["v"] = normal(tokens, hkv, d).to(torch.bfloat16)
        return state
    state["k_cache"], state["k_scales"] = _quantise(normal(nb, BLOCK, hkv, d) * channel)
    state["v_cache"], state["v_scales"] = _quantise(normal(nb, BLOCK, hkv, d))
    state["q"] = normal(tokens, case["hq"], d).to(torch.bfloat16)
    state["out"] = torch.empty_like(state["q"])
    state["scale"] = 1.0 / math.sqrt(d)
    return state


# --------------------------------------------------------------- plain forms

def _plain_write(st):
    """The touched blocks gathered, their scales raised, old and new codes rounded, all put back."""
    dev = st["k"].device
    t = torch.arange(st["tokens"], device=dev)
    starts, lens, tables = st["starts"].long(), st["lens"].long(), st["tables"].long()
    seq = torch.searchsorted(starts[1:], t, right=True)
    pos = lens[seq] - (starts[seq + 1] - starts[seq]) + t - starts[seq]
    block, at = torch.unique(tables[seq, pos // BLOCK], return_inverse=True)
    offset = pos % BLOCK
    first = torch.full(block.shape, BLOCK, device=dev).index_reduce_(0, at, offset, "amin")
    old = torch.arange(BLOCK, device=dev) < first[:, None]

    def one(x, cache, scales):
        x, codes, before = x.float(), cache[block], scales[block]
        top = torch.zeros_like(before).index_reduce_(0, at, x.abs().amax(2), "amax")
        want = (top / torch.full_like(top, 127.0)).clamp_min(FLOOR)
        now = torch.where(first[:, None] == 0, want, torch.maximum(want, before))
        ratio = torch.where(old[:, :, None], (before / now)[:, None], 1.0)[..., None]
        codes = torch.where(ratio < 1, torch.round(codes.float() * ratio).to(torch.int8), codes)
        new = torch.round(x * now.reciprocal()[at][:, :, None]).clamp(-127, 127)
        codes[at, offset] = new.to(torch.int8)
        cache[block] = codes
        scales[block] = now

    one(st["k"], st["k_cache"], st["k_scales"])
    one(st["v"], st["v_cache"], st["v_scales"])
    return dict(k_codes=st["k_cache"], v_codes=st["v_cache"], k_scales=st["k_scales"],
                v_scales=st["v_scales"])


def _plain_attention(st):
    """Blocks gathered and widened, sequences padded to the longest, one masked softmax."""
    case = st["case"]
    d, hkv, window = case["d"], case["hkv"], case["window"]
    dev = st["q"].device
    blocks = st["tables"].long().clamp_min(0)

    def gathered(cache, scales):
        x = cache[blocks].float() * scales[blocks][:, :, None, :, None]
        return x.flatten(1, 2)                               # [seqs, keys, kv heads, d]

    k, v = gathered(st["k_cache"], st["k_scales"]), gathered(st["v_cache"], st["v_scales"])
    starts, lens = st["starts"].long(), st["lens"].long()
    n = starts[1:] - starts[:-1]
    j = torch.arange(st["max_query_len"], device=dev)
    rows = (starts[:-1, None] + j).clamp_max(st["tokens"] - 1)
    q = st["q"].float()[rows].unflatten(2, (hkv, -1))        # [seqs, rows, kv heads, group, d]
    pos = (lens - n)[:, None] + torch.minimum(j[None], n[:, None] - 1)
    key = torch.arange(k.shape[1], device=dev)
    hidden = key > pos[:, :, None]
    if window > 0:
        hidden |= key <= pos[:, :, None] - window
    s = torch.einsum("srhgd,skhd->shgrk", q, k) * st["scale"]
    s.masked_fill_(hidden[:, None, None], -math.inf)
    s -= s.amax(-1, keepdim=True)
    s.exp_()
    total = s.sum(-1, keepdim=True)
    v = v.masked_fill((key >= lens[:, None])[:, :, None, None], 0.0)
    o = torch.einsum("shgrk,skhd->shgrd", s, v) / total
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)               # [seqs, rows, query heads, d]
    t = torch.arange(st["tokens"], device=dev)
    seq = torch.searchsorted(starts[1:], t, right=True)
    return o[seq, t - starts[seq]].to(st["q"].dtype)


def _plain_copy(st):
    pairs = torch.from_numpy(st["pairs"]).to(st["buffers"][0].device).long()
    src, dst = pairs[:, 0], pairs[:, 1]
    return [b.index_copy_(0, dst, b.index_select(0, src)) for b in st["buffers"]]


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"write": _plain_write, "attention": _plain_attention, "copy": _plain_copy}[op](state)
    from paged_kv_cache_43_gb300 import pkv
    st = state
    if op == "write":
        pkv.write_int8(st["k"], st["v"], st["tables"], st["lens"], st["starts"], st["k_cache"],
                       st["v_cache"], st["k_scales"], st["v_scales"],
                       max_query_len=st["max_query_len"])
        return dict(k_codes=st["k_cache"], v_codes=st["v_cache"], k_scales=st["k_scales"],
                    v_scales=st["v_scales"])
    if op == "attention":
        pkv.attention_int8(st["out"], st["q"], st["k_cache"], st["v_cache"], st["tables"],
                           st["lens"], st["starts"], st["scale"], st["k_scales"], st["v_scales"],
                           max_query_len=st["max_query_len"],
                           max_context_len=st["max_context_len"], num_decode_seqs=st["decodes"],
                           sliding_window=st["case"]["window"])
        return st["out"]
    pkv.copy_blocks(st["buffers"], st["pairs"])
    return st["buffers"]


# --------------------------------------------------------------- definitions

def _exact_write(st):
    """Scales in 64 bits, block by block; codes are whole numbers and are compared as such."""
    out = {}
    tables, lens, starts = (st[n].cpu().tolist() for n in ("tables", "lens", "starts"))
    for name in ("k", "v"):
        scales = st[name + "_scales"].double()
        rows = st[name].double().abs().amax(2)
        for s in range(st["seqs"]):
            t, end, p = starts[s], starts[s + 1], lens[s] - (starts[s + 1] - starts[s])
            while t < end:
                n = min(BLOCK - p % BLOCK, end - t)
                b = tables[s][p // BLOCK]
                want = (rows[t:t + n].amax(0) / 127.0).clamp_min(FLOOR)
                scales[b] = want if p % BLOCK == 0 else torch.maximum(want, scales[b])
                t, p = t + n, p + n
        out[name + "_scales"] = scales
        out[name + "_codes"] = None
    return out


def _exact_attention(st):
    """Sequence by sequence and kv head by kv head, from the definition."""
    case = st["case"]
    hkv, window = case["hkv"], case["window"]
    group = case["hq"] // hkv
    lens, starts = st["lens"].cpu().tolist(), st["starts"].cpu().tolist()
    out = torch.empty(st["q"].shape, dtype=torch.float64, device=st["q"].device)
    for s in range(st["seqs"]):
        length, t0, t1 = lens[s], starts[s], starts[s + 1]
        at = st["tables"][s, :-(-length // BLOCK)].long()
        row = torch.arange(length - (t1 - t0), length, device=out.device)[:, None]
        key = torch.arange(length, device=out.device)[None]
        seen = (key <= row) & (key > row - window) if window > 0 else key <= row
        for h in range(hkv):
            k = st["k_cache"][at, :, h].double() * st["k_scales"][at, h].double()[:, None, None]
            v = st["v_cache"][at, :, h].double() * st["v_scales"][at, h].double()[:, None, None]
            k, v = k.flatten(0, 1)[:length], v.flatten(0, 1)[:length]
            heads = slice(h * group, (h + 1) * group)
            x = st["q"][t0:t1, heads].double().transpose(0, 1) @ k.T / math.sqrt(case["d"])
            w = torch.softmax(x.masked_fill(~seen, -math.inf), -1)
            out[t0:t1, heads] = (w @ v).transpose(0, 1)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "write":
        return _exact_write(st)
    if case["op"] == "attention":
        return _exact_attention(st)
    out = []
    for b in st["buffers"]:
        if not b.dtype.is_floating_point:
            out.append(None)
            continue
        x = b.double()
        for a, z in st["pairs"].tolist():
            x[z] = b[a].double()
        out.append(x)
    return out
