"""Batches of drafted tokens over a paged cache, and plain 64-bit forms of what the
drafted-step calls compute, with the bounds their results are held to."""
import numpy as np
import torch

BLOCK = 16
EPS = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # half a step, relative


def ancestors(rng, n, back=6):
    """Mask rows (python ints) of a random tree of n drafts in topological order."""
    seen = []
    for i in range(n):
        p = int(rng.integers(max(-1, i - back), i)) if i else -1
        seen.append((seen[p] if p >= 0 else 0) | 1 << i)
    return seen


def mask_words(rows, words):
    out = np.zeros((len(rows), words), np.uint64)
    for t, b in enumerate(rows):
        for w in range(words):
            out[t, w] = b >> 64 * w & (1 << 64) - 1
    return torch.from_numpy(out.view(np.int64))


class Batch:
    """n drafts behind `before` keys for each sequence; every cache row that no key is in
    holds NaN."""

    def __init__(self, n, before, *, hq, hkv, d, dtype=torch.bfloat16, seed=0, masks=None,
                 extra_rows=0, blocks=None):
        self.rng = rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        randn = lambda *s: torch.randn(s, generator=g)
        self.n, self.L = list(n), [a + b for a, b in zip(n, before)]
        self.hq, self.hkv, self.d, self.dtype = hq, hkv, d, dtype
        self.fp8 = dtype == torch.float8_e4m3fn
        self.row = torch.bfloat16 if self.fp8 else dtype
        nblk = [-(-x // BLOCK) for x in self.L]
        nb = blocks or sum(nblk) + 5
        ids = rng.permutation(nb)[:sum(nblk)]
        self.table = np.full((len(n), max(max(nblk), 1)), -1, np.int32)
        at = 0
        for s, b in enumerate(nblk):
            self.table[s, :b] = ids[at:at + b]
            at += b
        self.starts = np.concatenate([[0], np.cumsum(self.n)]).astype(np.int32)
        self.tokens = int(self.starts[-1]) + extra_rows
        self.max_n, self.max_L = max(max(self.n), 1), max(max(self.L), 1)
        rows = masks if masks is not None else [b for k in self.n for b in ancestors(rng, k)]
        self.bits = list(rows) + [0] * extra_rows
        self.k = torch.full((nb, BLOCK, hkv, d), float("nan"))
        self.v = self.k.clone()
        for s, L in enumerate(self.L):
            for c in (self.k, self.v):
                x = randn(L, hkv, d)
                for b in range(nblk[s]):
                    e = min(BLOCK, L - b * BLOCK)
                    c[self.table[s, b], :e] = x[b * BLOCK:b * BLOCK + e]
        self.q = randn(self.tokens, hq, d).to(self.row)
        if self.fp8:
            self.k, self.v = ((c * 100).to(dtype) for c in (self.k, self.v))
            self.kd, self.vd = (0.01 * torch.rand(len(n), hkv, generator=g) + 0.005
                                for _ in range(2))
        else:
            self.k, self.v = self.k.to(dtype), self.v.to(dtype)
        self.scale = d ** -0.5

    def cuda(self):
        t = torch.from_numpy
        self.g = dict(q=self.q.cuda(), k=self.k.cuda(), v=self.v.cuda(), bt=t(self.table).cuda(),
                      cl=torch.tensor(self.L, dtype=torch.int32).cuda(),
                      qsl=t(self.starts).cuda(),
                      mask=mask_words(self.bits, -(-self.max_n // 64)).cuda())
        if self.fp8:
            self.g.update(kd=self.kd.cuda(), vd=self.vd.cuda())
        return self

    def call(self, out=None, **kw):
        from paged_kv_cache_43_gb300 import pkv
        g = self.g
        out = torch.full_like(g["q"], float("nan")) if out is None else out
        args = (out, g["q"], g["k"], g["v"], g["bt"], g["cl"], g["qsl"], g["mask"], self.scale)
        kw = dict(dict(max_query_len=self.max_n, max_context_len=self.max_L), **kw)
        if self.fp8:
            pkv.attention_tree_fp8(*args, g["kd"], g["vd"], **kw)
        else:
            pkv.attention_tree(*args, **kw)
        return out

    def keys(self, s, h):
        """K and V of a sequence's kv head in 64 bits [L, d]."""
        L = self.L[s]
        at = torch.from_numpy(self.table[s, :-(-L // BLOCK)]).long()
        k, v = (c.view(torch.uint8)[at, :, h].view(c.dtype) if self.fp8 else c[at, :, h]
                for c in (self.k, self.v))
        k, v = (x.double().flatten(0, 1)[:L] for x in (k, v))
        return (k * self.kd[s, h].double(), v * self.vd[s, h].double()) if self.fp8 else (k, v)

    def want(self):
        """(out [T, hq, d] in 64 bits, bound on |error|); rows of no sequence are NaN."""
        G = self.hq // self.hkv
        out = torch.full((self.tokens, self.hq, self.d), float("nan"), dtype=torch.float64)
        tol = torch.zeros_like(out)
        # weights: rounded to the V operand's type, and formed from scores that are off by
        # their sums' roundings (d products) and the exponential's
        w_eps = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8}.get(self.dtype, 2.0 ** -11)
        for s, n in enumerate(self.n):
            if not n:
                continue
            L, t0 = self.L[s], int(self.starts[s])
            seen = torch.ones(n, L, dtype=torch.bool)
            for i in range(n):
                for j in range(n):
                    seen[i, L - n + j] = bool(self.bits[t0 + i] >> j & 1)
            for h in range(self.hkv):
                k, v = self.keys(s, h)
                k, v = k.cuda(), v.cuda()
                sn = seen.cuda()
                for g in range(G):
                    q = self.q[t0:t0 + n, h * G + g].double().cuda()
                    x = (q @ k.T * self.scale).masked_fill(~sn, float("-inf"))
                    p = torch.softmax(x, -1)
                    p = torch.where(sn, p, 0.0)
                    p[~sn.any(1)] = 0.0
                    # (a key that is not seen does not reach the sum, whatever it holds)
                    v0 = torch.where(torch.isfinite(v), v, 0.0)
                    o = p @ v0
                    for i, j in torch.nonzero(sn & ~torch.isfinite(v).all(1)).tolist():
                        o[i] += p[i, j] * (v[j] - v0[j])
                    spread = torch.stack([(p[i, :, None] * (v0 - o[i]).abs()).sum(0)
                                          for i in range(n)])
                    if self.fp8:   # (the denominator sums the weights before they are rounded)
                        spread = p @ v0.abs() + o.abs()
                    size = (q.abs() @ torch.nan_to_num(k, 0, 0, 0).abs().T * abs(self.scale))
                    w = w_eps * 1.01 + 2.0 ** -20 + self.d * 2.0 ** -23 * size.amax(1, keepdim=True)
                    # The numerator and the denominator are fp32 sums of L terms: each product
                    # and partial sum is rounded once, so they are off by at most L 2^-24 of
                    # sum p |V| and of sum p = 1 (which moves the output by that share of |o| <=
                    # sum p |V|); normalising is two roundings more, merging splits four.
                    sums = (2 * L + 6) * 2.0 ** -24 * (p @ v0.abs())
                    out[t0:t0 + n, h * G + g] = o.cpu()
                    tol[t0:t0 + n, h * G + g] = (EPS[self.row] * o.abs() + w * spread + sums).cpu()
        return out, tol + 1e-30

    def check(self, out, want=None):
        want, tol = want or self.want()
        got = out.double().cpu()
        rows = slice(0, int(self.starts[-1]))
        same = (got == want) | (torch.isnan(got) & torch.isnan(want))
        ok = same | ((got - want).abs() <= tol)
        assert bool(ok[rows].all()), (
            f"{int((~ok[rows]).sum())} values off, worst "
            f"{float(torch.nan_to_num(((got - want).abs() / tol)[rows], 1e9).max()):.2f} of the bound")


def drafted(seq_lens, seed=0):
    """Random (n, before) of sequences whose keys number `seq_lens`."""
    rng = np.random.default_rng(seed)
    n = [int(rng.integers(1, min(L, 40) + 1)) for L in seq_lens]
    return n, [L - k for L, k in zip(seq_lens, n)]


def rope_reference(x, weight, eps, table, positions, interleaved):
    """(rows in 64 bits, bound on the fp32 arithmetic's error)."""
    x = x.double()
    if weight is not None:
        x = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt() * weight.double()
    half = table.shape[1] // 2
    c, s = table.double()[positions].split(half, 1) if half else (None, None)
    y, size = x.clone(), x.abs()
    if half:
        first = slice(0, 2 * half, 2) if interleaved else slice(0, half)
        second = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
        a, b = x[..., first], x[..., second]
        c, s = c[:, None], s[:, None]
        y[..., first], y[..., second] = a * c - b * s, b * c + a * s
        size[..., first] = size[..., second] = a.abs() + b.abs()
    # the norm's sum, root, and products: under 16 roundings; the rotation's: three
    return y, size * 2.0 ** -19
