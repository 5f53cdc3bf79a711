"""pkv_accept_drafts over paths of more drafts than a CTA looks up at a time (64), and than it has threads
(256): bit for bit against the same moves in numpy."""
import numpy as np
import pytest
import torch

from paged_kv_cache_43_gb300 import build, pkv

pytestmark = pytest.mark.gpu
N = 400


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    pkv.load()
    pkv.get_error(clear=True)
    yield
    assert pkv.get_error(clear=True) == 0


def paths(kind, count, rng):
    if kind == "last":                      # every row moves, across the chunks' limits
        return np.arange(N - count, N)
    if kind == "every other":
        return np.arange(count) * (N // max(count, 1)) + (N // max(count, 1) - 1)
    return np.sort(rng.permutation(N)[:count])


def setup(rows, counts, kind, before=(37, 5), seed=0):
    rng = np.random.default_rng(seed)
    L = [N + b for b in before]
    nblk = [-(-x // 16) for x in L]
    ids = rng.permutation(sum(nblk) + 3)[:sum(nblk)]
    bt = np.full((len(L), max(nblk)), -1, np.int32)
    bt[0, :nblk[0]], bt[1, :nblk[1]] = ids[:nblk[0]], ids[nblk[0]:]
    bufs = [rng.integers(0, 2 ** 31, (sum(nblk) + 3, 16, r)).astype(np.int32).view(np.float32) for r in rows]
    path = np.full((len(L), N), -9, np.int32)
    for s, c in enumerate(counts):
        path[s, :c] = paths(kind, c, rng)
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
    dev = dict(bufs=[t(b.view(np.int32)).view(torch.float32) for b in bufs], bt=t(bt), cl=t(np.array(L, np.int32)),
               qsl=t(np.arange(len(L) + 1, dtype=np.int32) * N), path=t(path),
               count=t(np.array(counts, np.int32)))
    dev["new"] = torch.full_like(dev["cl"], -1)
    return bufs, bt, L, path, dev


def moved(bufs, bt, L, path, counts):
    out = [b.copy() for b in bufs]
    for s, c in enumerate(counts):
        at = lambda p: (bt[s, p // 16], p % 16)
        for b, o in zip(bufs, out):
            for j in range(c):
                o.view(np.int32)[at(L[s] - N + j)] = b.view(np.int32)[at(L[s] - N + path[s, j])]
    return out


def run(dev):
    pkv.accept_drafts(dev["bufs"], dev["bt"], dev["cl"], dev["qsl"], dev["path"], dev["count"],
                      new_context_lens=dev["new"])


def same(dev, want, lens):
    for d, h in zip(dev["bufs"], want):
        assert np.array_equal(d.view(torch.int32).cpu().numpy(), h.view(np.int32))
    assert dev["new"].tolist() == lens


@pytest.mark.parametrize("count", [63, 64, 65, 127, 128, 129, 200, 256, 257, 300, 400])
@pytest.mark.parametrize("rows", [(64, 8), (1, 3), (512, 64, 4, 4, 1024, 3)])
@pytest.mark.parametrize("kind", ["random", "last", "every other"])
def test_long_paths(count, rows, kind):
    counts = [count, max(count - 30, 0)]
    bufs, bt, L, path, dev = setup(rows, counts, kind, seed=count)
    run(dev)
    same(dev, moved(bufs, bt, L, path, counts), [x - N + c for x, c in zip(L, counts)])


@pytest.mark.parametrize("at", [64, 255, 256, 257, 299])
@pytest.mark.parametrize("bad", ["equal", "past", "negative"])
def test_a_bad_entry_far_down_the_path(at, bad):
    counts = [300, 300]
    bufs, bt, L, path, dev = setup((8, 3), counts, "random")
    dev["path"][0, at] = {"equal": int(path[0, at - 1]), "past": N, "negative": -1}[bad]
    run(dev)
    assert pkv.get_error() == pkv.ERR_ACCEPTED
    same(dev, moved(bufs, bt, L, path, [0, 300]), [L[0], L[1] - N + 300])


def test_a_bad_block_far_down_the_path_keeps_its_rows():
    counts = [300, 300]
    bufs, bt, L, path, dev = setup((8, 3), counts, "last", before=(32, 48))
    dev["bt"][0, 2 + 200 // 16] = -5          # holds the places of drafts 192 .. 207 of the first sequence
    run(dev)
    assert pkv.get_error() == pkv.ERR_BLOCK_ID
    want = moved(bufs, bt, L, path, counts)
    still = moved(bufs, bt, L, path, [0, 300])
    gone = [j for j in range(300) if 192 <= j < 208 or 192 <= path[0, j] < 208]
    for w, b in zip(want, still):
        for j in gone:
            p = L[0] - N + j
            w.view(np.int32)[bt[0, p // 16], p % 16] = b.view(np.int32)[bt[0, p // 16], p % 16]
    same(dev, want, [L[0] - N + 300, L[1] - N + 300])
