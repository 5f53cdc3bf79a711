"""pkv_accept_drafts against the same moves in numpy: bit for bit."""
import numpy as np
import pytest
import torch

from paged_kv_cache_43_gb300 import build, pkv

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


class Drafts:
    def __init__(self, n, before, rows=((32,), (2, 64)), dtype=np.uint16, seed=0, most=None,
                 counts=None):
        rng = np.random.default_rng(seed)
        self.n, self.L = np.array(n), np.array(n) + np.array(before)
        nblk = [-(-x // 16) for x in self.L]
        nb = sum(nblk) + 3
        ids = rng.permutation(nb)[:sum(nblk)]
        self.bt = np.full((len(n), max(max(nblk), 1)), -1, np.int32)
        at = 0
        for s, b in enumerate(nblk):
            self.bt[s, :b] = ids[at:at + b]
            at += b
        self.bufs = [rng.integers(0, 60000, (nb, 16, *r)).astype(dtype) for r in rows]
        most = most or max(max(n), 1)
        self.path = np.full((len(n), most), -7, np.int32)
        self.count = np.zeros(len(n), np.int32)
        for s, k in enumerate(n):
            c = int(rng.integers(0, min(k, most) + 1)) if counts is None else counts[s]
            self.path[s, :c] = np.sort(rng.permutation(k)[:c])
            self.count[s] = c

    def want(self, skip=()):
        out = [b.copy() for b in self.bufs]
        new = self.L.astype(np.int32).copy()
        for s, (n, L) in enumerate(zip(self.n, self.L)):
            if s in skip:
                continue
            slot = lambda p: (self.bt[s, p // 16], p % 16)
            for b, o in zip(self.bufs, out):
                for j in range(self.count[s]):
                    o[slot(L - n + j)] = b[slot(L - n + self.path[s, j])]
            new[s] = L - n + self.count[s]
        return out, new

    def cuda(self):
        t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
        self.g = dict(bufs=[t(b) for b in self.bufs], bt=t(self.bt), cl=t(self.L.astype(np.int32)),
                      qsl=t(np.concatenate([[0], np.cumsum(self.n)]).astype(np.int32)),
                      path=t(self.path), count=t(self.count))
        self.g["new"] = torch.full_like(self.g["cl"], -1)
        return self

    def call(self, **kw):
        g = self.g
        pkv.accept_drafts(g["bufs"], g["bt"], g["cl"], g["qsl"], g["path"], g["count"],
                          new_context_lens=g["new"], **kw)

    def check(self, skip=()):
        want, new = self.want(skip)
        for d, h in zip(self.g["bufs"], want):
            assert np.array_equal(d.cpu().numpy(), h)
        assert np.array_equal(self.g["new"].cpu().numpy(), new)


@pytest.mark.parametrize("seed", range(6))
def test_random_paths(seed):
    rng = np.random.default_rng(seed)
    n = rng.integers(0, 70, 20)
    d = Drafts(n, rng.integers(0, 100, 20), seed=seed).cuda()
    d.call()
    d.check()


@pytest.mark.parametrize("row,dtype", [((1,), np.float32), ((3,), np.float32), ((8,), np.uint16),
                                       ((5, 64), np.uint8), ((32, 128), np.uint16),
                                       ((32, 128), np.float32), ((20,), np.uint8)])
def test_row_sizes(row, dtype):
    d = Drafts([30, 9, 1], [100, 3, 15], rows=(row,), dtype=dtype).cuda()
    d.call()
    d.check()


@pytest.mark.parametrize("count", [0, 1, 7, 8, 9, 17, 64])
def test_path_lengths(count):
    d = Drafts([64, 64], [5, 40], counts=[count, count]).cuda()
    d.call()
    d.check()


def test_a_chain_stays_and_the_last_drafts_move_far():
    d = Drafts([40, 40], [10, 23], counts=[40, 8])
    d.path[1, :8] = np.arange(32, 40)
    d.cuda().call()
    d.check()


def test_many_buffers_and_sequences():
    rng = np.random.default_rng(0)
    d = Drafts(rng.integers(1, 9, 300), rng.integers(0, 30, 300), rows=((8,),) * 131, most=4).cuda()
    d.call()
    d.check()


def test_no_buffers_makes_the_lengths():
    d = Drafts([5, 3], [10, 2], rows=(), counts=[3, 2]).cuda()
    d.call()
    d.check()
    assert pkv.get_error() == 0


def test_bad_paths_and_lengths_leave_their_sequence_alone():
    base = dict(n=[6, 6, 6], before=[20, 30, 40], counts=[3, 3, 3])
    for change, bit in ((lambda g: g["path"][1, :3].copy_(torch.tensor([1, 1, 4])), pkv.ERR_ACCEPTED),
                        (lambda g: g["path"][1, :3].copy_(torch.tensor([4, 2, 5])), pkv.ERR_ACCEPTED),
                        (lambda g: g["path"][1, :3].copy_(torch.tensor([0, 1, 6])), pkv.ERR_ACCEPTED),
                        (lambda g: g["path"][1, :3].copy_(torch.tensor([-1, 1, 2])), pkv.ERR_ACCEPTED),
                        (lambda g: g["count"][1].fill_(7), pkv.ERR_ACCEPTED),
                        (lambda g: g["count"][1].fill_(-1), pkv.ERR_ACCEPTED),
                        (lambda g: g["cl"][1].fill_(5), pkv.ERR_QUERY_LEN),
                        (lambda g: g["cl"][1].fill_(10 ** 6), pkv.ERR_CONTEXT_LEN)):
        d = Drafts(**base).cuda()
        change(d.g)
        d.call()
        assert pkv.get_error() == bit
        d.L[1] = int(d.g["cl"][1])
        d.check(skip=(1,))


def test_bad_block_ids_leave_their_rows():
    d = Drafts([20, 6], [20, 30], counts=[0, 3])
    d.path[0, :2], d.count[0] = [5, 14], 2          # rows 25, 34 to 20, 21; row 34 in block 2
    d.cuda()
    d.g["bt"][0, 2] = d.bufs[0].shape[0]
    d.call()
    assert pkv.get_error() == pkv.ERR_BLOCK_ID
    d.count[0] = 1
    want, new = d.want()
    new[0] += 1
    for x, h in zip(d.g["bufs"], want):
        assert np.array_equal(x.cpu().numpy(), h)
    assert np.array_equal(d.g["new"].cpu().numpy(), new)


def test_graph_replay_and_stream():
    d = Drafts([30, 9], [100, 3], counts=[5, 2]).cuda()
    keep = [b.clone() for b in d.g["bufs"]]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    d.call(stream=s)
    s.synchronize()
    d.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        d.call()
    for b, k in zip(d.g["bufs"], keep):
        b.copy_(k)
    d.path[0, :5] = [2, 3, 11, 20, 29]              # another path in the captured call
    d.g["path"].copy_(torch.from_numpy(d.path))
    g.replay()
    torch.cuda.synchronize()
    d.check()


def test_offsets_past_32_bits():
    nb = (1 << 31) // (16 * 1024) + 20
    b = torch.zeros((nb, 16, 1024), dtype=torch.bfloat16, device="cuda")
    bt = torch.tensor([[nb - 1, 3, nb - 5]], dtype=torch.int32, device="cuda")
    b[nb - 5, 2] = 1.5
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    pkv.accept_drafts([b], bt, i(40), i(0, 30), i(24)[None], i(1))
    assert bool((b[nb - 1, 10] == 1.5).all()) and float(b.sum(dtype=torch.float64)) == 2 * 1.5 * 1024


def test_refusals_of_gpu_tensors():
    d = Drafts([6], [20], counts=[3]).cuda()
    g = d.g
    args = dict(bufs=g["bufs"], bt=g["bt"], cl=g["cl"], qsl=g["qsl"], path=g["path"],
                count=g["count"])
    for bad in (dict(path=g["path"][0]), dict(count=g["count"].long()), dict(qsl=g["qsl"][:1]),
                dict(bufs=[g["bufs"][0], g["bufs"][1][:2]]), dict(bufs=[g["bufs"][0].to(torch.int8)]),
                dict(bufs=[g["bufs"][0][:, :8]]), dict(bufs=[g["bufs"][0].cpu()])):
        with pytest.raises(pkv.PkvError):
            pkv.accept_drafts(*{**args, **bad}.values())
    with pytest.raises(pkv.PkvError):
        pkv.accept_drafts(*args.values(), new_context_lens=g["cl"])
