"""pkv_copy_blocks on the GPU against the same copies made one after the other
in numpy: bit for bit, whatever the pairs' order and dependences."""
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


def run(shapes, pairs, seed=0, stream=None):
    """shapes: (dtype, page shape) of each buffer; all of nb blocks."""
    rng = np.random.default_rng(seed)
    host = [rng.integers(0, 256, nb_page, dtype=np.uint8) for nb_page in shapes]
    dev = [torch.from_numpy(h.copy()).cuda() for h in host]
    pkv.copy_blocks(dev, pairs, stream=stream)
    for h in host:
        for a, b in pairs:
            h[b] = h[a]
    torch.cuda.synchronize()
    for d, h in zip(dev, host):
        assert np.array_equal(d.cpu().numpy(), h)


PAGES = [4, 12, 32, 64, 100, 512, 4096, 8192, 8208, 16384, 16400, 32768, 50000]


@pytest.mark.parametrize("page", PAGES)
@pytest.mark.parametrize("n", [1, 2, 15, 511, 512, 513])
def test_disjoint_pairs(page, n):
    ids = np.random.default_rng(n).permutation(2 * n + 3)
    run([(2 * n + 3, page)], np.stack([ids[:n], ids[n:2 * n]], 1))


@pytest.mark.parametrize("seed", range(6))
def test_random_pairs_in_order(seed):
    """Chains, swaps, overwrites, a block onto itself: as if one by one."""
    rng = np.random.default_rng(seed)
    nb = int(rng.integers(2, 40))
    run([(nb, 48), (nb, 16384 + 16)], rng.integers(0, nb, (int(rng.integers(1, 120)), 2)), seed)


def test_many_buffers_of_different_pages():
    """More buffers than one launch takes, every page size in turn."""
    ids = np.random.default_rng(1).permutation(90)
    shapes = [(90, PAGES[i % len(PAGES)]) for i in range(131)]
    run(shapes, np.stack([ids[:40], ids[40:80]], 1))


def test_unaligned_base_takes_the_word_path():
    x = torch.arange(1 + 10 * 32, dtype=torch.int32, device="cuda")
    buf = x[1:].view(10, 32)               # 4-byte aligned, 128-byte pages
    want = buf.clone()
    want[3] = want[7]
    pkv.copy_blocks([buf], [(7, 3)])
    assert torch.equal(buf, want) and int(x[0]) == 0


def test_pages_past_32_bits():
    nb, page = 300000, 16384
    buf = torch.zeros((nb, page), dtype=torch.uint8, device="cuda")
    buf[nb - 1] = 7
    buf[1] = 9
    pkv.copy_blocks([buf], [(nb - 1, 0), (1, nb - 2)])
    assert (buf[0] == 7).all() and (buf[nb - 2] == 9).all()
    assert int(buf[2:nb - 2].max()) == 0


def test_nothing_to_do_and_tensors_of_any_type():
    a = torch.randn(6, 16, 2, 64, device="cuda").to(torch.bfloat16)
    s = torch.randn(6, 2, device="cuda")
    before = a.clone()
    pkv.copy_blocks([a, s], np.zeros((0, 2), np.int32))
    pkv.copy_blocks([], [(0, 1)])
    pkv.copy_blocks([a, s], [(2, 2)])
    assert torch.equal(a, before)
    want = s.clone()
    want[5] = s[0]
    pkv.copy_blocks([a, s], [(0, 5)])
    assert torch.equal(a[5], before[0]) and torch.equal(s, want)


def test_other_stream_and_graph():
    stream = torch.cuda.Stream()
    buf = torch.randn(8, 5000, device="cuda")
    stream.wait_stream(torch.cuda.current_stream())
    pkv.copy_blocks([buf], [(0, 1)], stream=stream)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        pkv.copy_blocks([buf], [(2, 3), (3, 4)], stream=stream)
    buf[2] = 42.0
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert (buf[2:5] == 42.0).all() and torch.equal(buf[0], buf[1])
