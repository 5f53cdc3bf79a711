"""Tree attention where the batch on the device differs from what the plan was made for: contexts far
shorter than max_context_len, sequences of more drafts than max_query_len, workspaces that hold anything."""
import pytest
import torch

from drafts import Batch
from paged_kv_cache_43_gb300 import build, pkv

pytestmark = pytest.mark.gpu
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    pkv.load()
    pkv.get_error(clear=True)
    yield
    assert pkv.get_error(clear=True) == 0


def call_with(b, fill, **kw):
    """A call whose workspace holds `fill` bytes before it (0xFF: every float a NaN)."""
    kw = dict(dict(max_query_len=b.max_n, max_context_len=b.max_L), **kw)
    meta = pkv.attn_meta(b.g["q"], b.g["bt"], b.g["cl"], **kw)
    ws = torch.full((pkv.workspace_size_tree(b.g["k"], meta) + 256,), fill, dtype=torch.uint8,
                    device="cuda")
    return b.call(workspace=ws, **kw)


@pytest.mark.parametrize("dtype", [BF16, E4M3, F32])
@pytest.mark.parametrize("n,hq,hkv,d", [(4, 8, 8, 128), (16, 2, 1, 128), (40, 8, 8, 128), (9, 16, 8, 64)])
@pytest.mark.parametrize("L", [[40], [100], [500], [1100], [2000], [70, 1300]])
def test_contexts_far_shorter_than_the_stated_most(dtype, n, hq, hkv, d, L):
    """The plan's workers are more than such contexts have steps of work."""
    b = Batch([n] * len(L), [x - n for x in L], hq=hq, hkv=hkv, d=d, dtype=dtype, seed=n + L[0]).cuda()
    want = b.want()
    for most in (1500, 20000, 131072):
        if most < max(L):
            continue
        for fill in (0xFF, 0x3F):
            b.check(call_with(b, fill, max_context_len=most), want)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_one_graph_over_growing_contexts(dtype):
    """A call captured once for long contexts, replayed while they grow from a few keys."""
    b = Batch([8, 8], [3992, 1992], hq=16, hkv=4, d=128, dtype=dtype, seed=3).cuda()
    out = b.call(max_context_len=4000)
    torch.cuda.synchronize()
    meta = pkv.attn_meta(b.g["q"], b.g["bt"], b.g["cl"], max_query_len=8, max_context_len=4000)
    ws = torch.full((pkv.workspace_size_tree(b.g["k"], meta),), 0xFF, dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.call(out, workspace=ws, max_context_len=4000)
    for L in ([8, 9], [33, 8], [129, 300], [640, 128], [1000, 1001], [4000, 2000]):
        b.L = L
        b.g["cl"].copy_(torch.tensor(L, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        b.check(out)
        ws.fill_(0xFF)


@pytest.mark.parametrize("dtype", [BF16, E4M3, F32])
@pytest.mark.parametrize("n,hq,d", [(8, 16, 128), (64, 8, 128), (30, 4, 64)])
def test_a_call_repeats_itself_bit_for_bit(dtype, n, hq, d):
    b = Batch([n, 3, n], [1500, 90, 5000], hq=hq, hkv=2, d=d, dtype=dtype, seed=n).cuda()
    first = call_with(b, 0xFF)
    for fill in (0, 0x3F, 0xFF):
        assert torch.equal(call_with(b, fill).view(torch.uint8), first.view(torch.uint8))
