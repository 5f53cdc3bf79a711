"""Tree attention in every kernel, chunked prefill, decoding and the rotation at once on streams of their own, one
batch of inputs each: every result is that of the call alone."""
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


def chain(n, before, **kw):
    """A batch whose masks are causal, and the same through the other attention call."""
    b = Batch(n, before, masks=[(2 << i) - 1 for k in n for i in range(k)], **kw).cuda()
    g = b.g

    def call(out):
        pkv.attention(out, g["q"], g["k"], g["v"], g["bt"], g["cl"], g["qsl"], b.scale,
                      max_query_len=b.max_n, max_context_len=b.max_L)
    return b, call


def test_calls_beside_each_other():
    work = []
    for seed, (n, before, hq, d, dtype) in enumerate([
            ([40, 64], [3000, 1500], 16, 64, BF16), ([64, 30], [2500, 700], 16, 128, BF16), ([8] * 20, [900] * 20, 8, 128, BF16),
            ([4] * 9, [2000] * 9, 8, 128, E4M3), ([50, 9], [1800, 400], 16, 64, E4M3), ([90], [3000], 8, 128, E4M3),
            ([20, 5], [600, 300], 8, 64, F32)]):
        b = Batch(n, before, hq=hq, hkv=2, d=d, dtype=dtype, seed=seed).cuda()
        work.append((b, lambda out, b=b: b.call(out)))
    work.append(chain([300, 200], [500, 40], hq=16, hkv=2, d=64, seed=20))
    work.append(chain([300, 200], [500, 40], hq=16, hkv=2, d=128, seed=21))
    work.append(chain([1] * 30, [1200] * 30, hq=16, hkv=2, d=128, seed=22))
    outs = [torch.full_like(b.g["q"], float("nan")) for b, _ in work]
    alone = [torch.full_like(o, float("nan")) for o in outs]
    for (b, call), o in zip(work, alone):
        call(o)
        torch.cuda.synchronize()
        b.check(o)
    streams = [torch.cuda.Stream() for _ in work]
    torch.cuda.synchronize()
    for turn in range(15):
        for o in outs:
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        for i in range(len(work)):
            j = (i + turn) % len(work)
            with torch.cuda.stream(streams[j]):
                work[j][1](outs[j])
                work[j][1](outs[j])
        torch.cuda.synchronize()
        assert pkv.get_error() == 0
        for o, a in zip(outs, alone):
            assert torch.equal(o.view(torch.uint8), a.view(torch.uint8))
