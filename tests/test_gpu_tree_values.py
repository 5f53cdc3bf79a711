"""Tree attention over values at the ends of their range."""
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


def row(b, c, s, p):
    """Key p's row of sequence s in a cache: [kv heads, d] (codes as bytes)."""
    c = c.view(torch.uint8) if b.fp8 else c
    return c[b.table[s, p // 16], p % 16]


@pytest.mark.parametrize("dtype", [BF16, E4M3, F32])
@pytest.mark.parametrize("n,d", [(6, 128), (40, 128), (20, 64)])
@pytest.mark.parametrize("split", [0, 64, 128, 1024])
def test_not_finite_v_of_a_far_key_is_not_lost(dtype, n, d, split):
    """The first keys score 200 nats below the others: their weights are zero in fp32, not in truth; a NaN
    among their V makes every row NaN or infinite there, however the keys are cut."""
    b = Batch([n], [1500], hq=2, hkv=1, d=d, dtype=dtype, seed=d)
    b.q = (b.q.float() * 0.1 + 3).to(b.row)
    c = 300.0 if b.fp8 else 3.0
    for p in range(b.L[0]):
        x = torch.full((1, d), -c if p < 64 else c).to(dtype)
        row(b, b.k, 0, p).copy_(x.view(torch.uint8) if b.fp8 else x)
    if b.fp8:
        b.kd.fill_(0.01)
        b.v = torch.where(torch.isnan(b.v.float()), 1.0, b.v.float()).to(dtype)
    b.scale = 200.0 / (18 * d)
    row(b, b.v, 0, 5)[0, 7] = 0x7F if b.fp8 else float("nan")
    b.cuda()
    out = b.call(kv_split_tokens=split).float()
    assert not bool(torch.isfinite(out[:, :, 7]).any())
    assert bool(torch.isfinite(out[:, :, :7]).all()) and bool(torch.isfinite(out[:, :, 8:]).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,d", [(6, 128), (40, 128), (20, 64)])
@pytest.mark.parametrize("split", [0, 64, 2048])
@pytest.mark.parametrize("rise", [3.0, 12.0, 35.0])
def test_rising_scores_over_large_v(dtype, n, d, split, rise):
    """V of about 1e25; the last keys' scores lie `rise` nats above the first's, in one step or many."""
    b = Batch([n, n], [1200, 100], hq=2, hkv=1, d=d, dtype=dtype, seed=n)
    b.v = (b.v.float() * 1e25).to(dtype)
    b.q[..., 0] = 8
    for s, L in enumerate(b.L):
        for p in range(L):
            up = rise * (p / L if s == 0 else p >= 70)
            row(b, b.k, s, p)[0, 0] = up / (8 * b.scale)
    b.cuda()
    out = b.call(kv_split_tokens=split)
    assert bool(torch.isfinite(out).all())
    b.check(out)
