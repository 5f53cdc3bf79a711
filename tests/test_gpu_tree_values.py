"""Tree attention over values at the ends of their range: V that is not finite far below the rest, large V with
scores that rise, drafts of K and V that are not finite in every kernel."""
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


def odd(b, what, s, p, h, e, value):
    c = row(b, b.k if what == "k" else b.v, s, p)
    c[h, e] = 0x7F if b.fp8 else value


@pytest.mark.parametrize("dtype", [BF16, E4M3, F32])
@pytest.mark.parametrize("hq,d", [(2, 128), (4, 128), (24, 128), (4, 64)])
@pytest.mark.parametrize("split", [0, 64, 128])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("before", [[50, 330], [0, 1100]])
def test_not_finite_k_of_drafts_reaches_only_rows_that_see_it(dtype, hq, d, split, value, before):
    """Rows that see such a K have scores that are not finite; all others are as without it."""
    if dtype == E4M3 and value == value:
        pytest.skip("e4m3 has no infinity")
    n = [14, 16]
    b = Batch(n, before, hq=hq, hkv=2, d=d, dtype=dtype, seed=6)
    if b.fp8:
        b.k, b.v = (torch.where(torch.isnan(c.float()), 1.0, c.float()).to(dtype) for c in (b.k, b.v))
    clean = b.want()
    seen = torch.zeros(30, dtype=torch.bool)
    for s, draft in ((0, 3), (1, 7), (1, 15)):
        odd(b, "k", s, before[s] + draft, 1, 77 % d, value)
        for i in range(n[s]):
            seen[int(b.starts[s]) + i] |= bool(b.bits[int(b.starts[s]) + i] >> draft & 1)
    b.cuda()
    out = b.call(kv_split_tokens=split).double().cpu()
    ok = (out - clean[0]).abs() <= clean[1]
    half = hq // 2
    assert bool(ok[:, :half].all()) and bool(ok[~seen].all())
    if value != value:   # (an infinite score of either sign: +inf gives NaN, -inf a weight of 0)
        assert bool(torch.isnan(out[seen][:, half:]).all())


@pytest.mark.parametrize("split", [0, 64, 128])
@pytest.mark.parametrize("hq,d", [(2, 128), (8, 64)])
def test_not_finite_v_of_drafts_in_fp32(split, hq, d):
    n, before = [14, 90], [50, 330]
    b = Batch(n, before, hq=hq, hkv=2, d=d, dtype=F32, seed=6)
    seen = torch.zeros(104, dtype=torch.bool)
    for s, draft in ((0, 3), (1, 37), (1, 88)):
        odd(b, "v", s, before[s] + draft, 1, 9, float("nan"))
        odd(b, "v", s, before[s] + draft, 1, 33, float("-inf"))
        for i in range(n[s]):
            seen[int(b.starts[s]) + i] |= bool(b.bits[int(b.starts[s]) + i] >> draft & 1)
    b.cuda()
    out, want = b.call(kv_split_tokens=split), b.want()
    bad = ~torch.isfinite(out.cpu())
    assert torch.equal(bad, ~torch.isfinite(want[0]))
    assert bool(bad[seen][:, hq // 2:].any(2).all())
    b.check(out, want)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("g", [17, 33, 65, 100, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("split", [0, 64])
def test_many_q_heads_a_kv_head(dtype, g, d, split):
    """Row tiles of a few tokens, or one."""
    b = Batch([3, 1, 5, 9], [60, 700, 1, 1400], hq=2 * g, hkv=2, d=d, dtype=dtype, seed=g).cuda()
    b.check(b.call(kv_split_tokens=split))
