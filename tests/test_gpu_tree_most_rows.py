"""Tree attention, sequences of more drafts than the stated most: their first max_query_len rows are zero, and
the rows behind those stay as they were."""
import pytest
import torch

from drafts import Batch, mask_words
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


@pytest.mark.parametrize("dtype", [BF16, E4M3, F32])
@pytest.mark.parametrize("hq,d", [(2, 128), (4, 64), (24, 128)])
def test_rows_behind_the_stated_most_stay(dtype, hq, d):
    b = Batch([3, 20, 5], [40, 50, 9], hq=hq, hkv=2, d=d, dtype=dtype).cuda()
    want, tol = b.want()
    out = b.call(max_query_len=8)
    assert pkv.get_error() == pkv.ERR_QUERY_LEN
    assert bool((out[3:11] == 0).all())
    assert bool(torch.isnan(out[11:23]).all())
    got = out.double().cpu()
    for rows in (slice(0, 3), slice(23, 28)):
        # (e4m3: a few of the random K and V are past 448 and NaN; the reference has them)
        same = torch.isnan(got[rows]) & torch.isnan(want[rows])
        assert bool((same | ((got[rows] - want[rows]).abs() <= tol[rows])).all())


@pytest.mark.parametrize("dtype", [BF16, E4M3, F32])
@pytest.mark.parametrize("hq,d", [(2, 128), (8, 64), (24, 128)])
@pytest.mark.parametrize("most", [33, 200, 5000])
@pytest.mark.parametrize("split", [0, 64])
def test_far_fewer_drafts_than_the_stated_most(dtype, hq, d, most, split):
    """Masks, tiles and workers are made for `most` rows; the sequences have 1 to 17."""
    if split and most == 5000:
        pytest.skip("that many parts of 64 keys for that many rows: a workspace of many GB")
    b = Batch([1, 17, 0, 4, 2], [1200, 333, 9, 0, 2500], hq=hq, hkv=2, d=d, dtype=dtype, seed=most).cuda()
    b.g["mask"] = mask_words(b.bits, -(-most // 64)).cuda()
    b.check(b.call(max_query_len=most, kv_split_tokens=split))
