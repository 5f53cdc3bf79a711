"""The bounded waits of the int8 kernels run out on purpose (pkv_debug_wait_test:
a copy is never started, the wait for it gives up after 20 us): the call
returns with PKV_ERR_TIMEOUT, and the next normal calls are right again.  No
fault, trap or hang is involved."""
import pytest
import torch

from paged_kv_cache_43_gb300 import pkv
from tests.test_gpu_int8 import _lib, attend, batch, wide  # noqa: F401 (the fixture)

pytestmark = pytest.mark.gpu

BATCHES = {
    # q_lens, contexts, decode run, max_context_len
    "split decode": ([1] * 4, [900, 33, 520, 400], 4, 900),
    "team decode": ([1] * 4, [900, 33, 520, 400], 4, 200000),
    "prefill": ([60, 200], [300, 700], 0, 700),
    "prefill in parts": ([60, 20], [2000, 700], 0, 2000),
    "mixed": ([1, 1, 90], [900, 100, 400], 2, 200000),
}


@pytest.mark.parametrize("name", sorted(BATCHES))
def test_waits_run_out_then_the_device_recovers(name):
    q, ctx, nd, bound = BATCHES[name]
    b = batch(ctx, q, 16, 4, 128, seed=17)
    kw = dict(num_decode_seqs=nd, max_context_len=bound, kv_split_tokens=64)
    cache, qs, bt, cl, qsl, scale = b
    pkv.debug_wait_test(True)
    try:
        for _ in range(2):
            out = torch.zeros_like(qs, device="cuda")
            pkv.attention_int8(out, qs.cuda(), *cache.gpu[:2], wide(bt, bound).cuda(), cl.cuda(),
                               qsl.cuda(), scale, *cache.gpu[2:], max_query_len=max(q), **kw)
            torch.cuda.synchronize()
            assert pkv.get_error(clear=True) & pkv.ERR_TIMEOUT
    finally:
        pkv.debug_wait_test(False)
    for _ in range(2):
        got, ref, tol = attend(*b, **kw)
        assert pkv.get_error(clear=True) == 0
        assert (abs(got - ref) <= tol).all()
