"""Stored scales of the int8 cache that no write makes, and scales at the ends
of their range: pkv_write_int8 bit for bit with the oracle, pkv_attention_int8
against the definition in fp64."""
import numpy as np
import pytest
import torch

from paged_kv_cache_43_gb300 import pkv
from tests.test_gpu_int8 import _lib, Cache, attend, batch, i32, rows, starts, tables, wide  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ write

@pytest.mark.parametrize("stored", [np.nan, np.inf, -np.inf, 0.0, -1.0, 2.0 ** -61, 2.0 ** -60])
@pytest.mark.parametrize("n", [1, 3])
@pytest.mark.parametrize("what", ["zero", "tiny", "nan", "ordinary"])
def test_write_replaces_a_stored_scale_that_is_not_one(stored, n, what):
    """A block continued under a scale that is NaN, infinite or below 2^-60: the
    scale in memory is a sound one afterwards, whatever the new rows hold."""
    cache = Cache(3, 2, 64, seed=n)
    for a, g in ((cache.ks, cache.gpu[2]), (cache.vs, cache.gpu[3])):
        a[:] = stored
        g.fill_(float(stored))
    gen = torch.Generator().manual_seed(5)
    k, v = rows(gen, 2 * n, 2, 64), rows(gen, 2 * n, 2, 64)
    if what != "ordinary":
        k[:], v[:] = {"zero": (0.0, -0.0), "tiny": (1e-30, -1e-25), "nan": (float("nan"),) * 2}[what]
    odd = cache.write(k, v, i32([[0], [2]]), i32([5 + n, 9 + n]), i32([0, n, 2 * n]), n)
    assert odd == (what == "nan")
    assert pkv.get_error() == (pkv.ERR_NONFINITE if odd else 0)
    cache.check()
    for scales in cache.gpu[2:]:
        held = scales[[0, 2]]
        assert torch.isfinite(held).all() and (held >= 2.0 ** -60).all()
