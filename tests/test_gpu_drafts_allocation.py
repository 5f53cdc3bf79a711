"""What the drafted-step calls get from the allocator: nothing, but for the tree's workspace where none is given;
nothing in the library itself."""
import pytest
import torch

from drafts import Batch
from paged_kv_cache_43_gb300 import build, pkv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    pkv.load()
    pkv.get_error(clear=True)


def device_and_torch():
    torch.cuda.synchronize()
    return torch.cuda.mem_get_info()[0], torch.cuda.memory_stats()["allocation.all.allocated"]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn, torch.float32])
@pytest.mark.parametrize("n", [4, 40])
def test_calls_allocate_nothing(dtype, n):
    b = Batch([n, n], [1500, 90], hq=8, hkv=2, d=128, dtype=dtype).cuda()
    g, T = b.g, 2 * n
    kw = dict(max_query_len=n, max_context_len=b.max_L)
    ws = torch.empty(max(pkv.workspace_size_tree(g["k"], pkv.attn_meta(g["q"], g["bt"], g["cl"], **kw)), 256),
                     dtype=torch.uint8, device="cuda")
    out = torch.empty_like(g["q"])
    row = b.row
    rows = dict(q_out=torch.empty_like(g["q"]), q=g["q"], k=torch.randn(T, 2, 128, device="cuda").to(row),
                v=torch.randn(T, 2, 128, device="cuda").to(row),
                positions=torch.arange(T, device="cuda"), cos_sin=torch.zeros(T, 64, device="cuda"),
                slot_mapping=torch.full((T,), -1, device="cuda"), k_cache=g["k"], v_cache=g["v"])
    scales = [torch.ones(2, device="cuda") for _ in range(2)] if b.fp8 else []
    k_out = torch.empty_like(rows["k"])
    path = torch.arange(n, dtype=torch.int32, device="cuda").repeat(2, 1)
    count = torch.tensor([n, 1], dtype=torch.int32, device="cuda")
    new = torch.empty_like(g["cl"])

    def step():
        (pkv.rope_write_fp8 if b.fp8 else pkv.rope_write)(*rows.values(), *scales)
        pkv.rope(rows["q_out"], k_out, rows["q"], rows["k"], rows["positions"], rows["cos_sin"])
        b.call(out, workspace=ws)
        pkv.accept_drafts([g["k"], g["v"]], g["bt"], g["cl"], g["qsl"], path, count, new_context_lens=new)

    step()
    before = device_and_torch()
    for _ in range(20):
        step()
    assert device_and_torch() == before
    assert pkv.get_error() == 0
    b.check(out)
