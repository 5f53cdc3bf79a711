"""What the int8 and page-copy calls refuse, through the C ABI and the binding,
before anything reaches a GPU (the pointers are never followed)."""
import ctypes

import numpy as np
import pytest
import torch

from paged_kv_cache_43_gb300 import build, pkv

E_NULL, E_DTYPE, E_SHAPE, E_GQA, E_ALIGN, E_META = -1, -2, -3, -4, -6, -8
P = 1 << 20   # an aligned address that nothing reads


@pytest.fixture(scope="module")
def lib():
    build.build()
    return pkv.load()


def desc(**kw):
    d = dict(num_blocks=10, block_size=16, num_kv_heads=2, head_size=64, dtype=pkv.PKV_INT8)
    d.update(kw)
    return pkv.CacheDesc(*d.values())


def meta(**kw):
    m = dict(num_seqs=1, num_tokens=1, num_q_heads=4, block_table_stride=2, max_query_len=1,
             max_context_len=20, num_decode_seqs=-1, sliding_window=0, kv_split_tokens=0)
    m.update(kw)
    return pkv.AttnMeta(*m.values())


def write(lib, d=None, m=None, **at):
    args = dict.fromkeys("k v bt cl qsl kc vc ks vs".split(), P)
    args.update(at)
    return lib.pkv_write_int8(*args.values(), ctypes.byref(d or desc()), ctypes.byref(m or meta()),
                              None)


def attend(lib, d=None, m=None, ws=None, **at):
    args = dict.fromkeys("out q kc vc bt cl qsl".split(), P)
    scales = dict(ks=P, vs=P)
    for n, x in at.items():
        (scales if n in scales else args)[n] = x
    return lib.pkv_attention_int8(*args.values(), 0.1, *scales.values(),
                                  ctypes.byref(d or desc()), ctypes.byref(m or meta()), ws, 0, None)


@pytest.mark.parametrize("call", [write, attend])
def test_descriptions(lib, call):
    for bad in (pkv.PKV_BF16, pkv.PKV_F32, pkv.PKV_FP8_E4M3, 9):
        assert call(lib, d=desc(dtype=bad)) == E_DTYPE
    for bad in (dict(block_size=32), dict(head_size=96), dict(num_kv_heads=0),
                dict(num_blocks=-1), dict(num_blocks=1 << 28)):
        assert call(lib, d=desc(**bad)) == E_SHAPE
    assert call(lib, m=meta(num_q_heads=5)) == E_GQA
    for bad in (dict(num_seqs=-1), dict(num_tokens=-1), dict(max_query_len=-1),
                dict(block_table_stride=0), dict(num_decode_seqs=2), dict(sliding_window=-1),
                dict(kv_split_tokens=100), dict(max_context_len=-1)):
        assert call(lib, m=meta(**bad)) == E_META


@pytest.mark.parametrize("call,names", [(write, "k v bt cl qsl kc vc ks vs"),
                                        (attend, "out q kc vc bt cl qsl ks vs")])
def test_pointers(lib, call, names):
    for n in names.split():
        assert call(lib, **{n: None}) == E_NULL, n
        assert call(lib, **{n: P + 2}) == E_ALIGN, n
    # nothing to do: no pointer is looked at
    for m in (meta(num_seqs=0, num_tokens=0), meta(num_tokens=0)):
        assert call(lib, m=m, **dict.fromkeys(names.split(), None)) == 0


def test_other_calls_refuse_an_int8_cache(lib):
    d, m = desc(), meta()
    r, rm = ctypes.byref(d), ctypes.byref(m)
    assert lib.pkv_write(P, P, P, 1, P, P, r, None) == E_DTYPE
    assert lib.pkv_write_fp8(P, P, P, 1, P, P, P, P, r, None) == E_DTYPE
    assert lib.pkv_attention_fp8(P, P, P, P, P, P, P, 0.1, P, P, r, rm, None, 0, None) == E_DTYPE
    assert lib.pkv_attention_cascade_fp8(P, P, P, P, P, P, P, 0.1, 1, P, P, r, rm, None, 0,
                                         None) == E_DTYPE
    none = ctypes.c_size_t(-1).value
    assert lib.pkv_attention_int8_workspace_size(ctypes.byref(desc(dtype=1)), rm) == none
    assert lib.pkv_attention_int8_workspace_size(r, ctypes.byref(meta(num_q_heads=3))) == none


def copy(lib, pairs, nb=4, page=(64,), bases=(P,), n=None):
    p = np.ascontiguousarray(pairs, dtype=np.int32)
    k = len(bases)
    return lib.pkv_copy_blocks((ctypes.c_void_p * k)(*bases), (ctypes.c_int64 * k)(*page), k, nb,
                               p.ctypes.data, len(p) if n is None else n, None)


def test_copy_refusals(lib):
    for bad in ((0, 4), (-1, 0), (4, 0), (0, -1)):
        assert copy(lib, [(0, 1), bad]) == E_SHAPE
    assert copy(lib, [(0, 1)], page=(0,)) == E_SHAPE
    assert copy(lib, [(0, 1)], page=((1 << 30) + 4,)) == E_SHAPE
    assert copy(lib, [(0, 1)], page=(66,)) == E_ALIGN
    assert copy(lib, [(0, 1)], bases=(P + 2,)) == E_ALIGN
    assert copy(lib, [(0, 1)], page=(64, 64), bases=(P, None)) == E_NULL
    assert copy(lib, [(0, 1)], n=-1) == E_SHAPE
    assert lib.pkv_copy_blocks(None, None, 1, 4, P, 1, None) == E_NULL
    assert lib.pkv_copy_blocks(None, None, 0, 4, None, 1, None) == 0
    assert lib.pkv_copy_blocks(P, P, 1, 4, None, 0, None) == 0


def test_binding_refuses_host_tensors():
    c = torch.zeros(4, 16, 2, 64, dtype=torch.int8)
    s = torch.zeros(4, 2)
    i = torch.zeros(2, dtype=torch.int32)
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(pkv.PkvError, match="CUDA"):
        pkv.write_int8(x, x, i[None], i[:1], i, c, c, s, s, max_query_len=1)
    with pytest.raises(pkv.PkvError, match="CUDA"):
        pkv.attention_int8(x, x, c, c, i[None], i[:1], i, 1.0, s, s, max_query_len=1,
                           max_context_len=1)
    with pytest.raises(pkv.PkvError, match="CUDA"):
        pkv.copy_blocks([c], [(0, 1)])
    for bad in ([0, 1, 2], [(0.0, 1.0)], [(0, 2 ** 32)], [(-1, 0)]):
        with pytest.raises(pkv.PkvError, match="pairs"):
            pkv.copy_blocks([c], np.asarray(bad))
